// Eight-wave "ping-pong" GEMM for 16-bit and 8-bit K-contiguous operands
// (TN) on gfx950: two waves on every SIMD, in two groups of four, take
// turns.  While one group issues nothing but MFMAs, the other reads its
// fragments for its next turn from LDS and (group 0) issues the global ->
// LDS copies; at each workgroup barrier the roles swap.  A SIMD's MFMA pipe
// therefore never waits for a fragment read, a copy issue or a wave that is
// late to a barrier while the other wave has work ("An Educational GEMM
// Ladder for Helios GPUs", Level 12, two waves per SIMD; its summary names
// the eight-wave ping-pong as the MI355X schedule).
//
// Operation and (P, Q, D) mapping as gemm_mfma.hpp: D[p][q] = sum_k P(p,k)
// Q(q,k), stored at C[q*ldc + p].  Block tile 256 x 256; SIMD s owns the
// 128 x 128 quadrant (p half s / 2, q half s % 2) and its two waves split
// it along q: the wave of group g computes 128 (p) x 64 (q) as 8 x 4 MFMA
// tiles of 16 x 16 (x 32 for FP16/BF16, x 128 for FP8) with 128
// accumulator registers, which leaves 128 for the fragments of one whole
// stage (96) and addressing at two waves per SIMD.
//
// LDS: 128 bytes of k per row per stage, XOR-swizzled as in the four-wave
// kernel; two slots for the P rows of a stage (256 x 128 B, 32 KiB each) and
// three for the Q rows (32 KiB each): 160 KiB.  Copies are direct global ->
// LDS through buffer descriptors (rows past the edge and k past K read zero).
//
// Per stage t each wave runs R(t) (read its fragments of stage t), a
// barrier, C(t) (all MFMAs of the stage), a wait for its own copies, a
// barrier; group 1 runs one barrier behind group 0, so that one group's C
// overlaps the other's R.  Ahead of its R(t), group 0 copies the P rows of
// stage t + 1 and group 1 the Q rows of stage t + 2, each into the slot that
// both groups finished reading a barrier earlier; each copy has two turns
// (its issuer's R and C) to land before the barrier that publishes it, and
// every turn carries half a stage of copies (32 KiB), which keeps the copy
// path at about half of what it delivers per CU.  The barriers wait only for
// LDS reads, so copies stay in flight across them.
//
// FP8 with factors of blocks of 128 k (Op::BLK, see OpB8): a stage is one block, so
// each MFMA starts from zero and the vector unit adds its result, times the factors,
// two MFMAs later; the stage's factors are loaded ahead of its copies.  The partial
// results take the registers of the last Q tile (BLK 2: half the P tiles), which is
// read during C.  8192^3 in BF16 401 us, 2.74 PFLOP/s, where the MFMAs alone (OpFP8)
// take 375, both at the power limit; with P row by row (BLK 2, four products more an
// MFMA: the vector unit is then as busy as the matrix pipe) 4096 x 4096 x 8192 130 us
// for 103; NN (PKM) 8192^3 421.
#pragma once

#include "common.hpp"
#include "gemm_mfma.hpp"

namespace dg {

template <class Op, int BQ_ = 256>
struct PpCfg {
  static constexpr int BP = 256, BQ = BQ_;
  static constexpr int NW = 8, NT = 512, NSIMD = 4;
  static constexpr int E = Op::ELEM, FC = Op::FC;
  static constexpr int ROWB = 128;                 // bytes of k per LDS row per stage
  static constexpr int BK = ROWB / E;              // k per stage
  static constexpr int CPE = 16 / E;               // elements per 16-byte chunk
  static constexpr int P_LDS = BP * ROWB;          // one P slot
  static constexpr int Q_LDS = BQ * ROWB;          // one Q slot
  static constexpr int Q_BASE = 2 * P_LDS;         // Q slots after the two P slots
  static constexpr int QSEG = BQ / 8 / NSIMD;      // copies per wave per stage of its operand
  static constexpr int PSEG = BP / 8 / NSIMD;
  // BQ 192: group 1 makes as many copies as group 0, the last of them zeros that go here.
  static constexpr int SPARE = 2 * P_LDS + 3 * Q_LDS;
  static constexpr int LDS = SPARE + (PSEG - QSEG) * NSIMD * 1024;
  static constexpr int WTP = BP / 2, WTQ = BQ / 4; // wave tile
  static constexpr int MT = 16;
  static constexpr int KI = E == 2 ? 32 : 128;     // k per MFMA
  static constexpr int TP = WTP / MT, TQ = WTQ / MT;
  static constexpr int KSTEPS = BK / KI;
  static constexpr int CPK = KI * E / 16;          // 16-byte chunks of k per k-step
  static_assert(LDS <= kLdsLimit, "LDS budget");
  static_assert((TP / (Op::OE == 4 ? 2 : 1)) * MT * Op::OE == 256, "staged epilogue rows of 256 bytes");
  static_assert(WTQ * 256 * NW <= LDS, "epilogue staging fits the stage buffers");
};

// KT: K ends inside a stage, so the copies carry per-lane tail masks.
// GA: row q of Q is row gt.index[q] of its storage.
// PKM: P is contiguous along p (NN's B; BLK 1 only): LDS rows of k, 256 bytes of p,
// swizzled and read with transposing reads as in the four-wave kernel.
// BQ 192 (BLK 1, PKM): three MFMA tiles a wave along q for four, where one round of
// those covers C.
template <class Op, bool KT, class TileOf, bool GA = false, bool PKM = false, int BQ_ = 256>
__device__ __forceinline__ void gemm_pp_body(const GemmArgs& a, TileOf tile_of, const Gather& gt = Gather{}) {
  using Cfg = PpCfg<Op, BQ_>;
  static_assert(BQ_ == 256 || (BQ_ == 192 && Op::BLK == 1 && !GA), "tiles of 192 rows are built for BLK 1");
  constexpr int E = Cfg::E, FC = Cfg::FC, ROWB = Cfg::ROWB, BK = Cfg::BK, CPE = Cfg::CPE;
  constexpr int TP = Cfg::TP, TQ = Cfg::TQ, MT = Cfg::MT, CPK = Cfg::CPK, KSTEPS = Cfg::KSTEPS;

  __shared__ __attribute__((aligned(1024))) char smem[Cfg::LDS];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave >> 2, simd = wave & 3;
  const int wp = simd >> 1, wq = simd & 1;
  const int64_t K = a.K;
  const int nst = (int)((K + BK - 1) / BK);
  const uint32_t kbytes16 = (uint32_t)(((K * E) + 15) & ~(int64_t)15);
  const int64_t ntiles = a.tiles_p * a.tiles_q;
  const int64_t tile = tile_of();
  if (tile >= ntiles) return;   // (the whole workgroup)

  // (BLK has no register to spare for what the stamps and the epilogue would keep
  // across the loop: no stamps, and the lane computed afresh.)
  auto stamp = [&](int at) {
    if constexpr (Op::BLK != 0) return;
    if (a.trace != nullptr && tid == 0 && tile < a.trace_n) {
      unsigned long long* t = a.trace + 4 * tile + at;
      t[0] = __builtin_amdgcn_s_memtime();
      t[1] = __builtin_amdgcn_s_memrealtime();
    }
  };
  stamp(0);

  int64_t tp, tq;
  tile_map(a.tiles_p, a.tiles_q, a.group, tile, &tp, &tq);
  const int64_t p0 = tp * Cfg::BP, q0 = tq * Cfg::BQ;
  const int64_t qrows = (a.Qn - q0) < Cfg::BQ ? (a.Qn - q0) : Cfg::BQ;
  const int64_t prows = (a.Pn - p0) < Cfg::BP ? (a.Pn - p0) : Cfg::BP;
  const char* qsrc = GA ? a.Q : a.Q + q0 * a.ldq;
  const char* psrc = PKM ? a.P + p0 : a.P + p0 * a.ldp;
  const uint32_t qn = (uint32_t)(((GA ? gt.rows : qrows) - 1) * a.ldq) + kbytes16;
  const uint32_t pn = PKM ? (K > 0 ? (uint32_t)((K - 1) * a.ldp) + (uint32_t)((prows + 15) & ~(int64_t)15) : 0u)
                          : (uint32_t)((prows - 1) * a.ldp) + kbytes16;

  // ---- copies: P rows by group 0, Q rows by group 1 ----
  // One copy instruction fills one 1 KiB LDS segment = 8 rows of 128 bytes;
  // the wave on SIMD s fills segments 4i + s of its operand's slot.  Lane l
  // lands at byte 16 l: row 8 (4i + s) + l / 8, physical chunk l % 8, which
  // holds logical chunk (l % 8) ^ key(row), key(row) = (row / 2) mod 8 =
  // (4 (s % 2) + l / 16) mod 8.  Rows past the edge need no test: their
  // offsets are at least rows * ld >= num_records.
  const int dkc = (lane & 7) ^ ((4 * (simd & 1) + (lane >> 4)) & 7);
  // BLK 2 changes the operands' parts: Q has two slots and is copied by group 0, P
  // three, so that P tiles can be read late.
  constexpr bool PLATE = Op::BLK == 2;
  static_assert(!(PLATE && GA), "rows behind an index are group 1's");
  const bool cp = (grp == 0) != PLATE;   // this group copies P
  const char* csrc = cp ? psrc : qsrc;
  const uint32_t cn = cp ? pn : qn;
  const int64_t cld = cp ? a.ldp : a.ldq;
  const uint32_t cv0 = (uint32_t)((8 * simd + (lane >> 3)) * cld + dkc * 16);
  const uint32_t cstep = (uint32_t)(32 * cld);
  [[maybe_unused]] uint32_t cvi[Cfg::QSEG];   // GA: offsets of the copies, one by one
  if constexpr (GA) {
#pragma unroll
    for (int i = 0; i < Cfg::QSEG; ++i)
      cvi[i] = grp == 0 ? (Op::BLK != 0 ? cv0 : cv0 + i * cstep)
                        : gather_row(gt, q0 + 8 * (i * Cfg::NSIMD + simd) + (lane >> 3), a.Qn, a.ldq, dkc * 16);
  }
  static_assert(!PLATE || Cfg::P_LDS == Cfg::Q_LDS, "either operand fits either's slots");
  // Where copy i of a stage goes (BQ 192: group 1's last ones are none).
  auto seg = [&](char* sb, int i) {
    return (i >= Cfg::QSEG && !cp ? smem + Cfg::SPARE + (i - Cfg::QSEG) * Cfg::NSIMD * 1024
                                  : sb + i * Cfg::NSIMD * 1024) + simd * 1024;
  };
  auto some = [&](int i, int left) { return i >= Cfg::QSEG && !cp ? 0u : (uint32_t)(left > 0 ? left : 0); };
  // PKM: copy i of the wave on SIMD s fills LDS rows k = 16 i + 4 s .. + 3; lane l
  // lands at row l / 16 of them, physical chunk l % 16 of 16 bytes, which holds
  // logical chunk ^ key(k), key(k) = 2 (k mod 8) + (k / 16) mod 2: two offsets, for
  // even and odd i.  (A read's lanes take sixteen bytes of eight k and of eight more
  // sixteen further: all banks once.)
  static_assert(!PKM || (Op::BLK == 1 && !GA), "built for factors of 128 rows");
  [[maybe_unused]] uint32_t cvk[2] = {cv0, cv0};
  if constexpr (PKM) {
    if (cp) {
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int c = (lane & 15) ^ (2 * (4 * (simd & 1) + (lane >> 4)) + o);
        cvk[o] = (uint32_t)((4 * simd + (lane >> 4)) * a.ldp + c * 16);
      }
    }
  }
  auto two_slot = [&](int t) { return smem + (t & 1) * Cfg::P_LDS; };
  auto three_slot = [&](int t) { return smem + Cfg::Q_BASE + (t % 3) * Cfg::Q_LDS; };
  auto p_slot = [&](int t) { return PLATE ? three_slot(t) : two_slot(t); };
  auto q_slot = [&](int t) { return PLATE ? two_slot(t) : three_slot(t); };
  // Stage t of this wave's operand into its slot.
  auto slot_of = [&](int t) { return grp == 0 ? (t & 1) * Cfg::P_LDS : Cfg::Q_BASE + (t % 3) * Cfg::Q_LDS; };
  auto copies = [&](int t, int slot) {
    char* sb = Op::BLK != 0 ? smem + slot : (grp == 0 ? two_slot(t) : three_slot(t));
    const uint32_t at = (uint32_t)t * ROWB;
    // (BLK copies zeros past the last stage: with a branch around its copies the
    // compiler waits for all of them where it waits for the factors.)
    const __amdgpu_buffer_rsrc_t r = make_rsrc(csrc + at, cn - at);
    uint32_t kill = 0;
    if constexpr (KT) {
      // Chunks at or past K read zero (bit 31 puts the offset past num_records).
      const int64_t rem64 = K - (int64_t)t * BK;
      const int rem = (int)(rem64 < BK ? rem64 : BK);
      kill = dkc * CPE >= rem ? kOobOffset : 0u;
    }
    static_assert(Cfg::PSEG == Cfg::QSEG || Op::BLK != 0, "both operands take the same number of copies");
    if constexpr (Op::BLK != 0) {
      // One offset register for all copies (eight for rows behind an index): the
      // descriptor moves down the rows instead.
      // (Signed, below 2^31: an unsigned saturating difference would go through
      // vector registers, and each copy through a loop over them.)
      if constexpr (PKM) {
        // (128 rows of P are below 2^31 bytes.)
        const int atk = t * (cp ? BK * (int)a.ldp : ROWB), step = cp ? 16 * (int)a.ldp : (int)cstep;
        const int leftk = t >= nst ? 0 : (int)cn - atk;
        const char* src = csrc + (t >= nst ? 0 : atk);
#pragma unroll
        for (int i = 0; i < Cfg::PSEG; ++i) {
          const __amdgpu_buffer_rsrc_t ri = make_rsrc(src + i * step, some(i, leftk - i * step));
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              ri, (__attribute__((address_space(3))) void*)seg(sb, i), 16,
              cvk[i & 1] | (cp ? 0u : kill), 0, 0, 0);
        }
        return;
      }
      const int left = t >= nst ? 0 : (int)(cn - at);
#pragma unroll
      for (int i = 0; i < Cfg::PSEG; ++i) {
        const int down = GA && grp == 1 ? 0 : i * (int)cstep;
        const __amdgpu_buffer_rsrc_t ri = make_rsrc(csrc + at + down, some(i, left - down));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            ri, (__attribute__((address_space(3))) void*)seg(sb, i), 16,
            (GA ? cvi[i] : cv0) | kill, 0, 0, 0);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < Cfg::PSEG; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          r, (__attribute__((address_space(3))) void*)(sb + (i * Cfg::NSIMD + simd) * 1024), 16,
          (GA ? cvi[i] : cv0 + i * cstep) | kill, 0, 0, 0);
  };

  // Any K (integers): the part of Q's chunks at and past K becomes zero once
  // this wave's copies of the last stage have landed, before the barrier that
  // publishes them.
  constexpr bool TRIM = Op::TRIM && KT && Op::BLK == 0;
  auto trim = [&](int t) {
    const int left = (int)((K - (int64_t)t * BK) - dkc * CPE) * E;   // bytes of this lane's chunk below K
    if (grp == 0 || left <= 0 || left >= 16) return;
    char* sb = q_slot(t);
#pragma unroll
    for (int i = 0; i < Cfg::QSEG; ++i) {
      u32x4* c = (u32x4*)(sb + (i * Cfg::NSIMD + simd) * 1024 + lane * 16);
      *c = mask_tail(*c, left);
    }
  };

  // BLK: the same for this wave's copies of stage t, of either operand (E4M3 has NaN,
  // which zeros do not cancel; PKM: P's rows past K read zero), if that is the last.
  // Assembly with a branch of its own: with one of the compiler's in the loop it moves
  // the accumulations past it, and 94 registers to memory, and with a last stage behind
  // the loop, its fragments masked, 8191 x 8189 x 8191 took 443 us, so 427.
  [[maybe_unused]] const int trimmed = __builtin_amdgcn_readfirstlane(K % CPE != 0 && !(PKM && cp) ? nst - 1 : -1);
  [[maybe_unused]] const int rem4 = __builtin_amdgcn_readfirstlane(4 * (int)(K - (int64_t)(nst - 1) * BK));
  auto trim_last = [&](int t, int slot) {
    if constexpr (Op::BLK != 0 && KT) {
      static_assert(Cfg::PSEG == 8 && Cfg::NSIMD == 4, "eight copies, 4096 bytes apart (the last two: see seg)");
      const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem + simd * 1024 + lane * 16;
      const uint32_t at = base + slot, at6 = Cfg::PSEG > Cfg::QSEG && !cp ? base + Cfg::SPARE : at + 6 * 4096;
      uint32_t m0, m1, m2, m3, q, u;
      // Word d of a chunk keeps n = clamp(left - 4 d, 0, 4) bytes, left those below K: all
      // ones shifted down twice by 16 - 4 n = clamp(64 dkc - 4 rem + 16 (d + 1), 0, 16).
      asm volatile(
          "s_cmp_lg_u32 %6, %11\n\ts_cbranch_scc1 .Ltrim%=\n\t"
          "v_lshlrev_b32 %4, 6, %8\n\tv_subrev_u32 %4, %7, %4\n\t"
          "v_add_u32 %0, 16, %4\n\tv_med3_i32 %0, %0, 0, 16\n\tv_lshrrev_b32 %5, %0, -1\n\tv_lshrrev_b32 %0, %0, %5\n\t"
          "v_add_u32 %1, 32, %4\n\tv_med3_i32 %1, %1, 0, 16\n\tv_lshrrev_b32 %5, %1, -1\n\tv_lshrrev_b32 %1, %1, %5\n\t"
          "v_add_u32 %2, 48, %4\n\tv_med3_i32 %2, %2, 0, 16\n\tv_lshrrev_b32 %5, %2, -1\n\tv_lshrrev_b32 %2, %2, %5\n\t"
          "v_add_u32 %3, 64, %4\n\tv_med3_i32 %3, %3, 0, 16\n\tv_lshrrev_b32 %5, %3, -1\n\tv_lshrrev_b32 %3, %3, %5\n\t"
          "ds_and_b32 %9, %0 offset:0\n\tds_and_b32 %9, %1 offset:4\n\t"
          "ds_and_b32 %9, %2 offset:8\n\tds_and_b32 %9, %3 offset:12\n\t"
          "ds_and_b32 %9, %0 offset:4096\n\tds_and_b32 %9, %1 offset:4100\n\t"
          "ds_and_b32 %9, %2 offset:4104\n\tds_and_b32 %9, %3 offset:4108\n\t"
          "ds_and_b32 %9, %0 offset:8192\n\tds_and_b32 %9, %1 offset:8196\n\t"
          "ds_and_b32 %9, %2 offset:8200\n\tds_and_b32 %9, %3 offset:8204\n\t"
          "ds_and_b32 %9, %0 offset:12288\n\tds_and_b32 %9, %1 offset:12292\n\t"
          "ds_and_b32 %9, %2 offset:12296\n\tds_and_b32 %9, %3 offset:12300\n\t"
          "ds_and_b32 %9, %0 offset:16384\n\tds_and_b32 %9, %1 offset:16388\n\t"
          "ds_and_b32 %9, %2 offset:16392\n\tds_and_b32 %9, %3 offset:16396\n\t"
          "ds_and_b32 %9, %0 offset:20480\n\tds_and_b32 %9, %1 offset:20484\n\t"
          "ds_and_b32 %9, %2 offset:20488\n\tds_and_b32 %9, %3 offset:20492\n\t"
          "ds_and_b32 %10, %0 offset:0\n\tds_and_b32 %10, %1 offset:4\n\t"
          "ds_and_b32 %10, %2 offset:8\n\tds_and_b32 %10, %3 offset:12\n\t"
          "ds_and_b32 %10, %0 offset:4096\n\tds_and_b32 %10, %1 offset:4100\n\t"
          "ds_and_b32 %10, %2 offset:4104\n\tds_and_b32 %10, %3 offset:4108\n\t"
          "s_waitcnt lgkmcnt(0)\n.Ltrim%=:"
          : "=&v"(m0), "=&v"(m1), "=&v"(m2), "=&v"(m3), "=&v"(q), "=&v"(u)
          : "s"(__builtin_amdgcn_readfirstlane(t)), "s"(rem4), "v"(dkc), "v"(at), "v"(at6), "s"(trimmed)
          : "scc", "memory");
    }
  };

  // ---- fragments ----
  // Lane l holds row l % 16 of its P and Q tiles; lane group l / 16 selects
  // its k: 16-bit, chunk 4 kk + l / 16 of the stage row (8 k); FP8, chunks
  // l / 16 and l / 16 + 4 (16 k each), which keeps the order of the
  // four-wave kernel's FP8 fragments.
  const int lr = lane & 15, lg = lane >> 4;
  const int sw = (lr >> 1) & 7;
  const uint32_t pf = (uint32_t)((wp * Cfg::WTP + lr) * ROWB);
  const uint32_t qf = (uint32_t)((wq * (Cfg::BQ / 2) + grp * Cfg::WTQ + lr) * ROWB);
  // BLK reads its last Q tile (GA: two; BLK 2: half the P tiles) during its C
  // turn, into the first one's registers (the slot, one of three, is not written
  // before the next turn but one).
  constexpr int NFA = PLATE ? TP / 2 : TP;
  constexpr int NFB = PLATE || Op::BLK == 0 || Cfg::BQ < 256 ? TQ : (GA ? TQ - 2 : TQ - 1);
  u32x4 fa[KSTEPS][NFA][FC], fb[KSTEPS][NFB][FC];
  // PKM: P tile i by four transposing reads (see the four-wave kernel): lane l
  // addresses eight p of k row 16 (l / 16) + (l % 16) / 2, whose key no lane changes.
  auto read_turned = [&](const char* sp, int i) {
    if constexpr (PKM) {
      typedef int i32x2v __attribute__((ext_vector_type(2)));
      const int key = (lr & ~1) + (lg & 1);
      const char* src = sp + (16 * lg + (lr >> 1)) * 256 + (((8 * wp + i) ^ key) << 4) + (lr & 1) * 8;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const i32x2v v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2v*)(src + (x >> 1) * 64 * 256 + (x & 1) * 8 * 256));
        fa[0][i][x >> 1][2 * (x & 1)] = (unsigned)v[0];
        fa[0][i][x >> 1][2 * (x & 1) + 1] = (unsigned)v[1];
      }
    }
  };
  auto read_frags = [&](int t) {
    const char* sp = p_slot(t);
    const char* sq = q_slot(t);
    if constexpr (PKM) {
#pragma unroll
      for (int i = 0; i < NFA; ++i) read_turned(sp, i);
    }
#pragma unroll
    for (int kk = 0; kk < KSTEPS; ++kk)
#pragma unroll
      for (int f = 0; f < FC; ++f) {
        const uint32_t off = (uint32_t)(((kk * CPK + f * (CPK / FC) + lg) ^ sw) << 4);
#pragma unroll
        for (int j = 0; j < NFB; ++j) fb[kk][j][f] = *(const u32x4*)(sq + qf + j * MT * ROWB + off);
        if constexpr (!PKM) {
#pragma unroll
          for (int i = 0; i < NFA; ++i) fa[kk][i][f] = *(const u32x4*)(sp + pf + i * MT * ROWB + off);
        }
      }
  };

  typename Op::Acc16 acc[TP][TQ];
#pragma unroll
  for (int i = 0; i < TP; ++i)
#pragma unroll
    for (int j = 0; j < TQ; ++j) acc[i][j] = typename Op::Acc16{0, 0, 0, 0};
  // BLK: this stage's factors, loaded ahead of its copies and fragments and
  // used a turn later: of the wave's 128 p one (a scalar) or (BLK 2) one per lane
  // and 64 of them, of q one per lane and MFMA tile.
  constexpr int NPF = Op::BLK == 2 ? TP / 4 : 1;
  [[maybe_unused]] float fq[TQ], fp[NPF];
  [[maybe_unused]] uint32_t fpo = 0, fpn = 0;
  constexpr bool EACH = GA || Cfg::BQ % 128 != 0;   // an offset for each of q's MFMA tiles
  [[maybe_unused]] uint32_t fqo[EACH ? TQ : 1], fqstep = 0;
  [[maybe_unused]] uint32_t fqn = 0;
  [[maybe_unused]] const float* fqs = nullptr;
  [[maybe_unused]] const float* fps = nullptr;
  if constexpr (Op::BLK != 0) {
    if constexpr (Op::BLK == 2) {
      fps = a.sp + p0 * a.sp_r;
      fpn = (uint32_t)(((prows - 1) * a.sp_r + 1) * 4);
      fpo = (uint32_t)((wp * Cfg::WTP + factor_row(lane)) * a.sp_r * 4);
    } else {
      const int64_t pb = p0 + wp * Cfg::WTP < a.Pn ? p0 + wp * Cfg::WTP : a.Pn - 1;
      fps = a.sp + (pb >> a.sp_shift) * a.sp_r;
    }
    fqs = GA ? a.sq : a.sq + (q0 >> a.sq_shift) * a.sq_r;
    const int qpast = EACH && !GA ? (int)(q0 & ((1 << a.sq_shift) - 1)) : 0;   // rows of the tile's first factor before it
    const int64_t rows = GA ? gt.rows : (qpast + qrows + (1 << a.sq_shift) - 1) >> a.sq_shift;
    fqn = (uint32_t)(((rows - 1) * a.sq_r + 1) * 4);
    const int q = wq * (Cfg::BQ / 2) + grp * Cfg::WTQ + lr;
    if constexpr (GA) {
#pragma unroll
      for (int j = 0; j < TQ; ++j) fqo[j] = gather_row(gt, q0 + q + j * MT, a.Qn, a.sq_r * 4, 0);
    } else if constexpr (EACH) {
#pragma unroll
      for (int j = 0; j < TQ; ++j) fqo[j] = (uint32_t)(((qpast + q + j * MT) >> a.sq_shift) * a.sq_r * 4);
    } else {
      // (The wave's 64 rows share a factor of 128.)
      fqo[0] = (uint32_t)((q >> a.sq_shift) * a.sq_r * 4);
      fqstep = a.sq_shift == 0 ? (uint32_t)(MT * a.sq_r * 4) : 0u;
    }
  }
  auto factors = [&](int t) {
    if constexpr (Op::BLK != 0) {
      if constexpr (Op::BLK == 2) {
        const __amdgpu_buffer_rsrc_t r = make_rsrc(fps + t * a.sp_k, fpn);
#pragma unroll
        for (int i = 0; i < NPF; ++i)
          fp[i] = __builtin_bit_cast(
              float, __builtin_amdgcn_raw_buffer_load_b32(r, (int)(fpo + i * (uint32_t)(64 * a.sp_r * 4)), 0, 0));
      } else {
        typedef const __attribute__((address_space(4))) float* Scalar;
        fp[0] = *(Scalar)(uintptr_t)(fps + t * a.sp_k);
      }
      const __amdgpu_buffer_rsrc_t r = make_rsrc(fqs + t * a.sq_k, fqn);
#pragma unroll
      for (int j = 0; j < TQ; ++j)
        fq[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                              r, (int)(EACH ? fqo[EACH ? j : 0] : fqo[0] + j * fqstep), 0, 0));
      // (Ahead of the copies: waiting for them then waits for no copy.)
      asm volatile("" ::: "memory");
    }
  };
  // BLK: the stage's MFMAs, Q tile by Q tile (BLK 2: P tile by P tile, whose
  // factors then serve TQ results), each result added two MFMAs later.
  auto compute_blocks = [&](int t) {
    if constexpr (Op::BLK != 0) {
      static_assert(KSTEPS == 1, "a stage is a block");
      constexpr int RING = 3, N = TP * TQ, IN = PLATE ? TQ : TP;   // IN: MFMAs of an outer tile
      auto ti = [](int u) { return PLATE ? u / IN : u % IN; };
      auto tj = [](int u) { return PLATE ? u % IN : u / IN; };
      f32x4 part[RING];
      [[maybe_unused]] f32x4 rows;
      float f[TQ];
#pragma unroll
      for (int j = 0; j < TQ; ++j) f[j] = PLATE ? fq[j] : fq[j] * fp[0];
#pragma unroll
      for (int u = 0; u < N + RING - 1; ++u) {
        if (u < N) part[u % RING] = Op::block(fa[0][ti(u) % NFA], fb[0][tj(u) % NFB]);
        // The registers of outer tile o - 1 are free: they take tile NF + o - 1.
        const int o = u / IN;
        if (u % IN == 0 && o > 0 && o <= (PLATE ? TP - NFA : TQ - NFB)) {
          const char* src = PLATE ? p_slot(t) + pf + (NFA + o - 1) * MT * ROWB : q_slot(t) + qf + (NFB + o - 1) * MT * ROWB;
#pragma unroll
          for (int c = 0; c < FC; ++c) {
            const u32x4 v = *(const u32x4*)(src + (uint32_t)(((c * (CPK / FC) + lg) ^ sw) << 4));
            if constexpr (PLATE) fa[0][o - 1][c] = v;
            else fb[0][o - 1][c] = v;
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        const int w = u - (RING - 1);
        if (w >= 0) {
          if constexpr (PLATE) {
            if (w % IN == 0) rows = tile_factors(fp[ti(w) / 4], ti(w));
            add_block(acc[ti(w)][tj(w)], part[w % RING], f[tj(w)], rows);
          } else {
            add_block(acc[ti(w)][tj(w)], part[w % RING], f[tj(w)]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  auto compute = [&](int t) {
    if constexpr (Op::BLK != 0) {
      compute_blocks(t);
      return;
    }
#pragma unroll
    for (int kk = 0; kk < KSTEPS; ++kk)
#pragma unroll
      for (int j = 0; j < TQ; ++j)
#pragma unroll
        for (int i = 0; i < TP; ++i) acc[i][j] = Op::mma16(fa[kk][i], fb[kk][j], acc[i][j]);
  };
  // Workgroup barrier after this wave's LDS reads have returned; global ->
  // LDS copies stay in flight across it (a fence on LDS would also wait for
  // them, as they write LDS).  Written as assembly with a memory clobber so
  // that the compiler moves no memory access across it; copies become
  // visible through the explicit vmcnt waits of the waves that issued them,
  // each followed by one of these barriers.
  auto barrier = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(kWaitLgkmcnt0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  // Prologue: P of stage 0 (group 0), Q of stages 0 and 1 (group 1), all
  // landed before the first barrier; group 1 then runs one barrier behind.
  // Every wave passes 2 nst + 2 barriers in all.
  if (nst > 0) copies(0, slot_of(0));
  if (grp == 1 && nst > 1) copies(1, slot_of(1));
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
  if constexpr (TRIM) {
    if (nst == 1 || nst == 2) trim(nst - 1);
  }
  trim_last(0, slot_of(0));
  if (grp == 1) trim_last(1, slot_of(1));
  barrier();
  if (grp == 1) barrier();
  const int ahead = grp == 0 ? 1 : 2;   // stages ahead this group copies
  for (int t = 0; t < nst; ++t) {
    factors(t);
    const int slot = Op::BLK != 0 ? slot_of(t + ahead) : 0;   // (here, not where trim_last would branch for it)
    if constexpr (PKM) {
      // (The compiler has all copies land before a transposing read: they go out
      // behind the reads.)
      read_frags(t);
      copies(t + ahead, slot);
    } else {
      if (Op::BLK != 0 || t + ahead < nst) copies(t + ahead, slot);
      read_frags(t);
    }
    barrier();
    compute(t);
    // This wave's copies have landed before the next barrier publishes
    // them.  (Fenced off from the MFMAs, so that the compiler cannot move
    // the wait ahead of them.)
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    if constexpr (TRIM) {
      if (t + 3 == nst) trim(t + 2);
    }
    trim_last(t + ahead, slot);
    barrier();
  }
  if (grp == 0) barrier();

  if constexpr (GA && Op::BLK != 0) {
    uint32_t none = 0u;   // rows with no source
#pragma unroll
    for (int j = 0; j < TQ; ++j) none |= fqo[j] == kOobOffset ? 1u << j : 0u;
    clear_rows(acc, none);
  }

  // Epilogue: every wave is past its last LDS read; each stages its own
  // 64 rows of C (64 x 256 bytes) through LDS.
  staged_epilogue<Op, Cfg::WTP, Cfg::WTQ, TP, TQ, MT, typename Op::Acc16, GA>(
      a, smem + wave * (Cfg::WTQ * 256), acc, Op::BLK != 0 ? lane_id() : lane, p0 + wp * Cfg::WTP,
      q0 + wq * (Cfg::BQ / 2) + grp * Cfg::WTQ, gt);
  stamp(2);
}

template <class Op, bool KT>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
gemm_pp_kernel(const GemmArgs a) {
  gemm_pp_body<Op, KT>(a, GridTile{});
}

}  // namespace dg
