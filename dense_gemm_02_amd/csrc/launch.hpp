// Launch descriptors shared by the host dispatch (dgemm.hip) and the
// translation units that instantiate the four-wave kernels
// (four_wave.hip, compiled once per format and layout).
#pragma once

#include "common.hpp"

namespace dg {

// A launchable configuration: a kernel symbol plus its tile geometry.  Every
// kernel runs one workgroup per tile.
struct Launch {
  const void* fn;
  const char* name;
  int bp, bq, threads, lds;
  bool p_trans;
};

// Entries of the block-tile table of the four-wave kernel (dgemm.hip,
// kTiles): 0 256x256, 1 256x128, 2 128x128 (two workgroups per CU),
// 3 128x128 with four LDS stages, 4 192x256, 5 256x192, and for int8 TN
// 6 64x128 (two workgroups per CU), 7 64x128 with four LDS stages.
constexpr int kNumTiles = 8;

// The four-wave launch of table entry `idx` for one input format and layout
// (`kt`: K ends inside a stage, so the copies need tail masks).  Entries a
// variant does not build fall back to 256 x 256 (the table masks them out).
Launch four_wave_f16_tn(int idx, bool kt);
Launch four_wave_f16_nn(int idx, bool kt);
Launch four_wave_bf16_tn(int idx, bool kt);
Launch four_wave_bf16_nn(int idx, bool kt);
Launch four_wave_fp8_tn(int idx, bool kt);
Launch four_wave_fp8_nn(int idx, bool kt);
Launch four_wave_fp8s_tn(int idx, bool kt);
Launch four_wave_fp8s_nn(int idx, bool kt);
Launch four_wave_mx8_tn(int idx, bool kt);
Launch four_wave_mx8_nn(int idx, bool kt);

// The eight-wave ping-pong kernel (gemm_pp.hpp), TN, 256 x 256: op 0 FP16,
// 1 BF16, 2 FP8, 3 FP8 with scale factors.
Launch ping_pong_tn(int op, bool kt);

// Int8 with FP32, FP16 and BF16 results (any K).
Launch four_wave_i8f_tn(int idx, bool kt);
Launch four_wave_i8f_nn(int idx, bool kt);
Launch four_wave_i8h_tn(int idx, bool kt);
Launch four_wave_i8h_nn(int idx, bool kt);
Launch four_wave_i8b_tn(int idx, bool kt);
Launch four_wave_i8b_nn(int idx, bool kt);
Launch ping_pong_i8_tn(int out, bool kt);   // out: dgemm_type
// Int8 with few rows on a side, or so few tiles that a long K leaves the CUs
// idle: the skinny kernel's launch for Pn x Qn x K, or false.
bool skinny_i8_tn(int out, int64_t Pn, int64_t Qn, int64_t K, Launch* L);
bool skinny_i8_nn(int out, int64_t Pn, int64_t Qn, Launch* L);

// Keeps a HIP failure for dgemm_last_hip_error and returns DGEMM_ERR_HIP.
int hip_failed(hipError_t e);

// A buffer descriptor covers less than 2^31 bytes.
constexpr int64_t kMaxDescBytes = (int64_t(1) << 31) - 64;

// The sum of K products of two int8 values fits 32 bits up to this K.
constexpr int64_t kMaxI8K = 131071;

// Rows, tokens, pairs and groups are counted in 32 bits on the device.
constexpr int64_t kMaxCount = 0x7fffffff;

inline bool aligned_to(const void* p, int64_t n) { return ((uintptr_t)p) % (uintptr_t)n == 0; }

// HIP takes fewer than 2^32 work-items a launch.
inline bool launchable(int64_t grid, int threads) { return grid <= 0xffffffffll / threads; }

// The row operators' launches have at most this many workgroups, and more rows
// take several (1024 threads a row would not be launchable from 2^22 rows on).
constexpr int64_t kMaxRowBlocks = int64_t(1) << 21;

// One launch on the caller's stream.
inline int launch_kernel(const void* fn, int64_t grid, int threads, void* arg, void* stream) {
  void* args[] = {arg};
  const hipError_t err = hipLaunchKernel(fn, dim3((unsigned)grid), dim3((unsigned)threads), args, 0,
                                         (hipStream_t)stream);
  return err == hipSuccess ? 0 : hip_failed(err);
}

}  // namespace dg
