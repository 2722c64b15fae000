"""GPU tests of tokens sorted by expert and back, against plain
implementations: the sort on whole numbers, the rows and gradients in 64 bits
(and against differences), and runs of the operators together.

Tolerances count roundings.  Combining k rows in FP32 in a fixed order: each
step rounds by at most 2^-24 of what has been added up, k 2^-24 sum |w y| in
all (to first order; taken twice), and the output type rounds once, eps / 2 of
the value.  A dot product of H terms in any order of FP32 additions: H 2^-24
sum |d y|.  A row times a weight: one FP32 rounding and one to the type."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]
IDS = ["f32", "f16", "bf16"]
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -140, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def lib():
    import dense_gemm_02_amd as L
    return L


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ---- sort ---------------------------------------------------------------------------

def plain_sort(ids, experts):
    """Counting sort of the pairs on the host."""
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    good = (flat >= 0) & (flat < experts)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[good], minlength=experts))])
    order = np.argsort(np.where(good, flat, experts), kind="stable")[:good.sum()]
    slot = np.full(flat.size, -1)
    slot[order] = np.arange(order.size)
    pair = np.full(flat.size, -1)
    pair[:order.size] = order
    return offsets, slot.reshape(ids.shape), pair


def check_sort(ids, experts):
    T, k = ids.shape
    offsets, slot, pair, token = lib().expert_sort(ids, experts, with_token=True)
    o, s, p = plain_sort(ids, experts)
    assert offsets.dtype == slot.dtype == pair.dtype == token.dtype == torch.int32
    assert np.array_equal(offsets.cpu().numpy(), o)
    assert np.array_equal(slot.cpu().numpy(), s)
    assert np.array_equal(pair.cpu().numpy(), p)
    assert np.array_equal(token.cpu().numpy(), np.where(p >= 0, p // max(k, 1), -1))
    three = lib().expert_sort(ids, experts)
    assert len(three) == 3 and all(torch.equal(x, y) for x, y in zip(three, (offsets, slot, pair)))


SORTS = [(1, 1, 1), (1, 8, 64), (16, 8, 64), (7, 3, 5), (63, 1, 2), (64, 1, 3), (65, 2, 7), (1000, 4, 16),
         (1023, 1, 128), (1024, 1, 1), (1025, 1, 1024), (511, 2, 1000), (4099, 8, 128), (16384, 2, 8), (20001, 6, 255),
         (65536, 8, 256), (131071, 1, 64), (40000, 8, 1024), (3, 1000, 11)]


@pytest.mark.parametrize("dtype", [torch.int64, torch.int32], ids=["i64", "i32"])
@pytest.mark.parametrize("T,k,E", SORTS)
def test_sort(T, k, E, dtype):
    print(f"sort {T}x{k} into {E}", flush=True)
    g = gen(T + k + E)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=dtype)
    check_sort(ids, E)
    ids[torch.rand((T, k), generator=g, device="cuda") < 0.1] = -1        # dropped pairs
    ids[torch.rand((T, k), generator=g, device="cuda") < 0.05] = E
    check_sort(ids, E)


@pytest.mark.parametrize("T,k,E", [(300, 2, 9), (5000, 8, 64), (70000, 3, 33)])
def test_sort_extremes(T, k, E):
    far = {torch.int64: 2 ** 40 + 1, torch.int32: 2 ** 31 - 1}
    for dtype in (torch.int64, torch.int32):
        for fill in (0, E - 1, -1, E, far[dtype], -far[dtype]):
            check_sort(torch.full((T, k), fill, dtype=dtype, device="cuda"), E)
        ids = (torch.arange(T * k, device="cuda", dtype=dtype) % E).reshape(T, k)
        check_sort(ids, E)
        check_sort((ids * 0 + E - 1 - ids), E)
        check_sort(torch.sort(ids.reshape(-1))[0].reshape(T, k), E)
    wide = torch.full((T, k), 2 ** 32, dtype=torch.int64, device="cuda")   # expert 0 in the low half
    check_sort(wide, E)


def test_sort_empty():
    L = lib()
    for T, k in ((0, 4), (5, 0)):
        offsets, slot, pair = L.expert_sort(torch.empty((T, k), dtype=torch.int64, device="cuda"), 3)
        assert offsets.tolist() == [0, 0, 0, 0] and slot.shape == (T, k) and pair.numel() == 0
    offsets, slot, pair = L.expert_sort(torch.zeros((5, 2), dtype=torch.int64, device="cuda"), 0)
    assert offsets.tolist() == [0] and (slot == -1).all() and (pair == -1).all()


# ---- rows ---------------------------------------------------------------------------

def routing(T, k, E, seed, drop=0.1):
    g = gen(seed)
    ids = torch.argsort(torch.rand((T, E), generator=g, device="cuda"), 1)[:, :k].contiguous()
    ids[torch.rand((T, k), generator=g, device="cuda") < drop] = -1
    w = torch.rand((T, k), generator=g, device="cuda")
    offsets, slot, pair = lib().expert_sort(ids, E)
    return ids, w, offsets, slot, pair


def rows(g, n, H, dtype, pad=0, off=0):
    base = torch.randn((n, H + pad + off), generator=g, device="cuda").to(dtype)
    return base[:, off:off + H]


def picked(y, slot):
    ok = (slot >= 0) & (slot < y.shape[0])
    return torch.where(ok[:, :, None], y.double()[slot.long().clamp(0, y.shape[0] - 1)], 0.0)


def near(got, want, bound):
    """|got - want| <= bound + half a step of the type."""
    bad = (got.double() - want).abs() > bound * (1 + 2.0 ** -10) + HALF[got.dtype] * (want.abs() + bound) + TINY[got.dtype]
    assert not bad.any(), (int(bad.sum()), float((got.double() - want).abs().max()))


def check_combine(y, slot, w, out=None):
    got = lib().expert_combine(y, slot, w, out=out)
    terms = picked(y, slot) * (1.0 if w is None else w.double()[:, :, None])
    near(got, terms.sum(1), 2 * slot.shape[1] * 2.0 ** -24 * terms.abs().sum(1))
    return got


def check_grad(dout, y, slot, w, dy=None):
    L = lib()
    T, k = slot.shape
    before = None if dy is None else dy.clone()
    got, dw = L.expert_combine_grad(dout, y, slot, w, dy=dy)
    ok = (slot >= 0) & (slot < y.shape[0])
    back = dout.double()[:, None, :] * (torch.ones_like(slot).double() if w is None else w.double())[:, :, None]
    n = slot[ok].long()
    near(got[n], back[ok], 2.0 ** -24 * back[ok].abs())
    if before is not None:
        rest = torch.ones(y.shape[0], dtype=torch.bool, device="cuda")
        rest[n] = False
        assert torch.equal(got[rest], before[rest])
    terms = picked(y, slot) * dout.double()[:, None, :]
    near(dw, terms.sum(2), y.shape[1] * 2.0 ** -24 * terms.abs().sum(2))
    assert (dw[~ok] == 0).all()
    return got, dw


ROWS = [(1, 1, 1, 1), (1, 8, 64, 4096), (16, 8, 64, 512), (5, 2, 3, 7), (33, 3, 9, 100), (7, 1, 4, 2048),
        (130, 4, 16, 1000), (257, 8, 32, 264), (65, 6, 8, 4104), (9, 2, 8, 8192), (3, 2, 4, 20000), (1000, 2, 8, 129),
        (20, 16, 40, 640)]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,k,E,H", ROWS)
def test_rows(T, k, E, H, dtype):
    print(f"rows {T}x{k} of {E}, H={H} {dtype}", flush=True)
    g = gen(T * 7 + H)
    _, w, offsets, slot, pair = routing(T, k, E, T + H)
    kept = int(offsets[-1])
    L = lib()
    x = rows(g, T, H, dtype)
    out = torch.full((T * k, H), 7.0, device="cuda").to(dtype)
    y = L.expert_dispatch(x, slot, out=out)
    assert torch.equal(y[:kept], x[pair[:kept].long() // k]) and (y[kept:] == 7).all()
    assert torch.equal(L.expert_dispatch(x, slot)[:kept], y[:kept])
    y = rows(g, T * k, H, dtype)
    check_combine(y, slot, w)
    check_combine(y, slot, None)
    assert torch.equal(L.expert_dispatch_grad(y, slot), L.expert_combine(y, slot))
    dout = rows(g, T, H, dtype)
    check_grad(dout, y, slot, w, dy=torch.full((T * k, H), 7.0, device="cuda").to(dtype))
    check_grad(dout, y, slot, None)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_rows_strides_and_offsets(dtype):
    """Rows off every alignment and of any pitch; what lies between stays."""
    L = lib()
    for H in (64, 100, 1000, 4096):
        for off in (0, 1, 2, 3, 4, 8):
            for pad in (0, 1, 8):
                g = gen(H + off + pad)
                T, k = 21, 3
                _, w, offsets, slot, pair = routing(T, k, 5, H)
                kept = int(offsets[-1])
                x, dout = rows(g, T, H, dtype, pad, off), rows(g, T, H, dtype, pad + 1, off)
                y = rows(g, T * k, H, dtype, pad, off)
                wide = torch.full((T * k, H + off + pad + 3), 7.0, device="cuda").to(dtype)
                L.expert_dispatch(x, slot, out=wide[:, off:off + H])
                assert torch.equal(wide[:kept, off:off + H], x[pair[:kept].long() // k])
                assert (wide[kept:] == 7).all() and (wide[:, :off] == 7).all() and (wide[:, off + H:] == 7).all()
                back = torch.full((T, H + off + pad + 3), 7.0, device="cuda").to(dtype)
                check_combine(y, slot, w, out=back[:, off:off + H])
                assert (back[:, :off] == 7).all() and (back[:, off + H:] == 7).all()
                dy = torch.full((T * k, H + off + pad + 3), 7.0, device="cuda").to(dtype)
                check_grad(dout, y, slot, w, dy=dy[:, off:off + H])
                assert (dy[:, :off] == 7).all() and (dy[:, off + H:] == 7).all()


def test_dropped_pairs_touch_nothing():
    """Slots outside the rows, tokens with no pair left, and rows of NaN and
    infinities that no slot names."""
    L = lib()
    T, k, H, n = 50, 4, 300, 60
    g = gen(2)
    slot = torch.randperm(n, generator=g, device="cuda")[:T].int().reshape(T, 1).repeat(1, k).contiguous()
    slot[:, 1], slot[:, 2], slot[:, 3] = -1, n, 2 ** 31 - 1
    slot[::5, 0] = -2 ** 31
    y = rows(g, n, H, torch.float32)
    named = torch.zeros(n, dtype=torch.bool, device="cuda")
    ok = (slot >= 0) & (slot < n)
    named[slot[ok].long()] = True
    y[~named] = float("nan")
    w = torch.rand((T, k), generator=g, device="cuda")
    w[~ok] = float("inf")
    out = check_combine(y, slot, torch.where(ok, w, 0.0))
    assert torch.equal(L.expert_combine(y, slot, w), out) and (out[::5] == 0).all()
    check_grad(rows(g, T, H, torch.float32), y, slot, torch.where(ok, w, 0.0), dy=torch.full((n, H), 7.0, device="cuda"))
    big = torch.full((n, H), 7.0, device="cuda")
    x = rows(g, T, H, torch.float32)
    L.expert_dispatch(x, slot, out=big)
    assert (big[~named] == 7).all()
    t_of = torch.arange(T, device="cuda")[:, None].expand(T, k)[ok]
    assert torch.equal(big[slot[ok].long()], x[t_of])


def test_special_values_pass():
    """Infinities and NaN of named rows reach their token and no other."""
    L = lib()
    slot = torch.arange(12, dtype=torch.int32, device="cuda").reshape(6, 2)
    for H in (40, 1024):
        y = torch.ones((12, H), device="cuda", dtype=torch.bfloat16)
        y[2, 3], y[5, 0], y[7, H - 1] = float("inf"), float("nan"), -float("inf")
        w = torch.full((6, 2), 0.5, device="cuda")
        out = L.expert_combine(y, slot, w)
        want = torch.ones((6, H), device="cuda", dtype=torch.bfloat16)
        want[1, 3], want[2, 0], want[3, H - 1] = float("inf"), float("nan"), -float("inf")
        assert torch.equal(torch.nan_to_num(out, 5.0), torch.nan_to_num(want, 5.0))
        _, dw = L.expert_combine_grad(torch.ones((6, H), device="cuda", dtype=torch.bfloat16), y, slot, w)
        assert dw[1, 0] == float("inf") and torch.isnan(dw[2, 1]) and dw[3, 1] == -float("inf")
        assert torch.isfinite(dw).sum() == 9


def test_empty():
    L = lib()
    e = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    x = torch.empty((0, 16), device="cuda")
    assert L.expert_dispatch(x, e).shape == (0, 16) and L.expert_combine(x, e).shape == (0, 16)
    none = torch.empty((4, 0), dtype=torch.int32, device="cuda")
    assert (L.expert_combine(torch.ones((5, 16), device="cuda"), none) == 0).all()
    gone = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    assert (L.expert_combine(torch.ones((0, 16), device="cuda"), gone) == 0).all()
    dy, dw = L.expert_combine_grad(torch.ones((4, 16), device="cuda"), torch.ones((0, 16), device="cuda"), gone)
    assert dy.shape == (0, 16) and (dw == 0).all()
    thin = torch.empty((4, 0), device="cuda")
    _, dw = L.expert_combine_grad(thin, torch.empty((8, 0), device="cuda"),
                                  torch.arange(8, dtype=torch.int32, device="cuda").reshape(4, 2))
    assert (dw == 0).all()


def test_rows_past_2_31_bytes():
    """Sorted rows whose byte offsets pass 32 bits."""
    L = lib()
    H, n = 8192, 140000                       # 2.3 GB of bf16
    y = torch.zeros((n, H), dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([[n - 1, 3], [0, n - 2]], dtype=torch.int32, device="cuda")
    x = torch.randn((2, H), generator=gen(1), device="cuda").bfloat16()
    L.expert_dispatch(x, slot, out=y)
    assert torch.equal(y[n - 1], x[0]) and torch.equal(y[3], x[0]) and torch.equal(y[n - 2], x[1])
    assert float(y.abs().sum(1).ne(0).sum()) == 4
    w = torch.tensor([[1.0, 1.0], [0.5, 0.25]], device="cuda")
    near(L.expert_combine(y, slot, w), x.double() * torch.tensor([[2.0], [0.75]], device="cuda").double(),
         4 * 2.0 ** -24 * 2 * x.double().abs())
    check = L.expert_combine_grad(x, y, slot, w, dy=y.clone())[0]
    assert torch.equal(check[n - 1], x[0])


# ---- runs of the operators together -------------------------------------------------

def test_gradients_against_differences():
    """Central differences of the whole way (dispatch, a product per expert,
    combine) along random directions, all in FP32: the function is bilinear in
    (x, weights), so a central difference is exact up to rounding."""
    L = lib()
    T, k, E, H, N = 23, 2, 5, 48, 32
    g = gen(7)
    _, w, offsets, slot, pair = routing(T, k, E, 4)
    off = offsets.tolist()
    W = torch.randn((E, N, H), generator=g, device="cuda")
    x, dout = torch.randn((T, H), generator=g, device="cuda"), torch.randn((T, N), generator=g, device="cuda")

    def products(rows_in, mats):
        out = torch.zeros((T * k, mats.shape[1]), device="cuda")
        for e in range(E):
            if off[e + 1] > off[e]:
                out[off[e]:off[e + 1]] = L.matmul(rows_in[off[e]:off[e + 1]], mats[e].t())
        return out

    def forward(x, w):
        rows_in = L.expert_dispatch(x, slot, out=torch.zeros((T * k, H), device="cuda"))
        y = products(rows_in, W)
        return L.expert_combine(y, slot, w), y

    out, y = forward(x, w)
    dy, dw = L.expert_combine_grad(dout, y, slot, w, dy=torch.zeros_like(y))
    dx = L.expert_dispatch_grad(products(dy, W.transpose(1, 2).contiguous()), slot)
    for seed in range(4):
        gx = torch.randn((T, H), generator=gen(100 + seed), device="cuda")
        gw = torch.randn((T, k), generator=gen(200 + seed), device="cuda")
        for vx, vw, got in ((gx, 0 * gw, (dx.double() * gx.double()).sum()),
                            (0 * gx, gw, (dw.double() * gw.double()).sum())):
            up, down = forward(x + vx, w + vw)[0], forward(x - vx, w - vw)[0]
            diff = ((up.double() - down.double()) / 2 * dout.double()).sum()
            # FP32 sums of 48 + 2 products, and the steps x + v, each off by
            # 2^-24 of at most the terms' magnitudes.
            size = sum((forward_abs(W, off, slot, E, a.abs() + b.abs(), (c.abs() + d.abs())) * dout.abs().double()).sum()
                       for a, b, c, d in ((x, vx, w, vw),))
            assert abs(float(got - diff)) <= 2 * 60 * 2.0 ** -24 * float(size)


def forward_abs(W, off, slot, E, x, w):
    y = torch.zeros((slot.numel(), W.shape[1]), dtype=torch.float64, device="cuda")
    ok = slot >= 0
    e_of = torch.bucketize(torch.arange(slot.numel(), device="cuda"), torch.tensor(off[1:], device="cuda"), right=True)
    t_of = torch.arange(slot.shape[0], device="cuda")[:, None].expand_as(slot)[ok]
    n = slot[ok].long()
    for i, t in zip(n.tolist(), t_of.tolist()):
        y[i] = W[int(e_of[i])].abs().double() @ x[t].double()
    return (picked(y, slot) * w.double()[:, :, None]).sum(1)


def test_training_step_in_bf16_with_the_dense_products():
    """Dispatch, gemm_bf16 per expert, combine, and back, against 64 bits: the
    forward and the gradients of x and of the router's weights."""
    L = lib()
    T, k, E, H, N = 64, 2, 4, 128, 96
    g = gen(17)
    _, w, offsets, slot, pair = routing(T, k, E, 6)
    off = offsets.tolist()
    bf = torch.bfloat16
    W = torch.randn((E, N, H), generator=g, device="cuda").to(bf)
    x = torch.randn((T, H), generator=g, device="cuda").to(bf)
    dout = torch.randn((T, N), generator=g, device="cuda").to(bf)

    def products(a, mats):
        out = torch.zeros((T * k, mats.shape[1]), device="cuda", dtype=bf)
        for e in range(E):
            if off[e + 1] > off[e]:      # C^T = W A^T: column-major of W x A^T is row-major A W^T
                L.matmul(mats[e], a[off[e]:off[e + 1]].t(), out=out[off[e]:off[e + 1]].t())
        return out

    a = L.expert_dispatch(x, slot, out=torch.zeros((T * k, H), device="cuda", dtype=bf))
    y = products(a, W)
    out = L.expert_combine(y, slot, w)
    dy, dw = L.expert_combine_grad(dout, y, slot, w, dy=torch.zeros_like(y))
    dx = L.expert_dispatch_grad(products(dy, W.transpose(1, 2).contiguous()), slot)

    e_of = torch.bucketize(torch.arange(T * k, device="cuda"), offsets[1:], right=True).clamp(max=E - 1)
    ok = (slot >= 0)
    s = slot.long().clamp(min=0)
    Wp = W.double()[e_of[s]]                                                    # [T, k, N, H]
    yp = (Wp * x.double()[:, None, None, :]).sum(3)
    ya = (Wp.abs() * x.double().abs()[:, None, None, :]).sum(3)
    m = (w.double() * ok)[:, :, None]
    # y rounds to bf16 (after an FP32 sum of H terms), out sums k of them
    near(out, (m * yp).sum(1), (m * (yp.abs() * 2.0 ** -8 + ya * (H + 8) * 2.0 ** -24)).sum(1))
    dwp = (yp * dout.double()[:, None, :]).sum(2) * ok
    near(dw, dwp, ((yp.abs() * 2.0 ** -8 + ya * (H + 8) * 2.0 ** -24) * dout.double().abs()[:, None, :]).sum(2)
         + N * 2.0 ** -24 * (yp.abs() * dout.double().abs()[:, None, :]).sum(2))
    back = m * dout.double()[:, None, :]                                        # dy, rounds to bf16
    dap = (Wp * back[..., None]).sum(2)
    daa = (Wp.abs() * back.abs()[..., None]).sum(2)
    near(dx, dap.sum(1), (dap.abs() * 2.0 ** -8 + daa * (2.0 ** -8 + (N + 8) * 2.0 ** -24) * (1 + 2.0 ** -8)).sum(1))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,k,E,N,K", [(1, 2, 4, 64, 96), (16, 8, 64, 300, 512), (200, 2, 8, 384, 1000),
                                       (700, 4, 16, 520, 256)])
def test_int8_experts_layer(T, k, E, N, K, dtype):
    """matmul_experts against its definition in 64 bits on the quantised values."""
    L = lib()
    g = gen(T + N)
    ids, w, offsets, slot, pair = routing(T, k, E, T + K)
    x = torch.randn((T, K), generator=g, device="cuda").to(dtype)
    b, sb = L.quantize_i8(torch.randn((E * N, K), generator=g, device="cuda"))
    b, sb = b.as_strided((E, N, K), (N * b.stride(0), b.stride(0), 1)), sb.reshape(E, N)
    got = L.matmul_experts(x, ids, w, b, sb)
    assert got.dtype == dtype
    q, sx = L.quantize_i8(x)
    want = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for j in range(k):
        e = ids[:, j].clamp(min=0)
        for t in range(T) if T <= 16 else range(0, T, 7):
            if ids[t, j] < 0:
                continue
            y = (b[int(e[t])].double() @ q[t].double()) * sx[t].double() * sb[int(e[t])].double()
            want[t] += w[t, j].double() * y
            size[t] += w[t, j].double() * y.abs()
    seen = torch.arange(T, device="cuda") % (1 if T <= 16 else 7) == 0
    # each y: three FP32 roundings and one to the type; then k steps in FP32
    y_step = 3 * 2.0 ** -24 + (0.0 if dtype == torch.float32 else HALF[dtype])
    near(got[seen], want[seen], (size * (y_step + 2 * k * 2.0 ** -24))[seen])


def test_layer_captured_into_a_graph_with_eager_work_between():
    L = lib()
    T, k, E, N, K = 48, 4, 16, 256, 512
    g = gen(3)
    b = torch.randint(-127, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    sb = torch.rand((E, N), generator=g, device="cuda") * 0.01
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    ids, w, _, _, _ = routing(T, k, E, 1)

    def step():
        out = L.matmul_experts(x, ids, w, b, sb)
        offsets, slot, pair = L.expert_sort(ids, E)
        y = L.expert_dispatch(x, slot, out=torch.zeros((T * k, K), dtype=x.dtype, device="cuda"))
        dy, dw = L.expert_combine_grad(x, y, slot, w, dy=torch.zeros_like(y))
        return out, slot, y, dy, dw, L.expert_dispatch_grad(dy, slot)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in range(4):
        x.copy_(torch.randn((T, K), generator=g, device="cuda"))
        ids.copy_(routing(T, k, E, 30 + seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, step()):
            assert torch.equal(got, want)


def test_two_graphs_in_turn():
    """Two captured graphs with a sort that needs its workspace, replayed in
    turn with eager calls between."""
    L = lib()
    state, graphs = [], []
    for seed, (T, k, E) in ((1, (3000, 4, 40)), (2, (5000, 2, 700))):
        ids = routing(T, k, E, seed)[0]
        x = rows(gen(seed), T, 200, torch.bfloat16)
        w = torch.rand((T, k), generator=gen(seed), device="cuda")

        def step(ids=ids, x=x, w=w, E=E):
            offsets, slot, pair = L.expert_sort(ids, E)
            return offsets, slot, pair, L.expert_combine(L.expert_dispatch(x, slot), slot, w)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        state.append((ids, step, out, (T, k, E)))
        graphs.append(graph)
    for turn in range(3):
        for (ids, _, _, shape), graph in zip(state, graphs):
            ids.copy_(routing(*shape, 50 + turn)[0])
        for graph in graphs:
            graph.replay()
        for _, step, out, _ in state:
            for got, want in zip(out, step()):
                assert torch.equal(got, want)


def test_layer_without_pairs():
    """No token, and tokens that no expert takes."""
    L = lib()
    b = torch.ones((3, 32, 64), dtype=torch.int8, device="cuda")
    sb = torch.ones((3, 32), device="cuda")
    none = L.matmul_experts(torch.ones((0, 64), device="cuda"), torch.zeros((0, 2), dtype=torch.int64, device="cuda"),
                            torch.ones((0, 2), device="cuda"), b, sb)
    assert none.shape == (0, 32)
    x = torch.randn((5, 64), generator=gen(1), device="cuda").half()
    out = L.matmul_experts(x, torch.full((5, 2), -1, device="cuda"), torch.ones((5, 2), device="cuda"), b, sb)
    assert out.shape == (5, 32) and out.dtype == torch.float16 and (out == 0).all()
    one = L.matmul_experts(x[:1], torch.full((1, 1), 2, device="cuda"), None, b, sb)
    q, s = L.quantize_i8(x[:1])
    near(one, q.double().sum(1, keepdim=True).expand(1, 32) * s.double()[:, None], 6 * 2.0 ** -24 * 64 * 127 * s.double()[:, None])


def test_two_streams_at_once():
    L = lib()
    cases = []
    for seed in (1, 2):
        ids, w, _, slot, _ = routing(9000, 4, 64, seed)
        cases.append((ids, w, rows(gen(seed), 9000, 512, torch.bfloat16)))

    def run(c, stream=None):
        ids, w, x = c
        offsets, slot, pair = L.expert_sort(ids, 64, stream=stream)
        return offsets, slot, pair, L.expert_combine(L.expert_dispatch(x, slot, stream=stream), slot, w, stream=stream)

    want = [run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(run(c, stream=s))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        for a, b in zip(r, want[i % 2]):
            assert torch.equal(a, b)


def test_results_repeat():
    L = lib()
    ids, w, _, slot, _ = routing(3000, 8, 32, 5)
    y, d = rows(gen(1), 24000, 1032, torch.bfloat16), rows(gen(2), 3000, 1032, torch.bfloat16)
    dy = torch.zeros_like(y)
    first = [t.clone() for t in (L.expert_combine(y, slot, w), *L.expert_combine_grad(d, y, slot, w, dy=dy))]
    for _ in range(3):
        for a, b in zip(first, (L.expert_combine(y, slot, w), *L.expert_combine_grad(d, y, slot, w, dy=dy))):
            assert torch.equal(a, b)


def test_python_refusals():
    L = lib()
    ids = torch.zeros((6, 2), dtype=torch.int64, device="cuda")
    slot = torch.arange(12, dtype=torch.int32, device="cuda").reshape(6, 2)
    x, y = torch.randn((6, 8), device="cuda"), torch.randn((12, 8), device="cuda")
    w = torch.rand((6, 2), device="cuda")
    value = [
        lambda: L.expert_sort(ids.reshape(-1), 3), lambda: L.expert_sort(ids[:, :1], 3), lambda: L.expert_sort(ids, -1),
        lambda: L.expert_dispatch(y, slot), lambda: L.expert_dispatch(x, slot, out=y.half()),
        lambda: L.expert_dispatch(x, slot, out=y[:, :7]), lambda: L.expert_dispatch(x, slot, rows=11, out=y),
        lambda: L.expert_dispatch(x.t().contiguous().t(), slot), lambda: L.expert_combine(y, slot, w, out=y),
        lambda: L.expert_combine_grad(y, y, slot, w), lambda: L.expert_combine_grad(x, y, slot, w, dy=x),
        lambda: L.expert_combine_grad(x.half(), y, slot, w),
    ]
    kind = [
        lambda: L.expert_sort(ids.float(), 3), lambda: L.expert_dispatch(x, slot.long()),
        lambda: L.expert_combine(y.double(), slot), lambda: L.expert_combine(y, slot, w.half()),
        lambda: L.expert_combine(y, slot, w[:5]), lambda: L.expert_combine(y, slot[:, :1]),
        lambda: L.expert_combine_grad(x, y, slot, w, dweights=w.half()),
    ]
    for calls, error in ((value, ValueError), (kind, TypeError)):
        for i, c in enumerate(calls):
            with pytest.raises(error):
                c()
                print("not refused:", error, i)
    with pytest.raises(L.DgemmError) as e:
        L.expert_sort(ids, 1025)
    assert e.value.status == 6
    with pytest.raises(L.DgemmError) as e:        # rows of pitch 0
        L.expert_dispatch(x[:1].expand(6, 8), slot)
    assert e.value.status == 3


def test_streams_by_argument():
    """Work given a stream is that stream's, its results and workspace too."""
    L = lib()
    ids, w, _, slot, pair = routing(5000, 4, 40, 9)
    x = rows(gen(2), 5000, 256, torch.bfloat16)
    b = torch.randint(-127, 128, (40, 64, 256), generator=gen(3), device="cuda", dtype=torch.int8)
    sb = torch.rand((40, 64), generator=gen(4), device="cuda")
    want = L.matmul_experts(x, ids, w, b, sb)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        _, slot2, pair2 = L.expert_sort(ids, 40, stream=stream)
        got = L.matmul_experts(x, ids, w, b, sb, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(slot2, slot) and torch.equal(pair2, pair) and torch.equal(got, want)
