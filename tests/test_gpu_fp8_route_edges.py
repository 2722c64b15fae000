"""GPU tests of what the documentation of the block-scaled FP8 and router
functions allows at its ends: saturated and tiny scores, NaN in the padding of
narrow operands, the smallest and the largest operands (places past 2^32),
indices that occur twice, several threads and captured graphs at once.
Tolerances are those of test_gpu_fp8.py and test_gpu_route.py."""

import threading

import numpy as np
import pytest
import torch

from test_gpu_fp8 import FP8, GROUPED, IDS, TYPES, check_quantised, exact, factors, fp8s, gen, kernels, lib, near, \
    product
from test_gpu_route import check

pytestmark = pytest.mark.gpu


# ---- the router ---------------------------------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("k", [2, 12, 13])
def test_scores_that_are_equal_in_64_bits_stand_by_their_logits(score, groups, k):
    """Sigmoids of 40 and more are 1 in 64 bits, softmax shares 800 below the largest 0: without a bias the logits say
    which is larger, however many choices there are."""
    L = lib()
    T, E = 9, 32
    base = torch.arange(E, device="cuda", dtype=torch.float32)
    rows = [(base * 7 + 5 * t) % E for t in range(T)]
    logits = torch.stack(rows) + 40.0
    if score == "softmax":
        logits = torch.where(logits == logits.amax(1, keepdim=True), 0.0, logits - 900.0)
    ids, w = L.expert_route(logits, k, score=score, groups=groups)
    assert torch.equal(ids.long(), logits.argsort(dim=1, descending=True, stable=True)[:, :k])
    assert bool(torch.isfinite(w).all())
    if groups == 4:
        ids, _ = L.expert_route(logits, k, score=score, groups=groups, top_groups=2)
        stay = logits.reshape(T, 4, 8).amax(2).argsort(dim=1, descending=True, stable=True)[:, :2]
        mask = torch.zeros((T, 4), dtype=torch.bool, device="cuda").scatter_(1, stay, True).repeat_interleave(8, 1)
        assert torch.equal(ids.long(), torch.where(mask, logits, -3e38).argsort(dim=1, descending=True, stable=True)[:, :k])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("sign", [-1.0, 1.0], ids=["lowest", "highest"])
def test_biases_at_the_ends_of_float32(score, sign):
    """Experts masked by the lowest value of float32 (or lifted by the highest): the sum of a group's two best is past
    float32's range, and the group still counts."""
    end = sign * float(torch.finfo(torch.float32).max)
    for E, G, tg, k in ((32, 8, 4, 12), (6, 2, 1, 3), (21, 7, 6, 11), (256, 8, 4, 8), (96, 32, 9, 7)):
        g = gen(E)
        logits = torch.randn((40, E), generator=g, device="cuda")
        size = E // G
        bias = torch.linspace(-0.1, 0.1, E, device="cuda")
        bias[size:] = end                                   # one group as it is
        check(logits, k, bias=bias, score=score, groups=G, top_groups=tg, group_best=2)
        bias = torch.where(torch.rand((E,), generator=g, device="cuda") < 0.6, end, 0.0)
        check(logits, k, bias=bias, score=score, groups=G, top_groups=tg, group_best=2)
        for _ in range(20):
            bias = sign * torch.rand((E,), generator=g, device="cuda") * 3.4e38
            check(logits, k, bias=bias, score=score, groups=G, top_groups=tg, group_best=2)


def by_logits(logits, k, groups=1, top_groups=1):
    """The k largest logits, of equal ones the lower index first, of the groups that hold the largest."""
    l = logits.double() + 0.0
    if top_groups < groups:
        T, E = l.shape
        stay = l.reshape(T, groups, E // groups).amax(2).argsort(dim=1, descending=True, stable=True)[:, :top_groups]
        mask = torch.zeros((T, groups), dtype=torch.bool, device="cuda").scatter_(1, stay, True)
        l = torch.where(mask.repeat_interleave(E // groups, 1), l, -3e38)
    return l.argsort(dim=1, descending=True, stable=True)[:, :k]


# (experts, groups, top_groups, k) of routers that take a whole wave a token: sixteen choices and more, more than 256
# experts, more than sixteen groups, more than sixteen experts for each lane of a group.
WAVES = [(32, 1, 1, 16), (32, 1, 1, 17), (32, 4, 2, 16), (64, 4, 2, 20), (320, 1, 1, 4), (320, 4, 2, 13), (1024, 1, 1, 64),
         (96, 32, 9, 7), (252, 12, 5, 8)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("router", WAVES, ids=lambda r: "{}-{}-{}-{}".format(*r))
def test_a_wave_a_token_chooses_by_the_logits(router, score):
    """Sigmoids of 40 and more, softmax shares 800 below the largest, equal in 64 bits; zeros of either sign."""
    L = lib()
    E, groups, top_groups, k = router
    T = 9
    base = torch.arange(E, device="cuda", dtype=torch.float32)
    logits = torch.stack([(base * 7 + 5 * t) % E for t in range(T)]) + 40.0          # (7 and E: no common divisor, or 252)
    if score == "softmax":
        logits = torch.where(logits == logits.amax(1, keepdim=True), 0.0, logits - 1900.0)
    kw = dict(score=score, groups=groups, top_groups=top_groups)
    for renormalize in (True, False):
        ids, w = L.expert_route(logits, k, renormalize=renormalize, **kw)
        assert torch.equal(ids.long(), by_logits(logits, k, groups, top_groups))
        assert bool(torch.isfinite(w).all())
    zeros = torch.zeros((T, E), device="cuda")
    zeros[:, ::2] = -0.0
    zeros[3:6, 1::3] = 1.0
    zeros[6:, 2::5] = -1.0
    ids, _ = check(zeros, k, dweights=torch.randn((T, k), generator=gen(E), device="cuda"), **kw)
    assert torch.equal(ids.long(), by_logits(zeros, k, groups, top_groups))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("depth", [20.0, 60.0, 84.0, 92.0, 100.0, 110.0])
def test_groups_of_tiny_scores(score, depth):
    """Sums of a group's two best scores far below 1, where FP32 exponentials lose places and then all of them: which
    groups stay is still that of 64 bits."""
    g = gen(int(depth))
    T, E, G = 64, 64, 8
    logits = torch.rand((T, E), generator=g, device="cuda") * 2.0 ** -8 - depth
    logits[:, 3] = -depth + 5.0
    logits[: T // 2, 8:] -= 30.0 * (torch.rand((T // 2, E - 8), generator=g, device="cuda") < 0.7)
    if score == "softmax":
        logits[:, 3] = 0.0
    check(logits, 8, score=score, groups=G, top_groups=3, group_best=2)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("k", [12, 13, 14, 15, 16, 17])
def test_choices_around_sixteen(dtype, k):
    """As many choices as a token has lanes, and a few fewer or more; distinct values, many equal ones, and values a few
    last places apart."""
    g = gen(k)
    for E, G, tg in ((256, 8, 4), (64, 1, 1), (20, 1, 1)):
        for spread in (2.0, 2.0 ** -20):
            logits = (torch.randn((150, E), generator=g, device="cuda") * spread + 1.0).to(dtype)
            dw = torch.randn((150, k), generator=g, device="cuda")
            bias = torch.linspace(-1e-3, 1e-3, E, device="cuda").round(decimals=4)
            check(logits, k, dweights=dw, groups=G, top_groups=tg)
            check(logits, k, dweights=dw, bias=bias, score="sigmoid", groups=G, top_groups=tg, group_best=2)
            check(logits, k, bias=bias, groups=G, top_groups=tg)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_route_smallest_and_widest(dtype):
    for E, k, G, tg in ((1, 1, 1, 1), (2, 2, 1, 1), (2, 2, 2, 1 + 1), (1024, 64, 1, 1), (1023, 64, 33, 5), (1024, 1, 1024, 1)):
        for T in (1, 5):
            logits = torch.randn((T, E), generator=gen(E + T), device="cuda").to(dtype)
            dw = torch.randn((T, k), generator=gen(1), device="cuda")
            check(logits, k, dweights=dw, score="softmax", groups=G, top_groups=tg)
            check(logits, k, dweights=dw, score="sigmoid", groups=G, top_groups=tg, renormalize=False)


def test_gradient_of_ids_that_occur_many_times_is_the_same_every_time():
    L = lib()
    logits = torch.randn((200, 24), generator=gen(2), device="cuda")
    for k in (8, 24):
        ids = torch.randint(0, 3, (200, k), generator=gen(3), device="cuda", dtype=torch.int32)
        dw = torch.randn((200, k), generator=gen(4), device="cuda")
        first = L.expert_route_grad(dw, logits, ids)
        for _ in range(20):
            assert torch.equal(L.expert_route_grad(dw, logits, ids), first)


# ---- FP8 ---------------------------------------------------------------------------

# What the matrix unit cuts off of a sum of products of every size, of its magnitudes: seven of eight neighbours less
# than 2^(E - 13) each, E the largest sum of exponents (see below).  A product is a multiple of 2^-6 of its own 2^E, so
# one that is cut has an E below the largest by more than 7, and the largest is above -12 + 7: one of its values at most
# is subnormal, that is 2^-3 of 2^-6 or more, and the largest product 2^(E - 3) or more.
CUT = 7 * 2.0 ** -10 + 127 * 2.0 ** -23


@pytest.mark.parametrize("kernel", [("tn", "256x256_pp"), ("tn", "128x128_w4"), ("tn", "skinny_a:32x32x1"),
                                    ("tn", "skinny_b:16x16x2"), ("nn", "256x256_pp"), ("nn", "256x64_w4"),
                                    ("nn", "skinny_32x32")], ids="-".join)
@pytest.mark.parametrize("zeros", [False, True], ids=["dense", "zeros"])
def test_what_the_matrix_unit_cuts_off(monkeypatch, kernel, zeros):
    """Eight neighbours' products, bit for bit: each loses, toward zero, what lies below 2^(E - 13), E the largest sum of
    exponents of two values with a product other than zero, where subnormal values have the exponent -6.  A sum of
    eight multiples of 2^(E - 13) below 2^(E + 2) each is exact in FP32."""
    layout, name = kernel
    monkeypatch.setenv("DGEMM_CONFIG", f"b8f32_{layout}_{name}")
    L = lib()
    g = gen(5 + zeros)
    n, K = 128, 128
    for at in (0, 8, 40, 120):
        byte = torch.randint(1, 0x7f, (2, n, 8), generator=g, device="cuda", dtype=torch.uint8)
        tiny = torch.rand(byte.shape, generator=g, device="cuda") < 0.3
        byte = torch.where(tiny, 1 + byte % 15, byte)
        byte |= torch.randint(0, 2, byte.shape, generator=g, device="cuda", dtype=torch.uint8) << 7
        if zeros:
            byte *= torch.rand(byte.shape, generator=g, device="cuda") >= 0.4
        full = torch.zeros((2, n, K), dtype=torch.uint8, device="cuda")
        full[:, :, at:at + 8] = byte
        A, B = full[0], full[1] if layout == "tn" else full[1].t().contiguous()
        c = torch.empty((n, n), device="cuda")
        ones = torch.ones((n, 1), device="cuda")
        L.gemm_fp8_block(layout, n, n, K, A, K, B, K, c, n, ones, torch.ones((1, 1), device="cuda"))
        c = (c.t() if layout == "tn" else c).double()
        x, y = (t.contiguous().view(FP8).double() for t in byte)
        p = x[:, None, :] * y[None]
        exponents = [torch.clamp(torch.frexp(t.abs())[1] - 1, min=-6) for t in (x, y)]
        E = torch.where(p != 0, exponents[0][:, None, :] + exponents[1][None], -99).amax(2, keepdim=True)
        step = torch.exp2(E.double() - 13)
        assert torch.equal(c, (torch.trunc(p / step) * step).sum(2))
        assert bool(((c - p.sum(2)).abs() <= 7 * 2.0 ** -10 * p.abs().sum(2)).all())


def test_a_subnormal_value_in_the_largest_product():
    """288 * 2^-9 = 0.5625 counts as 2^(8 - 6): its neighbours end at 2^-11, 0.00139 at 2 of those, 0.0349 at 71."""
    L = lib()
    a, b = torch.zeros((16, 128), device="cuda"), torch.zeros((16, 128), device="cuda")
    a[:, :4] = torch.tensor([-0.05078125, 0.34375, -288.0, -3.25])
    b[:, :4] = torch.tensor([-0.02734375, 0.1015625, -2.0 ** -9, 0.005859375])
    c = L.matmul(a.to(FP8), b.to(FP8).t(), scale_a=torch.ones((16, 1), device="cuda"),
                 scale_b=torch.ones((1, 16), device="cuda"), out_dtype=torch.float16)
    want = 0.5625 + 71 * 2.0 ** -11 + 2 * 2.0 ** -11 - 0.01904296875
    assert bool((c == torch.tensor(want, dtype=torch.float16)).all())
    p = a[0].double() * b[0].double()
    assert 7 * 2.0 ** -13 * float(p.abs().sum()) < float(p.sum()) - want < 7 * 2.0 ** -10 * float(p.abs().sum())


@pytest.mark.parametrize("K", [1, 15, 17, 100, 127])
def test_narrow_products_whatever_the_padding_holds(K):
    """K <= 128, where factors of blocks are vectors too, results in float32: padding of NaN has no part in it."""
    L = lib()
    g = gen(K)
    a, b = fp8s(g, (50, K)), fp8s(g, (70, K))
    sa, sb = factors(g, 50, K, 1), factors(g, 70, K, 1)
    c64, mass = exact(a, b, sa, sb)
    near(L.matmul(a, b.t(), scale_a=sa, scale_b=sb.t()), c64, mass, K)
    q, sq = L.quantize_fp8(torch.randn((50, K), generator=g, device="cuda"))
    q.as_strided((50, q.stride(0)), (q.stride(0), 1)).view(torch.uint8)[:, K:] = 0x7f
    c64, mass = exact(q, b, sq, sb)
    near(L.matmul(q, b.t(), scale_a=sq, scale_b=sb.t()), c64, mass, K, 7 * 2.0 ** -13 + 127 * 2.0 ** -23)


@pytest.mark.parametrize("layout", ["tn", "nn"])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_single_rows_and_columns(layout, dtype):
    L = lib()
    for M, N, K in ((1, 1, 1), (1, 1, 300), (1, 200, 129), (200, 1, 129), (1, 1, 5000)):
        for ba, bb in ((1, 1), (128, 1), (1, 128)):
            g = gen(M + N + K)
            a = fp8s(g, (M, K))
            bt = fp8s(g, (N, K))
            sa, sb = factors(g, M, K, ba), factors(g, N, K, bb)
            c = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
            A = a.as_strided((M, a.stride(0)), (a.stride(0), 1))
            if layout == "tn":
                ldb, ldc, B = bt.stride(0), M, bt.as_strided((N, bt.stride(0)), (bt.stride(0), 1))
                c = c.t().contiguous()
            else:
                ldb, ldc = -(-N // 16) * 16, N
                B = torch.full((K, ldb), 0x7f, dtype=torch.uint8, device="cuda")
                B[:, :N] = bt.view(torch.uint8).t()
            L.gemm_fp8_block(layout, M, N, K, A, a.stride(0), B, ldb, c, ldc, sa, sb)
            c64, mass = exact(a, bt, sa, sb)
            near(c.t() if layout == "tn" else c, c64, mass, K)


@pytest.mark.parametrize("layout", ["tn", "nn"])
def test_factors_of_128_rows_on_both_sides(monkeypatch, layout):
    """Tiles along either operand that begin inside such a block of rows, on every kernel."""
    L = lib()
    M, N, K = 700, 650, 400
    g = gen(17)
    a, bt = fp8s(g, (M, K)), fp8s(g, (N, K))
    sa, sb = factors(g, M, K, 128), factors(g, N, K, 128)
    c64, mass = exact(a, bt, sa, sb)
    A = a.as_strided((M, a.stride(0)), (a.stride(0), 1))
    if layout == "tn":
        ldb, ldc, B = bt.stride(0), M, bt.as_strided((N, bt.stride(0)), (bt.stride(0), 1))
    else:
        ldb, ldc = 656, N
        B = torch.full((K, ldb), 0x7f, dtype=torch.uint8, device="cuda")
        B[:, :N] = bt.view(torch.uint8).t()
    for name in kernels(layout, "bf16"):
        monkeypatch.setenv("DGEMM_CONFIG", name)
        c = torch.full((N, M) if layout == "tn" else (M, N), 7.0, dtype=torch.bfloat16, device="cuda")
        L.gemm_fp8_block(layout, M, N, K, A, a.stride(0), B, ldb, c, ldc, sa, sb)
        near(c.t() if layout == "tn" else c, c64, mass, K)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_matmul_of_single_rows_and_columns_of_any_width(dtype):
    """One token, one channel, one k, straight from the quantisation, whose pitch a single row's stride does not say."""
    L = lib()
    for K in (1, 17, 100, 112, 127, 128, 129, 300):
        for M, N in ((1, 70), (50, 1), (1, 1), (1, 200), (20, 30)):
            g = gen(K)
            x, w = torch.randn((M, K), generator=g, device="cuda"), torch.randn((N, K), generator=g, device="cuda")
            for ba, bb in ((1, 128), (1, 1)):
                a, sa = L.quantize_fp8(x, block_rows=ba)
                b, sb = L.quantize_fp8(w, block_rows=bb)
                c64, mass = exact(a, b, sa, sb)
                near(L.matmul(a, b.t(), scale_a=sa, scale_b=sb.t(), out_dtype=dtype), c64, mass, K, CUT)
                bt, sbt = L.quantize_fp8(w.t(), block_rows=128) if bb == 128 else (None, None)
                if bt is not None:                          # row-major: its factors are those of blocks of k as well
                    c64, mass = exact(a, bt.t(), sa, sbt.t())
                    near(L.matmul(a, bt, scale_a=sa, scale_b=sbt, out_dtype=dtype), c64, mass, K, CUT)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_matmul_takes_factors_of_any_stride_with_one_block_of_k(dtype):
    """A column of a larger matrix of factors, as with more blocks of k."""
    L = lib()
    for M, N, K in ((50, 70, 100), (130, 300, 128), (1, 70, 17), (50, 1, 16)):
        g = gen(M)
        a, b = fp8s(g, (M, K)), fp8s(g, (N, K))
        for ba, bb in ((1, 1), (1, 128), (128, 1)):
            sa, sb = factors(g, M, K + 256, ba).contiguous()[:, 1:2], factors(g, N, K + 256, bb).contiguous()[:, 2:3]
            c64, mass = exact(a, b, sa, sb)
            near(L.matmul(a, b.t(), scale_a=sa, scale_b=sb.t(), out_dtype=dtype), c64, mass, K)
            near(L.matmul(a, b.t(), scale_a=sa.contiguous(), scale_b=sb.t(), out_dtype=dtype), c64, mass, K)


def test_matmul_refuses_factors_of_128_rows_on_both_sides():
    """Whatever their number of values: they are never read as one for each row."""
    L = lib()
    for M, N, K in ((64, 64, 8192), (16, 16, 2048), (300, 200, 400)):
        g = gen(M)
        a, b = fp8s(g, (M, K)), fp8s(g, (N, K))
        sa, sb = factors(g, M, K, 128), factors(g, N, K, 128)
        for dtype in TYPES:
            with pytest.raises(ValueError, match="one for each row"):
                L.matmul(a, b.t(), scale_a=sa, scale_b=sb.t(), out_dtype=dtype)


STRIPS = [(order, rows, few, stages) for order in "ab" for rows, few, depth in
          ((16, 16, 2), (16, 32, 2), (32, 16, 2), (32, 32, 2), (32, 64, 1)) for stages in range(1, depth + 1)]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("strip", STRIPS, ids=lambda s: "{}-{}x{}-{}".format(*s))
def test_every_strip_of_few_rows(monkeypatch, strip, dtype):
    """TN strips against either operand as the few rows, with one and two stages of copies in flight: fewer stages than
    waves and many more, K whole, ending inside a block and inside a chunk of 16, ragged strips on both sides."""
    import ctypes
    h = lib().load_library()
    order, rows, few, stages = strip
    tag = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}[dtype]
    name = f"b8{tag}_tn_skinny_{order}"
    monkeypatch.setenv("DGEMM_CONFIG", f"{name}:{rows}x{few}x{stages}")
    buf = ctypes.create_string_buffer(256)
    assert h.dgemm_fp8_block_config(TYPES.index(dtype), 1, 1, 128, 700, 700, 700, buf, 256) == 0
    tile = f"{few}x{rows}" if order == "a" else f"{rows}x{few}"
    lds = max(8 * stages * ((rows + few) * 128 + 512), 4 * 8 * rows * few)
    assert buf.value.decode().startswith(f"{name} tile={tile} threads=512 lds={lds} "), buf.value
    for i, (M, N, K) in enumerate(((1, 1, 1), (33, 130, 129), (130, 33, 512), (64, 64, 1000), (129, 70, 2048),
                                   (70, 129, 2315), (31, 200, 4111), (200, 31, 5000))):
        for ba, bb in ((128, 1), (1, 128), (1, 1)):
            if K > 128 or dtype != torch.float32:            # (one block, FP32 results: the path of vectors)
                product(gen(i), "tn", M, N, K, ba, bb, dtype, order="rows" if i % 2 else "blocks")


def test_strips_chosen_by_size():
    """Sizes that take strips of their own accord, many rows on either side."""
    import ctypes
    h = lib().load_library()
    buf = ctypes.create_string_buffer(256)
    seen = set()
    for i, (M, N, K) in enumerate(((7788, 1, 2315), (57, 1813, 6839), (3507, 62, 2909), (354, 1220, 300), (7362, 44, 300),
                                   (8192, 16, 8192), (16, 8192, 8192), (20, 5000, 2100), (5000, 40, 2100), (40, 5000, 2100),
                                   (300, 17, 4096), (17, 300, 4096), (600, 33, 700), (33, 600, 700))):
        assert h.dgemm_fp8_block_config(2, 1, 128, 1, M, N, K, buf, 256) == 0
        seen.add(" ".join(buf.value.decode().split()[:4]))
        product(gen(200 + i), "tn", M, N, K, 128, 1, torch.bfloat16)
        product(gen(300 + i), "tn", M, N, K, 1, 128, torch.float16)
    assert sum("skinny" in s for s in seen) >= 8, seen


def test_quantize_into_part_of_a_matrix():
    L = lib()
    x = torch.randn((130, 200), generator=gen(5), device="cuda")
    for turned in (False, True):
        for block in (1, 128):
            src = x.t().contiguous().t() if turned else x
            want, ws = L.quantize_fp8(src, block_rows=block)
            room = torch.full((140, 256), 0x55, dtype=torch.uint8, device="cuda").view(FP8)
            scales = torch.full((140, 5), -1.0, device="cuda")
            n = ws.shape[0]
            L.quantize_fp8(src, block_rows=block, out=room[3:133, 16:216], scale=scales[2:2 + n, 1:3])
            bytes_ = room.view(torch.uint8)
            assert torch.equal(bytes_[3:133, 16:216], want.contiguous().view(torch.uint8))
            assert torch.equal(scales[2:2 + n, 1:3], ws)
            bytes_[3:133, 16:216] = 0x55
            scales[2:2 + n, 1:3] = -1.0
            assert bool((bytes_ == 0x55).all()) and bool((scales == -1.0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("block", [1, 128])
def test_quantize_many_rows_of_odd_numbers(dtype, block):
    """Enough rows for two a wave, the last one alone; a last group of column-major tiles that is not full."""
    L = lib()
    for rows, K, turned in ((16387, 1029, False), (2691, 300, True), (2049, 8193, False)):
        g = gen(rows)
        x = torch.randn((K, rows) if turned else (rows, K), generator=g, device="cuda").to(dtype)
        x = x.t() if turned else x
        q, s = L.quantize_fp8(x, block_rows=block)
        check_quantised(x, q, s, block)


def test_quantize_refuses_scales_that_overlap():
    L = lib()
    x = torch.ones((4, 300), device="cuda")
    one = torch.zeros((1,), device="cuda")
    with pytest.raises(L.DgemmError):
        L.quantize_fp8(x, scale=one.expand(4, 3))
    with pytest.raises(L.DgemmError):
        L.quantize_fp8(x, scale=torch.zeros((4, 1), device="cuda").expand(4, 3))


def test_grouped_index_names_rows_twice_and_none():
    L = lib()
    g = gen(9)
    a, sa = fp8s(g, (10, 300)), factors(g, 10, 300, 1)
    b, sb = fp8s(g, (3, 70, 300)), torch.rand((3, 1, 3), generator=g, device="cuda")
    index = torch.tensor([4, 4, 4, -1, 10, 9, 0, 2 ** 31 - 1, -2 ** 31, 4], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 5, 5, 9], dtype=torch.int32, device="cuda")
    out = torch.full((10, 70), 3.0, device="cuda")
    L.matmul_grouped(a, b, off, sa, sb, out=out, row_index=index)
    for r, e in enumerate((0, 0, 0, 0, 0, 2, 2, 2, 2)):
        i = int(index[r])
        if not 0 <= i < 10:
            assert bool((out[r] == 0).all())
            continue
        c64, mass = exact(a[i:i + 1], b[e], sa[i:i + 1], sb[e])
        near(out[r:r + 1], c64, mass, 300)
    assert bool((out[9] == 3.0).all())          # behind the last group: left


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_grouped_rows_of_no_source_are_zeros_whatever_the_weights_hold(monkeypatch, dtype):
    """Weights of NaN and factors of infinity and NaN reach the rows that have a source, not those whose index names
    none, on every kernel."""
    L = lib()
    tag = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}[dtype]
    for name in GROUPED:
        monkeypatch.setenv("DGEMM_CONFIG", f"b8{tag}_grouped_{name}")
        for counts, N, K in (([5, 40, 3], 200, 256), ([130, 0, 300], 390, 400), ([1, 1, 1], 64, 100)):
            g = gen(N)
            rows = sum(counts)
            a, sa = fp8s(g, (37, K)), factors(g, 37, K, 1).contiguous()
            b, sb = fp8s(g, (3, N, K)), torch.stack([factors(g, N, K, 128) for _ in counts]).contiguous()
            b.view(torch.uint8)[0, 7, 5] = 0x7f
            sb[0, -1, 0], sb[2, 0, -1], sb[2, -1, 0] = float("inf"), float("nan"), -float("inf")
            sa[11] = float("nan")
            index = torch.randint(0, 37, (rows,), generator=g, device="cuda", dtype=torch.int32)
            index[::3] = torch.tensor([-1, 37, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")[
                torch.randint(0, 4, (len(index[::3]),), generator=g, device="cuda")]
            off = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
            out = torch.full((rows, N), 3.0, dtype=dtype, device="cuda")
            L.matmul_grouped(a, b, off, sa, sb, out=out, row_index=index)
            none = (index < 0) | (index >= 37)
            assert bool((out[none] == 0).all()), name
            some = torch.arange(rows, device="cuda") < counts[0]     # of the first expert
            assert bool(torch.isnan(out[some & ~none][:, 7]).all()), name


# ---- places past 2^32 ---------------------------------------------------------------

def blob(g, shape):
    """E4M3 within four binades, cheaply: one row's bytes rolled on by row."""
    n = int(np.prod(shape))
    out = torch.empty((n,), dtype=torch.uint8, device="cuda")
    part = torch.randint(40, 72, (min(n, (1 << 24) + 17),), generator=g, device="cuda", dtype=torch.uint8)
    for at in range(0, n, part.numel()):
        out[at:at + part.numel()] = part[:min(part.numel(), n - at)]
    return out.view(FP8).reshape(shape)


def test_operands_and_results_past_32_bits():
    L = lib()
    g = gen(41)
    # Many rows of A, a few of B, and the other way round.
    M, N, K = 300000, 16, 16384
    a, b = blob(g, (M, K)), blob(g, (N, K))
    sa, sb = factors(g, M, K, 1), factors(g, N, K, 128)
    at = slice(M - 300, M)
    c64, mass = exact(a[at], b, sa[at], sb)
    c = L.matmul(a, b.t(), scale_a=sa, scale_b=sb.t(), out_dtype=torch.bfloat16)
    near(c[at], c64, mass, K)
    c = L.matmul(b, a.t(), scale_a=sb, scale_b=sa.t(), out_dtype=torch.bfloat16)
    near(c[:, at].t(), c64, mass, K)
    del a, c
    # A result of more than 2^32 elements.
    M, N, K = 131072, 33000, 128
    a, b = blob(g, (M, K)), blob(g, (N, K))
    sa, sb = factors(g, M, K, 128), factors(g, N, K, 1)
    c = L.matmul(a, b.t(), scale_a=sa, scale_b=sb.t(), out_dtype=torch.bfloat16)
    cut = slice(N - 40, N)
    c64, mass = exact(a, b[cut], sa, sb[cut])
    near(c[:, cut], c64, mass, K)


def test_experts_past_32_bits():
    L = lib()
    g = gen(42)
    E, N, K, T, k = 20, 16384, 14336, 6, 2
    b = blob(g, (E, N, K))
    sb = torch.rand((E, N // 128, K // 128), generator=g, device="cuda")
    a, sa = fp8s(g, (T, K)), factors(g, T, K, 1)
    off = torch.zeros((E + 1,), dtype=torch.int32, device="cuda")
    off[E - 1:] = torch.tensor([4, 6], dtype=torch.int32, device="cuda")
    off[1:E - 1] = 4
    out = L.matmul_grouped(a, b, off, sa, sb, out_dtype=torch.bfloat16)
    for e, at in ((0, slice(0, 4)), (E - 1, slice(4, 6))):
        c64, mass = exact(a[at], b[e], sa[at], sb[e])
        near(out[at], c64, mass, K)


def test_quantize_and_route_past_32_bits():
    L = lib()
    g = gen(43)
    rows, K = 270000, 16384
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    part = torch.randn((1000, K), generator=g, device="cuda").to(torch.bfloat16)
    x.view(270, 1000, K).copy_(part)
    for block in (1, 128):
        q, s = L.quantize_fp8(x, block_rows=block)
        at = slice(rows - 1000 + 1000 % 128, rows) if block == 1 else slice(rows // 128 * 128 - 1280, rows)
        wq, ws = L.quantize_fp8(x[at], block_rows=block)
        assert torch.equal(q[at].view(torch.uint8), wq.view(torch.uint8))
        assert torch.equal(s[-ws.shape[0]:], ws)
        del q, s
    xt = x.view(K, rows).t()         # column-major, rows contiguous
    q, s = L.quantize_fp8(xt)
    wq, ws = L.quantize_fp8(xt[-300:].t().contiguous().t())
    assert torch.equal(q[-300:].contiguous().view(torch.uint8), wq.contiguous().view(torch.uint8))
    assert torch.equal(s[-300:], ws)
    del x, xt, q, s
    T, E = (1 << 22) + 5, 1024
    logits = torch.empty((T, E), dtype=torch.bfloat16, device="cuda")
    logits[:-5].view(4096, 1024, E).copy_(torch.randn((1024, E), generator=g, device="cuda").to(torch.bfloat16))
    logits[-5:] = logits[:5] * 2
    ids, w = L.expert_route(logits, 4)
    wi, ww = L.expert_route(logits[-500:].contiguous(), 4)
    assert torch.equal(ids[-500:], wi) and torch.equal(w[-500:], ww)
    d = L.expert_route_grad(w, logits, ids, renormalize=False)
    assert torch.equal(d[-500:], L.expert_route_grad(ww, logits[-500:].contiguous(), wi, renormalize=False))


# ---- several at once -----------------------------------------------------------------

def layer_of(seed, T=40, E=16, k=4, N=264, K=400):
    L = lib()
    g = gen(seed)
    b, sb = zip(*[L.quantize_fp8(torch.randn((N, K), generator=g, device="cuda"), block_rows=128) for _ in range(E)])
    b, sb = torch.stack([t.view(torch.uint8) for t in b]).view(FP8), torch.stack(sb)
    x = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)
    gate = torch.randn((K, E), generator=g, device="cuda").to(torch.bfloat16) * 0.05
    logits = x @ gate

    def run():
        ids, w = L.expert_route(logits, k, score="sigmoid", groups=4, top_groups=2, group_best=2)
        y = L.matmul_experts(x, ids, w, b, sb)
        return y, L.expert_route_grad(w, logits, ids, score="sigmoid")

    return x, logits, run


def test_threads_on_their_own_streams():
    """The layer from four threads at once, each on a stream of its own, gives what it gives alone."""
    made = [layer_of(s, T=30 + 50 * s) for s in range(4)]
    want = [run() for _, _, run in made]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = made[i][2]()
                stream.synchronize()
                if not all(torch.equal(p, q) for p, q in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_two_captured_layers_replayed_side_by_side():
    made = [layer_of(s) for s in (7, 8)]
    graphs = []
    for _, _, run in made:
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        graphs.append((graph, out))
    streams = [torch.cuda.Stream() for _ in graphs]
    for seed in range(4):
        for x, logits, _ in made:
            x.copy_(torch.randn(x.shape, generator=gen(seed), device="cuda").to(x.dtype))
            logits.copy_(torch.randn(logits.shape, generator=gen(seed + 9), device="cuda").to(logits.dtype))
        torch.cuda.synchronize()
        for s, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (_, out), (_, _, run) in zip(graphs, made):
            assert all(torch.equal(p, q) for p, q in zip(out, run()))


def test_streams_by_handle():
    L = lib()
    x = torch.randn((64, 512), generator=gen(1), device="cuda")
    want, ws = L.quantize_fp8(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, s = L.quantize_fp8(x, stream=side.cuda_stream)
    ids, w = L.expert_route(x, 5, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8)) and torch.equal(s, ws)
    check(x, 5)
    assert torch.equal(ids, L.expert_route(x, 5)[0])
