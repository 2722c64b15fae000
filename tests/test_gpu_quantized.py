"""GPU tests of the int8 linear layers against plain implementations in 64
bits: rows to int8, the int8 product with scales, and the grouped products.

Tolerances count roundings.  A product's sum is an exact integer; FP32 then
rounds it, the product of the two factors and the product of both, half a
step (2^-24) each, and the output type rounds once more by at most half a step:
|c - c64| <= (3 * 2^-24 * (1 + 2^-10) + eps / 2) |c64|, plus half the output
type's smallest step next to zero.  Quantised values are compared bit for bit:
a quotient in 64 bits is off by 2^-53, and no quotient of two FP32 numbers up
to 127.5 that is not the middle of two integers itself comes nearer to one
than 2^-32 of its value."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]
IDS = ["f32", "f16", "bf16"]
HALF = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def lib():
    import dense_gemm_02_amd as L
    return L


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(g, shape, pad=0):
    """int8 values over the whole range in rows of a pitch that is a multiple
    of 16, the padding filled with other values."""
    cols = -(-shape[-1] // 16) * 16 + 16 * pad
    q = torch.randint(-128, 128, shape[:-1] + (cols,), generator=g, device="cuda", dtype=torch.int8)
    return q[..., :shape[-1]]


def factors(g, n):
    return torch.rand((n,), generator=g, device="cuda") * 0.02 + 1e-4


def exact(a, b, sa, sb):
    """(a @ b) * sa * sb in 64 bits (the sums are exact)."""
    return (a.double() @ b.double().contiguous()) * (sa.double().reshape(-1, 1) * sb.double().reshape(1, -1))


def near(c, c64):
    u = 3 * 2.0 ** -24 * (1 + 2.0 ** -10) + HALF[c.dtype]
    bad = (c.double() - c64).abs() > u * c64.abs() + TINY[c.dtype]
    assert not bad.any(), (int(bad.sum()), float((c.double() - c64).abs().max()))


# ---- quantize_i8 ------------------------------------------------------------------

def plain_quantize(x):
    x = x.double()
    amax = x.abs().amax(1) if x.shape[1] else x.new_zeros(x.shape[0])
    scale = (amax / 127).float()
    s = scale.double()[:, None]
    ok = torch.isfinite(s) & (s > 0)
    q = torch.round(torch.where(ok, x / torch.where(ok, s, 1.0), 0.0)).clamp(-127, 127).to(torch.int8)
    return q, scale


def check_quantize(x, **kw):
    q, scale = lib().quantize_i8(x, **kw)
    q0, s0 = plain_quantize(x)
    assert torch.equal(torch.nan_to_num(scale, 7.0), torch.nan_to_num(s0, 7.0))
    assert torch.equal(torch.isnan(scale), torch.isnan(s0))
    assert torch.equal(q, q0), int((q != q0).sum())
    return q, scale


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 16), (3, 7), (2, 63), (5, 64), (7, 65), (4, 255), (9, 256), (6, 257),
                                    (33, 1000), (17, 2048), (5, 4096), (3, 4100), (2, 8192), (3, 8193), (2, 16384),
                                    (2, 16391), (1, 40000), (300, 513), (1025, 128)])
def test_quantize_sizes(dtype, rows, K):
    print(f"quantize {dtype} {rows}x{K}", flush=True)
    g = gen(rows * 31 + K)
    x = torch.randn((rows, K), generator=g, device="cuda") * torch.exp(torch.randn((rows, 1), generator=g,
                                                                                     device="cuda"))
    check_quantize(x.to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_quantize_strides_and_offsets(dtype):
    # rows off every alignment, results into a wider matrix whose rest stays
    base = torch.randn((40, 1037), generator=gen(3), device="cuda").to(dtype)
    for off in (0, 1, 2, 3, 5, 8):
        for K in (1, 100, 512, 1000):
            x = base[:, off:off + K]
            out = torch.full((40, 1100), 99, dtype=torch.int8, device="cuda")
            scale = torch.full((42,), -1.0, device="cuda")
            q, s = check_quantize(x, out=out[:, off + 1:off + 1 + K], scale=scale[1:41])
            assert (out[:, :off + 1] == 99).all() and (out[:, off + 1 + K:] == 99).all()
            assert scale[0] == -1 and scale[41] == -1
    check_quantize(base[::3, 5:900])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_quantize_middles(dtype):
    """Quotients on and next to the middle between two integers: rows whose
    scale is a power of two, so that x / scale is exact, and values one step
    to either side."""
    for e in (-9, -2, 0, 3):
        s = 2.0 ** e
        mid = (torch.arange(-127, 127, device="cuda") + 0.5) * s
        t = mid.to(dtype)
        up = torch.nextafter(mid.float(), torch.tensor(float("inf"), device="cuda")).to(dtype)
        dn = torch.nextafter(mid.float(), torch.tensor(-float("inf"), device="cuda")).to(dtype)
        x = torch.cat([t, up, dn, torch.tensor([127.0 * s], device="cuda").to(dtype)])[None]
        assert float(x.abs().max()) == 127 * s
        check_quantize(x)
    # scales of every mantissa, values at the nearest type value to a middle
    g = gen(5)
    amax = torch.rand((400, 1), generator=g, device="cuda") + 1
    x = ((torch.randint(0, 127, (400, 300), generator=g, device="cuda") + 0.5) * (amax.to(dtype).float() / 127))
    x = torch.cat([amax, x.clamp(max=1) * 1.0], 1).to(dtype)
    check_quantize(x)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_quantize_special_rows(dtype):
    x = torch.randn((12, 300), generator=gen(9), device="cuda").to(dtype)
    x[0] = 0
    x[1, 7] = float("inf")
    x[2, 299] = -float("inf")
    x[3, 0] = float("nan")
    x[4, 5], x[4, 6] = float("nan"), float("inf")
    x[5] = torch.finfo(dtype).max
    x[6] = torch.finfo(dtype).tiny
    x[7] = 0
    x[7, 3] = torch.finfo(dtype).smallest_normal
    x[8] = x[8].sign() * torch.finfo(dtype).max
    if dtype != torch.float16:   # subnormals of the scale
        x[9] *= 2.0 ** -120
        x[10] *= 1e-38
        x[11] = torch.arange(300, device="cuda").to(dtype) * 2.0 ** -133
    q, s = check_quantize(x)
    assert s[0] == 0 and (q[:5] == 0).all()
    assert torch.isinf(s[1]) and torch.isinf(s[2]) and torch.isnan(s[3]) and torch.isnan(s[4])


def test_quantize_empty():
    L = lib()
    q, s = L.quantize_i8(torch.empty((0, 5), device="cuda"))
    assert q.shape == (0, 5) and s.shape == (0,)
    q, s = L.quantize_i8(torch.empty((4, 0), device="cuda"))
    assert q.shape == (4, 0) and (s == 0).all()


# ---- the product ------------------------------------------------------------------

EDGE = [1, 2, 3, 7, 15, 16, 17, 31, 32, 33, 47, 64, 65, 127, 128, 129, 255, 256, 257, 300]


def shapes(seed, n=22):
    rng = np.random.default_rng(seed)
    out = [(1, 1, 1), (1, 1, 70), (70, 1, 1), (1, 70, 1), (257, 255, 129), (33, 65, 300), (16, 300, 515),
           (300, 16, 517), (32, 257, 1024), (513, 5, 2050), (40, 48, 4100)]
    return out + [tuple(int(rng.choice(EDGE)) for _ in range(3)) for _ in range(n)]


def operands(layout, M, N, K, seed, pad=0):
    g = gen(seed)
    a = ints(g, (M, K), pad)
    b = ints(g, (N, K), pad).t() if layout == "tn" else ints(g, (K, N), pad)
    return a, b, factors(g, M), factors(g, N)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("layout", ["tn", "nn"])
def test_product_small_shapes(layout, dtype):
    for i, (M, N, K) in enumerate(shapes(11 + len(layout))):
        print(f"product {layout} {dtype} {M}x{N}x{K}", flush=True)
        a, b, sa, sb = operands(layout, M, N, K, 100 + i, pad=i % 3)
        c = lib().matmul(a, b, scale_a=sa, scale_b=sb, out_dtype=dtype)
        assert c.dtype == dtype and c.shape == (M, N)
        near(c, exact(a, b, sa, sb))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("layout,M,N,K", [
    ("tn", 600, 520, 333), ("nn", 515, 777, 1029), ("tn", 1024, 256, 64), ("nn", 1024, 256, 4096),
    ("tn", 2048, 2048, 512), ("tn", 4096, 4096, 256), ("nn", 4096, 4097, 272), ("tn", 4099, 4093, 387),
    ("tn", 2560, 2304, 1040), ("tn", 1536, 4352, 4096), ("tn", 4352, 1536, 4112), ("nn", 4352, 1536, 4100)])
def test_product_tiles(layout, M, N, K, dtype):
    print(f"product {layout} {dtype} {M}x{N}x{K}", flush=True)
    a, b, sa, sb = operands(layout, M, N, K, M + N + K, pad=1)
    near(lib().matmul(a, b, scale_a=sa, scale_b=sb, out_dtype=dtype), exact(a, b, sa, sb))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("many", [1, 15, 31, 33, 250, 8159, 8161, 8200])
def test_product_few_rows(many, dtype):
    """Few rows on either side of the product, each number of 16-row tiles and
    its edges, K whole, inside a chunk, below a stage and over many."""
    for few in (1, 15, 16, 17, 32, 33, 63, 64, 65, 100, 128):
        for K in (1, 128, 500, 2048, 4240) if few in (1, 17, 64, 100) else (333,):
            if many > 300 and few not in (1, 17, 64, 100):
                continue
            print(f"few {few} many {many} K={K} {dtype}", flush=True)
            a, b, sa, sb = operands("tn", few, many, K, few + many + K, pad=K % 2)
            near(lib().matmul(a, b, scale_a=sa, scale_b=sb, out_dtype=dtype), exact(a, b, sa, sb))
            near(lib().matmul(b.t(), a.t(), scale_a=sb, scale_b=sa, out_dtype=dtype), exact(b.t(), a.t(), sb, sa))
            a, b, sa, sb = operands("nn", few, many, K, few + many + K, pad=K % 2)
            near(lib().matmul(a, b, scale_a=sa, scale_b=sb, out_dtype=dtype), exact(a, b, sa, sb))
            a, b, sa, sb = operands("nn", many, few, K, few + many + K, pad=K % 2)
            near(lib().matmul(a, b, scale_a=sa, scale_b=sb, out_dtype=dtype), exact(a, b, sa, sb))


# (M, N) that make the skinny kernels take each of their tiles (p x q).
SKINNY = [
    ("nn", "16x16", 3, 5), ("nn", "16x16", 37, 212), ("nn", "16x32", 4428, 11), ("nn", "32x16", 7, 5018),
    ("nn", "32x32", 17, 5077), ("nn", "32x64", 4728, 33), ("nn", "32x128", 65, 5544), ("nn", "64x16", 2, 11341),
    ("nn", "64x32", 19, 11294), ("nn", "64x64", 33, 11088), ("nn", "64x128", 67, 11757), ("nn", "128x16", 1, 26184),
    ("nn", "128x32", 17, 26188), ("nn", "128x64", 34, 29448),
    ("tn", "128x32", 69, 7056), ("tn", "16x16", 5, 9), ("tn", "16x32", 3, 6219), ("tn", "32x16", 20, 3269),
    ("tn", "32x32", 18, 5677), ("tn", "64x32", 34, 6335), ("tn", "16x32", 3170, 18), ("tn", "32x128", 6845, 65),
    ("tn", "32x16", 6174, 1), ("tn", "32x32", 5601, 18), ("tn", "32x64", 6295, 35), ("tn", "16x32", 300, 511)]


@pytest.mark.parametrize("layout,tile,M,N", SKINNY)
def test_product_every_skinny_tile(layout, tile, M, N):
    """K below a stage (128), a whole number of stages, ending inside one and
    inside a chunk, and more stages than waves; factors one or one a row."""
    import ctypes
    L = lib()
    buf = ctypes.create_string_buffer(256)
    for K in (1, 100, 128, 500, 1024, 2100, 2560):
        assert L.load_library().dgemm_kernel_config(7, 1 if layout == "tn" else 0, M, N, K, buf, 256) == 0
        assert "skinny" in buf.value.decode() and f"tile={tile} " in buf.value.decode(), buf.value
        a, b, sa, sb = operands(layout, M, N, K, M + N + K, pad=K % 3)
        for dtype in TYPES:
            print(f"skinny {layout} {tile} {M}x{N}x{K} {dtype}", flush=True)
            near(L.matmul(a, b, scale_a=sa, scale_b=sb, out_dtype=dtype), exact(a, b, sa, sb))
        near(L.matmul(a, b, scale_a=sa[:1], scale_b=sb[:1]), exact(a, b, sa[:1], sb[:1]))


TILES_TN = ["256x256_w4", "128x128_w4", "128x128_w4_s4", "192x256_w4", "256x192_w4", "256x256_pp",
            "64x128_w4", "64x128_w4_s4"]
TILES_NN = ["256x256_w4", "256x128_w4", "256x192_w4"]


@pytest.mark.parametrize("layout,tile", [("tn", t) for t in TILES_TN] + [("nn", t) for t in TILES_NN])
@pytest.mark.parametrize("tag,dtype", [("i8f", torch.float32), ("i8h", torch.float16), ("i8b", torch.bfloat16)])
def test_product_every_kernel_every_tail(monkeypatch, layout, tile, tag, dtype):
    """Each block kernel from one stage of K (128) to five, whole and ending
    inside a chunk, on ragged tiles."""
    monkeypatch.setenv("DGEMM_CONFIG", f"{tag}_{layout}_{tile}")
    for K in (1, 16, 100, 128, 129, 200, 256, 257, 384, 399, 512, 600, 639):
        M, N = 300, 333
        print(f"{tag} {layout} {tile} K={K}", flush=True)
        a, b, sa, sb = operands(layout, M, N, K, K)
        near(lib().matmul(a, b, scale_a=sa, scale_b=sb, out_dtype=dtype), exact(a, b, sa, sb))


def test_product_longest_sum():
    """K = 131071 of -128 * -128: the largest sum there is, and it is exact."""
    K = 131071
    a = torch.full((3, -(-K // 16) * 16), -128, dtype=torch.int8, device="cuda")[:, :K]
    b = torch.full((20, -(-K // 16) * 16), -128, dtype=torch.int8, device="cuda")[:, :K]
    one = torch.ones(1, device="cuda")
    for x, y in ((a, b.t()), (b, a.t())):
        c = lib().matmul(x, y, scale_a=one, scale_b=one)
        assert (c == torch.tensor(float(K * 16384), device="cuda")).all()
    with pytest.raises(lib().DgemmError) as e:
        z = torch.zeros((1, 131088), dtype=torch.int8, device="cuda")[:, :131072]
        lib().matmul(z, z.t(), scale_a=one, scale_b=one)
    assert e.value.status == 6


@pytest.mark.parametrize("layout", ["tn", "nn"])
def test_product_factors(layout):
    """One factor or one a row, and what zero, infinite and NaN factors give
    (FP32 rules on the exact sum)."""
    M, N, K = 70, 90, 256
    a, b, sa, sb = operands(layout, M, N, K, 5)
    a[3] = 0
    one = torch.tensor([0.25], device="cuda")
    L = lib()
    near(L.matmul(a, b, scale_a=one, scale_b=sb), exact(a, b, one, sb))
    near(L.matmul(a, b, scale_a=sa, scale_b=one), exact(a, b, sa, one))
    near(L.matmul(a, b, scale_a=one, scale_b=one), exact(a, b, one, one))
    sa[0], sa[1], sb[2], sb[3] = float("inf"), float("nan"), 0.0, float("inf")
    c = L.matmul(a, b, scale_a=sa, scale_b=sb)
    acc = (a.double() @ b.double().contiguous()).float()
    want = acc * (sa[:, None] * sb[None, :])
    assert torch.equal(torch.isnan(c), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(c), torch.nan_to_num(want))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_product_into_part_of_a_matrix(dtype):
    """Results into rows of a wider matrix off every alignment; the rest stays."""
    L = lib()
    for M, N, K, off in ((300, 140, 256, 1), (17, 300, 320, 3), (260, 260, 200, 5)):
        for layout in ("tn", "nn"):
            a, b, sa, sb = operands(layout, M, N, K, off)
            wide = torch.full((N if layout == "tn" else M, (M if layout == "tn" else N) + 13), 7.0, device="cuda")
            wide = wide.to(dtype)
            n = M if layout == "tn" else N
            part = wide[:, off:off + n]
            c = L.matmul(a, b, scale_a=sa, scale_b=sb, out=part.t() if layout == "tn" else part)
            near(c, exact(a, b, sa, sb))
            assert (wide[:, :off] == 7).all() and (wide[:, off + n:] == 7).all()


def test_product_empty():
    L = lib()
    e = torch.empty((0, 32), dtype=torch.int8, device="cuda")
    f = torch.ones((5, 32), dtype=torch.int8, device="cuda")
    one = torch.ones(1, device="cuda")
    assert L.matmul(e, f.t(), scale_a=one, scale_b=one).shape == (0, 5)
    assert L.matmul(f, e.t(), scale_a=one, scale_b=one).shape == (5, 0)
    z = torch.empty((4, 0), dtype=torch.int8, device="cuda")
    assert (L.matmul(z, z.t(), scale_a=one, scale_b=one) == 0).all()
    w = torch.empty((0, 16), dtype=torch.int8, device="cuda")
    assert (L.matmul(z, w, scale_a=one, scale_b=one) == 0).all()


def test_product_after_quantize_is_near_the_float_product():
    """x W^T through quantize_i8 and the product: the error is that of the two
    roundings to int8, half a step of each row's scale: |e| <= sum_k (|x| sw/2 +
    |w| sx/2 + sx sw/4), plus what FP32 and bf16 round."""
    g = gen(21)
    x = torch.randn((37, 500), generator=g, device="cuda")
    w = torch.randn((130, 500), generator=g, device="cuda")
    L = lib()
    (qx, sx), (qw, sw) = L.quantize_i8(x), L.quantize_i8(w)
    y = L.matmul(qw, qx.t(), scale_a=sw, scale_b=sx).t()
    assert y.is_contiguous()
    y64 = x.double() @ w.double().t().contiguous()
    sx, sw = sx.double()[:, None], sw.double()[None, :]
    bound = (x.double().abs().sum(1, keepdim=True) * sw + sx * w.double().abs().sum(1)[None, :]) / 2 + 500 * sx * sw / 4
    assert ((y.double() - y64).abs() <= bound * (1 + 1e-6)).all()


# ---- grouped ----------------------------------------------------------------------

def grouped_case(counts, N, K, seed, gather, rows_a=None, tail=0, lead=0):
    """offsets from counts (starting at row `lead`), `tail` rows behind the
    last group, operands and the exact result (NaN where nothing is written)."""
    g = gen(seed)
    E = len(counts)
    off = torch.tensor([lead] + [lead + int(v) for v in np.cumsum(counts)], dtype=torch.int32, device="cuda")
    rows = lead + int(sum(counts)) + tail
    b = ints(g, (E, N, K))
    sb = factors(g, E * N).reshape(E, N)
    rows_a = rows if not gather else (rows_a or max(1, rows // 2 + 3))
    a, sa = ints(g, (rows_a, K)), factors(g, rows_a)
    idx = torch.randint(0, rows_a, (rows,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    return a, b, off, sa, sb, idx, rows


def grouped_exact(a, b, off, sa, sb, idx, rows):
    out = torch.full((rows, b.shape[1]), float("nan"), dtype=torch.float64, device="cuda")
    o = off.tolist()
    for e in range(b.shape[0]):
        r = torch.arange(o[e], o[e + 1], device="cuda")
        src = r if idx is None else idx.long()[r]
        ok = ((src >= 0) & (src < a.shape[0])).double()[:, None]
        src = src.clamp(0, a.shape[0] - 1)
        out[o[e]:o[e + 1]] = exact(a[src], b[e].t(), sa[src] if sa.numel() > 1 else sa,
                                   sb[e] if sb.numel() > 1 else sb) * ok
    return out


COUNTS = [[1], [0], [5, 0, 3], [0, 0, 7, 0], [16, 16, 16], [17, 1, 33, 0, 64], [128, 127, 129], [300, 1, 0, 600],
          [2] * 40, [0, 1] * 70, [1] * 130, [900]]


@pytest.mark.parametrize("gather", [False, True], ids=["sorted", "gather"])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_grouped_counts(dtype, gather):
    for i, counts in enumerate(COUNTS):
        for N, K in ((96, 256), (200, 77), (1, 16), (513, 600)):
            if len(counts) > 40 and N > 300:
                continue
            print(f"grouped {dtype} {counts[:6]} N={N} K={K}", flush=True)
            tail, lead = (i % 3) * 5, (i % 2) * 3
            c = grouped_case(counts, N, K, 50 + i, gather, tail=tail, lead=lead)
            a, b, off, sa, sb, idx, rows = c
            out = torch.full((rows, N), 7.0, device="cuda").to(dtype)
            got = lib().matmul_grouped(a, b, off, sa, sb, out=out, row_index=idx)
            want = grouped_exact(*c)
            written = ~torch.isnan(want[:, 0])
            assert (got[~written] == 7).all()
            near(got[written], want[written])


@pytest.mark.parametrize("gather", [False, True], ids=["sorted", "gather"])
@pytest.mark.parametrize("counts,N,K", [([700, 3, 1500, 0, 290], 1000, 1024), ([256] * 8, 512, 2048),
                                        ([4000, 100], 384, 512), ([40] * 32, 768, 1040), ([1100] * 3, 2304, 912),
                                        ([8] * 64, 512, 2048), ([24] * 16, 1024, 1111)])
def test_grouped_larger(counts, N, K, gather):
    c = grouped_case(counts, N, K, N + K, gather)
    print(f"grouped {counts[:6]} N={N} K={K}", flush=True)
    near(lib().matmul_grouped(*c[:5], out_dtype=torch.bfloat16, row_index=c[5]), grouped_exact(*c))


@pytest.mark.parametrize("gather", [False, True], ids=["sorted", "gather"])
@pytest.mark.parametrize("kernel", ["256x256_pp", "128x128_w4", "128x128_w4_s4", "128x64_w4_s4", "skinny16", "skinny32", "skinny64"])
def test_grouped_every_kernel(monkeypatch, kernel, gather):
    """Each kernel a grouped product can take, on groups below, at and past its
    tile, K from below a stage to several, whole and ending inside a chunk."""
    monkeypatch.setenv("DGEMM_CONFIG", "i8_grouped_" + kernel)
    for i, (counts, N) in enumerate((([1, 0, 15, 16, 17, 0, 33], 70), ([257, 31, 128, 0, 64, 65], 300),
                                     ([0, 300, 1], 513), ([3] * 70, 40))):
        for K in (1, 100, 128, 256, 399, 1040):
            for dtype in TYPES:
                print(f"grouped {kernel} {counts[:6]} N={N} K={K} {dtype}", flush=True)
                c = grouped_case(counts, N, K, 70 + i + K, gather, tail=3, lead=2)
                got = torch.full((c[6], N), 7.0, device="cuda").to(dtype)
                lib().matmul_grouped(*c[:5], out=got, row_index=c[5])
                want = grouped_exact(*c)
                written = ~torch.isnan(want[:, 0])
                assert (got[~written] == 7).all()
                near(got[written], want[written])


@pytest.mark.parametrize("layout,tile", [("tn", t) for t in TILES_TN + ["skinny"]] + [("nn", t) for t in TILES_NN])
@pytest.mark.parametrize("tag,dtype", [("i8f", torch.float32), ("i8h", torch.float16), ("i8b", torch.bfloat16)])
def test_every_kernel_stores_at_any_alignment(monkeypatch, layout, tile, tag, dtype):
    """Rows of results at every offset of a 16-byte grid, of odd and even
    pitches; what lies before and behind them stays."""
    if tile != "skinny":
        monkeypatch.setenv("DGEMM_CONFIG", f"{tag}_{layout}_{tile}")
    M, N = (300, 17) if tile == "skinny" else (303, 290)
    a, b, sa, sb = operands(layout, M, N, 272, 9)
    want = exact(a, b, sa, sb)
    rows, n = (N, M) if layout == "tn" else (M, N)
    for off in range(16 // dtype.itemsize + 1):
        for extra in (9, 10, 16):
            print(f"{tag} {layout} {tile} offset {off} pitch {n + extra}", flush=True)
            wide = torch.full((rows, n + extra), 7.0, device="cuda").to(dtype)
            part = wide[:, off:off + n]
            near(lib().matmul(a, b, scale_a=sa, scale_b=sb, out=part.t() if layout == "tn" else part), want)
            assert (wide[:, :off] == 7).all() and (wide[:, off + n:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("kernel", ["256x256_pp", "128x128_w4", "128x128_w4_s4", "128x64_w4_s4", "skinny16", "skinny32", "skinny64"])
def test_grouped_stores_at_any_alignment(monkeypatch, kernel, dtype):
    monkeypatch.setenv("DGEMM_CONFIG", "i8_grouped_" + kernel)
    c = grouped_case([70, 0, 3, 260], 141, 200, 17, False, tail=3, lead=2)
    want = grouped_exact(*c)
    written = ~torch.isnan(want[:, 0])
    for off in range(16 // dtype.itemsize + 1):
        for extra in (9, 10, 16):
            print(f"grouped {kernel} {dtype} offset {off} pitch {141 + extra}", flush=True)
            wide = torch.full((c[6], 141 + extra), 7.0, device="cuda").to(dtype)
            got = lib().matmul_grouped(*c[:5], out=wide[:, off:off + 141])
            near(got[written], want[written])
            assert (got[~written] == 7).all() and (wide[:, :off] == 7).all() and (wide[:, off + 141:] == 7).all()


def test_grouped_indexes_without_a_row():
    """Indexes outside a count as zeros with the factor 0; the same row many
    times; an a with no rows."""
    a, b, off, sa, sb, idx, rows = grouped_case([20, 0, 45], 130, 144, 3, True)
    idx[::3] = -1
    idx[1] = a.shape[0]
    idx[2] = 2 ** 31 - 1
    idx[4] = -2 ** 31
    idx[5:15] = 6
    got = lib().matmul_grouped(a, b, off, sa, sb, row_index=idx)
    near(got, grouped_exact(a, b, off, sa, sb, idx, rows))
    assert (got[(idx < 0) | (idx >= a.shape[0])] == 0).all()
    got = lib().matmul_grouped(a[:0], b, off, sa[:0], sb, row_index=idx)
    assert (got == 0).all()


def test_grouped_one_factor_and_shared_weights():
    a, b, off, sa, sb, idx, rows = grouped_case([30, 70, 1], 90, 160, 4, False)
    one = torch.tensor([0.125], device="cuda")
    L = lib()
    near(L.matmul_grouped(a, b, off, one, one), grouped_exact(a, b, off, one, one, None, rows))
    near(L.matmul_grouped(a, b, off, sa, one), grouped_exact(a, b, off, sa, one, None, rows))
    same = b[:1].expand(3, 90, 160)
    near(L.matmul_grouped(a, same, off, one, sb), grouped_exact(a, same, off, one, sb, None, rows))


def test_grouped_offsets_beyond_the_rows_are_clamped():
    a, b, off, sa, sb, idx, rows = grouped_case([30, 40], 64, 128, 6, False)
    bad = torch.tensor([-5, 30, 10 ** 9], dtype=torch.int32, device="cuda")
    near(lib().matmul_grouped(a, b, bad, sa, sb), grouped_exact(a, b, off, sa, sb, idx, rows))


def test_grouped_far_weights():
    """Weights whose last group begins past 2^31 bytes."""
    G, N, K = 3, 256, 256
    base = torch.zeros((2 * 2 ** 30 + 2 ** 27,), dtype=torch.int8, device="cuda")
    step = (2 ** 30 + 2 ** 25)
    b = torch.as_strided(base, (G, N, K), (step, K, 1))
    g = gen(8)
    b.copy_(torch.randint(-128, 128, (G, N, K), generator=g, device="cuda", dtype=torch.int8))
    a, sa, sb = ints(g, (90, K)), factors(g, 90), factors(g, G * N).reshape(G, N)
    off = torch.tensor([0, 20, 21, 90], dtype=torch.int32, device="cuda")
    near(lib().matmul_grouped(a, b, off, sa, sb), grouped_exact(a, b, off, sa, sb, None, 90))


# ---- streams and graphs -----------------------------------------------------------

def test_on_a_side_stream_and_captured():
    L = lib()
    g = gen(31)
    x = torch.randn((33, 512), generator=g, device="cuda", dtype=torch.float32).bfloat16()
    w, sw = ints(g, (300, 512)), factors(g, 300)

    def layer(stream=None):
        q, s = L.quantize_i8(x, stream=stream)
        return L.matmul(w, q.t(), scale_a=sw, scale_b=s, out_dtype=torch.bfloat16, stream=stream)

    want = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer()
    by_name = layer(stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(by_name, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    for seed in range(3):
        x.copy_(torch.randn((33, 512), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, layer())


def test_stream_arguments():
    """A stream by object, by raw handle and the null stream's handle."""
    L = lib()
    x = torch.randn((20, 300), generator=gen(1), device="cuda")
    q, s = L.quantize_i8(x)
    w, sw = ints(gen(2), (50, 300)), factors(gen(3), 50)
    want = L.matmul(w, q.t(), scale_a=sw, scale_b=s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        q2, s2 = L.quantize_i8(x=x, stream=stream)
        y = L.matmul(w, q2.t(), scale_a=sw, scale_b=s2, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(q2, q) and torch.equal(s2, s) and torch.equal(y, want)


@pytest.mark.parametrize("layout", ["tn", "nn"])
def test_gemm_i8_on_storage(layout):
    """The tensor-level call with pitches of its own, and what it refuses."""
    L = lib()
    M, N, K, ld = 40, 50, 70, 96
    g = gen(4)
    A = torch.randint(-128, 128, (M, ld), generator=g, device="cuda", dtype=torch.int8)
    B = torch.randint(-128, 128, (N if layout == "tn" else K, ld), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = factors(g, M), factors(g, N)
    b = B[:, :K].t() if layout == "tn" else B[:, :N]
    for dtype in TYPES:
        C = torch.zeros((N if layout == "tn" else M, 64), device="cuda").to(dtype)
        L.gemm_i8(layout, M, N, K, A, ld, B, ld, C, 64, sa, sb)
        got = C[:, :M].t() if layout == "tn" else C[:, :N]
        near(got, exact(A[:, :K], b, sa, sb))
    with pytest.raises(ValueError):
        L.gemm_i8(layout, M + 1, N, K, A, ld, B, ld, C, 64, torch.ones(1, device="cuda"), sb)
    with pytest.raises(ValueError):
        L.gemm_i8(layout, M, N, K, A, ld, B, ld, C[:-1].clone(), 64, sa, sb)
    with pytest.raises(ValueError):
        L.gemm_i8(layout, M, N, K, A, ld, B, ld, C, 64, sa[:5], sb)
    with pytest.raises(TypeError):
        L.gemm_i8(layout, M, N, K, A, ld, B, ld, C.to(torch.int32), 64, sa, sb)
    with pytest.raises(L.DgemmError):
        L.gemm_i8(layout, M, N, K, A, ld - 8, B, ld, C, 64, sa, sb)


def test_python_refusals():
    L = lib()
    g = gen(6)
    q, s = ints(g, (40, 64)), factors(g, 40)
    w, sw = ints(g, (50, 64)), factors(g, 50)
    one = torch.ones(1, device="cuda")
    x = torch.randn((4, 8), device="cuda")
    off = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    wide = torch.empty((50, 40), device="cuda").t()
    value = [
        lambda: L.matmul(q, w.t()), lambda: L.matmul(q, w.t(), scale_a=s),
        lambda: L.matmul(q, w, scale_a=s, scale_b=sw), lambda: L.matmul(q, w.t(), scale_a=s[:7], scale_b=sw),
        lambda: L.matmul(q, w.t(), scale_a=s, scale_b=sw, out=wide[:, :49]),
        lambda: L.matmul(q, w.t(), scale_a=s, scale_b=sw, out=wide, out_dtype=torch.float16),
        lambda: L.matmul(q[:, ::2], w[:, ::2].t(), scale_a=s, scale_b=sw),
        lambda: L.quantize_i8(x[0]), lambda: L.quantize_i8(x.t()), lambda: L.quantize_i8(x, out=q),
        lambda: L.quantize_i8(x, scale=s), lambda: L.matmul_grouped(q, w, off, s, sw),
        lambda: L.matmul_grouped(q, w[None, :, :32], off, s, sw), lambda: L.matmul_grouped(q, w[None], off, s[:3], sw),
        lambda: L.matmul_grouped(q, w[None], off, s, sw[:3]),
        lambda: L.matmul_grouped(q, w[None], off, s, sw, out=torch.empty((39, 50), device="cuda")),
    ]
    kind = [
        lambda: L.matmul(q, x.t(), scale_a=s, scale_b=sw), lambda: L.matmul(q, w.t(), scale_a=s.double(), scale_b=sw),
        lambda: L.matmul(q, w.t(), scale_a=s, scale_b=sw, out_dtype=torch.int32),
        lambda: L.quantize_i8(x.double()), lambda: L.quantize_i8(q),
        lambda: L.matmul_grouped(x, w[None], off, s, sw), lambda: L.matmul_grouped(q, w[None], off.long(), s, sw),
        lambda: L.matmul_grouped(q, w[None], off[:1], s, sw),
        lambda: L.matmul_grouped(q, w[None], off, s, sw, row_index=off.long()),
        lambda: L.matmul(x, x.t(), out_dtype=torch.float16),
    ]
    for calls, error in ((value, ValueError), (kind, TypeError)):
        for i, c in enumerate(calls):
            with pytest.raises(error):
                c()
                print("not refused:", error, i)
    odd = torch.zeros((4, 20), dtype=torch.int8, device="cuda")      # a pitch of 20 bytes
    with pytest.raises(L.DgemmError) as e:
        L.matmul(odd, odd.t(), scale_a=one, scale_b=one)
    assert e.value.status == 5
    with pytest.raises(ValueError):                                  # a row's last 16 bytes have to be there
        L.matmul(odd[:1, :5].clone(), odd[:1, :5].clone().t(), scale_a=one, scale_b=one)
