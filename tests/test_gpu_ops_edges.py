"""GPU tests of the int8 and expert operators at the ends of what their
documentation allows: operands that may be null, the longest pitches, row
counts past one launch, matrices large enough to go past the caches."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def lib():
    import dense_gemm_02_amd as L
    return L


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("dtype", [0, 1, 2], ids=["f32", "f16", "bf16"])
def test_combine_grad_without_sorted_rows(dtype):
    """No sorted rows: dO and Y may be null, and dW is zeros (short rows, one
    wave a token, and long ones)."""
    grad = lib().load_library().expert_combine_grad
    T, k = 9, 3
    slot = torch.arange(T * k, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for H in (0, 7, 64, 5000):
        print(f"combine_grad rows=0 H={H} type {dtype}", flush=True)
        dw = torch.full((T * k + 1,), 7.0, device="cuda")
        assert grad(T, k, H, dtype, None, H, None, 0, H, slot.data_ptr(), None, None, H, dw.data_ptr(), stream) == 0
        assert (dw[:-1] == 0).all() and dw[-1] == 7


@pytest.mark.parametrize("K,ldb", [(1, 2 ** 31 - 64), (2, 2 ** 30 - 32), (3, 2 ** 29), (5, 2 ** 28 + 2 ** 27),
                                   (7, 2 ** 28 + 2 ** 25)])
@pytest.mark.parametrize("tile", [None, "256x256_w4", "256x128_w4", "256x192_w4"])
def test_row_major_b_of_the_longest_pitch(monkeypatch, tile, K, ldb):
    """K * ldb at its limit with a few rows of B: what A holds behind K (other
    values here) meets nothing, whichever kernel runs.  Rows of B are of the
    values' full range on both sides of the N columns that count."""
    import ctypes
    L = lib()
    M, N = (4096, 4096) if tile is None else (300, 333)
    if tile is not None:
        monkeypatch.setenv("DGEMM_CONFIG", f"i8f_nn_{tile}")
    buf = ctypes.create_string_buffer(256)
    assert L.load_library().dgemm_kernel_config(6, 0, M, N, K, buf, 256) == 0
    assert buf.value.decode().startswith("i8f_nn_" + (tile or "256x256_w4")), buf.value
    print(f"K={K} ldb={ldb} {buf.value.decode()}", flush=True)
    g = gen(K)
    A = torch.randint(-128, 128, (M, 16), generator=g, device="cuda", dtype=torch.int8)
    B = torch.full((K, ldb), 77, device="cuda", dtype=torch.int8)
    B[:, :N] = torch.randint(-128, 128, (K, N), generator=g, device="cuda", dtype=torch.int8)
    C = torch.empty((M, N), device="cuda")
    one = torch.ones(1, device="cuda")
    L.gemm_i8("nn", M, N, K, A, 16, B, ldb, C, N, one, one)
    # sums of at most 7 * 2^14: exact in FP32
    assert torch.equal(C.double(), A[:, :K].double() @ B[:, :N].double())
