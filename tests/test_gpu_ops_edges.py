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
