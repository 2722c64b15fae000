"""Host-only checks of the int8 and expert operators at the ends of what their
documentation allows: sizes that fit no launch, and arguments of the Python
functions.  No kernel is launched here."""

import ctypes

import pytest
import torch

from test_ops_host import FAKE, OK, UNSUP, grouped, lib  # noqa: F401


def config(lib, dtype, layout, M, N, K):
    buf = ctypes.create_string_buffer(256)
    st = lib.dgemm_kernel_config(dtype, layout, M, N, K, buf, 256)
    return st, dict(x.split("=") for x in buf.value.decode().split()[1:] if "=" in x), buf.value.decode().split(" ")[0]


# One token against 2^k channels and the other way round, and a few: the
# largest sides whose operands could still be in memory.
@pytest.mark.parametrize("few", [1, 16, 17, 64])
@pytest.mark.parametrize("layout", [0, 1], ids=["nn", "tn"])
@pytest.mark.parametrize("dtype", [1, 2, 6, 7, 8], ids=["f16", "bf16", "i8f", "i8h", "i8b"])
def test_long_sides_fit_a_launch_or_are_refused(lib, dtype, layout, few):  # noqa: F811
    for k in range(20, 33):
        for n in (2 ** k - 1, 2 ** k):
            for M, N in ((few, n), (n, few)):
                # (B row-major has K rows of N within one descriptor.)
                K = 16 if layout == 1 or N == few else max(1, (2 ** 31 - 64) // (-(-N // 16) * 16) // 2)
                st, c, name = config(lib, dtype, layout, M, N, K)
                assert st in (OK, UNSUP)
                items = -(-M // 32) * 32 * (-(-N // 32) * 32)
                if st == OK:
                    assert int(c["grid"]) * int(c["threads"]) < 2 ** 32, (M, N, name)
                elif layout == 1 or N == few:
                    assert items >= 2 ** 32, (M, N, name)


def test_int8_strips_give_way_to_blocks(lib):  # noqa: F811
    """Strips of 32 of 2^28 rows would be 2^32 work-items; tiles of 64 x 128 fit."""
    assert config(lib, 7, 1, 2 ** 27, 1, 16)[2] == "i8_tn_skinny_b"
    assert config(lib, 7, 1, 1, 2 ** 27, 16)[2] == "i8_tn_skinny_a"
    for M, N in ((2 ** 28, 1), (1, 2 ** 28)):
        st, c, name = config(lib, 7, 1, M, N, 16)
        assert st == OK and name.startswith("i8h_tn_"), name


def test_grouped_tiles_past_a_launch_are_refused(lib):  # noqa: F811
    n = 2 ** 17
    assert grouped(lib, G=n, rows=n, N=8192, ra=n, na=1, nb=1, gb=0, ldc=8192) == UNSUP


class Elsewhere:
    """Stands for a tensor, or a stream, of a device this host need not have."""
    is_cuda = True

    def __init__(self, index):
        self.device = torch.device("cuda", index)


class OtherStream:
    device = torch.device("cuda", 1)


def test_stream_finds_the_device_in_any_argument():
    """A stream of another device than the tensors' is refused as such, which
    takes their device: from any position, number or None before it."""
    from dense_gemm_02_amd.quantized import takes_stream
    ran = []
    call = takes_stream(lambda *args, **kw: ran.append((args, kw)))
    t = Elsewhere(0)
    for args, kw in (((t,), {}), ((), {"ids": t}), ((), {"experts": 8, "ids": t}), ((), {"out": None, "x": t}),
                     ((), {"out_dtype": torch.float16, "x": t}), ((8, t), {})):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call(*args, stream=OtherStream(), **kw)
    for args, kw in (((), {}), ((8,), {"out": None}), ((), {"x": torch.zeros(3)})):
        with pytest.raises(TypeError, match="device tensors"):
            call(*args, stream=OtherStream(), **kw)
    assert not ran


class Shaped(Elsewhere):
    def __init__(self, *shape):
        super().__init__(0)
        self.shape = shape

    def dim(self):
        return len(self.shape)


@pytest.mark.parametrize("x,ids,b", [((5, 64), (7, 2), (3, 32, 64)), ((7, 64), (5, 2), (3, 32, 64)),
                                     ((5, 64), (10,), (3, 32, 64)), ((64,), (1, 2), (3, 32, 64)),
                                     ((5, 60), (5, 2), (3, 32, 64)), ((5, 64), (5, 2), (32, 64))])
def test_experts_layer_refuses_what_does_not_match(x, ids, b):
    import dense_gemm_02_amd as L
    with pytest.raises(ValueError, match="one row for each token|do not chain"):
        L.matmul_experts(Shaped(*x), Shaped(*ids), None, Shaped(*b), Shaped(3, 32))
