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


# ---- the kernels that the GPU tests force by name -----------------------------------

@pytest.mark.parametrize("tag,code", [("i8f", 6), ("i8h", 7), ("i8b", 8)])
def test_forced_dense_kernels_are_the_named_ones(lib, monkeypatch, tag, code):  # noqa: F811
    """A name that no kernel bears would leave the choice as it was."""
    from test_gpu_quantized import TILES_NN, TILES_TN
    for layout, tiles in ((1, TILES_TN), (0, TILES_NN)):
        for tile in tiles:
            want = f"{tag}_{'tn' if layout else 'nn'}_{tile}"
            monkeypatch.setenv("DGEMM_CONFIG", want)
            for M, N in ((300, 333), (303, 290)):
                for K in (1, 16, 100, 128, 129, 200, 256, 257, 272, 384, 399, 512, 600, 639):
                    st, _, name = config(lib, code, layout, M, N, K)
                    assert st == OK and name == want, (name, want, K)


def grouped_config(lib, c_type, gather, groups, rows, N, K):  # noqa: F811
    buf = ctypes.create_string_buffer(256)
    st = lib.dgemm_grouped_config(c_type, gather, groups, rows, N, K, buf, 256)
    words = buf.value.decode().split()
    return st, dict(x.split("=") for x in words[1:] if "=" in x), words[0] if words else ""


GROUPED = ["256x256_pp", "128x128_w4", "128x128_w4_s4", "128x64_w4_s4", "skinny16", "skinny32", "skinny64"]


@pytest.mark.parametrize("kernel", GROUPED)
def test_forced_grouped_kernels_are_the_named_ones(lib, monkeypatch, kernel):  # noqa: F811
    import test_gpu_quantized as T
    for test in (T.test_grouped_every_kernel, T.test_grouped_stores_at_any_alignment):
        marks = [m for m in test.pytestmark if m.name == "parametrize" and m.args[0] == "kernel"]
        assert marks and list(marks[0].args[1]) == GROUPED
    monkeypatch.setenv("DGEMM_CONFIG", "i8_grouped_" + kernel)
    for c_type in (0, 1, 2):
        for gather in (0, 1):
            for groups, rows, N in ((7, 87, 70), (6, 550, 300), (3, 306, 513), (70, 215, 40), (4, 338, 141)):
                for K in (1, 100, 128, 200, 256, 399, 1040):
                    st, _, name = grouped_config(lib, c_type, gather, groups, rows, N, K)
                    assert st == OK and name == "i8_grouped_" + kernel, (name, K)


def test_every_grouped_kernel_is_chosen_somewhere(lib):  # noqa: F811
    seen = {grouped_config(lib, 2, 1, g, r, N, K)[2]
            for g in (1, 2, 8, 64, 256) for r in (8, 64, 256, 512, 1024, 2048, 8192, 32768)
            for N in (256, 1024, 2048, 4096, 14336) for K in (64, 256, 1024, 4096, 14336)}
    assert seen == {"i8_grouped_" + k for k in GROUPED}


def test_grouped_config_refusals(lib):  # noqa: F811
    assert grouped_config(lib, 3, 0, 4, 10, 20, 30)[0] == 8 and grouped_config(lib, -1, 0, 4, 10, 20, 30)[0] == 8
    for bad in ((-1, 10, 20, 30), (4, -1, 20, 30), (4, 10, -1, 30), (4, 10, 20, -1)):
        assert grouped_config(lib, 0, 0, *bad)[0] == 1
    for bad in ((2 ** 31, 1, 1, 1), (1, 1, 2 ** 31, 1), (2 ** 16, 1, 2 ** 16, 1), (1, 2 ** 29, 1, 1), (1, 1, 2 ** 29, 1),
                (1, 1, 1, 131072), (2 ** 17, 2 ** 17, 8192, 32)):
        assert grouped_config(lib, 0, 0, *bad)[0] == UNSUP
    for none in ((0, 10, 20, 30), (4, 0, 20, 30), (4, 10, 0, 30)):
        st, _, name = grouped_config(lib, 0, 1, *none)
        assert st == OK and name == "none"
    assert lib.dgemm_grouped_config(0, 0, 4, 10, 20, 30, None, 0) == OK
    short = ctypes.create_string_buffer(b"x" * 16)
    assert lib.dgemm_grouped_config(0, 0, 4, 10, 20, 30, short, 8) == OK and short.raw[7:9] == b"\0x"


def test_grouped_launches_stay_below_the_limit(lib):  # noqa: F811
    """What the header promises of the sizes that fit, and no grid past them."""
    for g in (1, 3, 64, 1000, 2 ** 17, 2 ** 20):
        for rows in (1, 100, 2 ** 14, 2 ** 20, 2 ** 26 + 1, 2 ** 29 - 16):
            for N in (1, 32, 33, 1000, 2047):
                if g * N > 2 ** 31 - 1:
                    continue
                for K in (1, 1000, 100000):
                    st, c, _ = grouped_config(lib, 2, 0, g, rows, N, K)
                    if -(-N // 32) * 32 * (rows + 15 * g) < 2 ** 32:
                        assert st == OK
                    assert st == UNSUP or int(c["grid"]) * int(c["threads"]) < 2 ** 32


def test_grouped_groups_past_the_search_are_refused(lib):  # noqa: F811
    """The search over the groups counts them in 32 bits, 64 at a time: with
    2^31 - 1 of them it would never end."""
    for n in (2 ** 20 + 1, 2 ** 31 - 64, 2 ** 31 - 63, 2 ** 31 - 1):
        assert grouped(lib, G=n, N=1, ldc=1, nb=1, gb=0, rows=1, ra=1, na=1) == UNSUP
        assert grouped(lib, G=n, N=1, ldc=1, nb=1, gb=0, rows=0) == UNSUP      # before the calls without work
        assert grouped_config(lib, 0, 0, n, 1, 1, 32)[0] == UNSUP
    assert grouped_config(lib, 0, 0, 2 ** 20, 1, 1, 32)[0] == OK
