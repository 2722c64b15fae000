"""Host-only checks of the ends of what the block-scaled FP8 and router entry
points document.  No kernel is launched here."""

import ctypes
import os

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from dense_gemm_02_amd import binding
    if not os.path.exists(binding.library_path()):
        from dense_gemm_02_amd import build
        build.build()
    return binding.load_library()


FAKE = 1 << 20            # aligned fake device address; never dereferenced here
OK, DIM, NULL, LD, LAYOUT, ALIGN, UNSUP, TYPE = 0, 1, 2, 3, 4, 5, 6, 8


def quantize(lib, rows=4, K=300, block_rows=1, sr=1, sk=4, X=FAKE + 1):
    """(X is misaligned: a call that passes the checks of strides is refused for that.)"""
    return lib.quantize_fp8(rows, K, X, K, 2, 0, block_rows, FAKE, K, FAKE, sr, sk, None)


def test_quantize_refuses_overlapping_scales(lib):
    for sr, sk in ((1, 4), (1, 100), (3, 1), (5, 1), (2, 8), (7, 2), (1 << 62, 1), (1, 1 << 62)):
        assert quantize(lib, sr=sr, sk=sk) == ALIGN, (sr, sk)
    for sr, sk in ((0, 0), (0, 1), (1, 0), (1, 1), (1, 3), (2, 1), (2, 6), (4, 2), (0, 1 << 62), (1 << 62, 0)):
        assert quantize(lib, sr=sr, sk=sk) == LD, (sr, sk)
    # One factor along an axis: its stride says nothing.
    assert quantize(lib, rows=1, sr=0, sk=1) == ALIGN and quantize(lib, rows=1, sr=0, sk=0) == LD
    assert quantize(lib, K=100, sr=1, sk=0) == ALIGN and quantize(lib, K=100, sr=0, sk=0) == LD
    assert quantize(lib, rows=1, K=1, sr=0, sk=0) == ALIGN
    assert quantize(lib, rows=128, block_rows=128, sr=0, sk=1) == ALIGN
    assert quantize(lib, rows=129, block_rows=128, sr=0, sk=1) == LD
    assert quantize(lib, rows=2 ** 63 - 1, block_rows=128, sr=1, sk=2 ** 62) == ALIGN


def test_row_counts_near_the_end_of_64_bits(lib):
    big = 2 ** 63 - 1
    for rows_a, rows_b in ((1, 1), (128, 1), (1, 128), (128, 128)):
        for M, N in ((big, 1), (1, big), (big, big)):
            assert lib.gemm_fp8_block(M, N, 128, FAKE, 128, FAKE, 128, FAKE, big, 2, FAKE, rows_a, 1, 1, FAKE, rows_b, 1,
                                      1, 1, None) == UNSUP
    assert lib.gemm_fp8_grouped(1, 1, 2 ** 31 - 1, 128, FAKE, 1, 128, None, FAKE, 128, 0, FAKE, 2 ** 31, 2, FAKE, 1, 1,
                                FAKE, 1, 1, 1, FAKE, None) == UNSUP


def test_every_kernel_of_few_rows_can_be_named(lib, monkeypatch):
    """DGEMM_CONFIG takes the strips with their rows, few rows and stages of copies: kernels that sizes choose rarely can
    be tested."""
    buf = ctypes.create_string_buffer(256)
    for tag, c in (("f32", 0), ("f16", 1), ("bf16", 2)):
        for order in "ab":
            for rows, few, stages in ((16, 16, 1), (16, 16, 2), (16, 32, 1), (16, 32, 2), (32, 16, 1), (32, 16, 2),
                                      (32, 32, 1), (32, 32, 2), (32, 64, 1)):
                monkeypatch.setenv("DGEMM_CONFIG", f"b8{tag}_tn_skinny_{order}:{rows}x{few}x{stages}")
                assert lib.dgemm_fp8_block_config(c, 1, 128, 1, 700, 700, 4111, buf, 256) == 0
                tile = f"{few}x{rows}" if order == "a" else f"{rows}x{few}"
                lds = max(8 * stages * ((rows + few) * 128 + 512), 4 * 8 * rows * few)
                assert buf.value.decode().startswith(f"b8{tag}_tn_skinny_{order} tile={tile} threads=512 lds={lds} ")
    for none in ("b8bf16_tn_skinny_a:16x64x1", "b8bf16_tn_skinny_a:32x64x2", "b8bf16_tn_skinny_b:16x16x3"):
        monkeypatch.setenv("DGEMM_CONFIG", none)
        assert lib.dgemm_fp8_block_config(2, 1, 128, 1, 8192, 8192, 8192, buf, 256) == 0
        assert buf.value.decode().startswith("b8bf16_tn_256x256_pp ")


def test_factors_of_128_rows_on_both_sides_are_not_taken_for_vectors():
    """With as many blocks of k as rows and columns, the factors of blocks on both sides hold M and N values."""
    from dense_gemm_02_amd.binding import _block_factors
    for M, N, K in ((64, 64, 8192), (16, 16, 2048), (16, 16, 2047), (2, 2, 129), (16384, 16384, 16384), (16384, 128, 16384)):
        a, b = (torch.empty((1,), dtype=torch.float8_e4m3fn).expand(shape) for shape in ((M, K), (K, N)))
        blocks = -(-K // 128)
        sa, sb = torch.ones((-(-M // 128), blocks)), torch.ones((blocks, -(-N // 128)))
        assert sa.numel() == M and sb.numel() == N
        for dtype in (None, torch.float32, torch.bfloat16):
            assert _block_factors(a, b, sa, sb, dtype)
        # Vectors in two dimensions are vectors.
        assert not _block_factors(a, b, torch.ones((M, 1)), torch.ones((1, N)), None)
        assert not _block_factors(a, b, torch.ones((1, 1)), torch.ones((1, 1)), None)
