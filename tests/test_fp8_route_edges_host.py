"""Host-only checks of the ends of what the block-scaled FP8 and router entry
points document.  No kernel is launched here."""

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
