"""Outputs over inputs that other CTAs still read are refused before any launch, without a GPU:
the activation of a GEMM in place of its output, and a residual that overlaps it without being it."""
import pytest

from fp8_mixed_precision_mxq_b200 import _lib

A16, FAR = 4096, 1 << 24


def epi(residual=None):
    return _lib.Epilogue(0, 1, residual, None, 1)


def refused(status):
    return status == _lib.ERR_INVALID_ARG and "overlaps" in _lib.last_error()


@pytest.mark.parametrize("M", [1, 64, 1000])
def test_bf16_gemm_in_place_of_its_operand(M):
    """y = x + x W^T cannot be written over x, whether or not x is named as the residual."""
    L, K, N = _lib.lib(), 512, 512
    for a, y in ((FAR, FAR), (FAR, FAR + M * K * 2 - 16), (FAR, FAR - M * N * 2 + 16)):
        for r in (None, a, y):
            assert refused(L.mxq_gemm_bf16_residual(a, M, K, A16, N, None, epi(r), y, None)), (a, y, r)
        assert refused(L.mxq_gemm_bf16_gated(a, M, K, A16, None, A16, None, N, 3, -1, y, None, None)), (a, y)
    assert refused(L.mxq_gemm_bf16_gated(FAR, M, K, A16, None, A16, None, N, 3, 1, FAR, 2 * FAR, None))
    assert refused(L.mxq_gemm_bf16_gated(FAR, M, K, A16, None, A16, None, N, 3, 1, 2 * FAR, FAR, None))


@pytest.mark.parametrize("M", [1, 64, 1000])
@pytest.mark.parametrize("fmt", [0, 1])
def test_outputs_over_a_quantized_operand(M, fmt):
    L, K, N = _lib.lib(), 512, 512
    codes, sf = L.mxq_codes_bytes(M, K, fmt), L.mxq_sf_bytes(M, K)
    w = _lib.WDesc(A16, A16, None, N, K)
    for y in (FAR, FAR + codes - 16, FAR - M * N * 2 + 16, 2 * FAR, 2 * FAR + sf - 16, 2 * FAR - 16):
        assert refused(L.mxq_gemm_residual(FAR, 2 * FAR, fmt, M, K, A16, A16, N, None, epi(), y, None)), y
        assert refused(L.mxq_gemm_gated(FAR, 2 * FAR, fmt, M, K, w, w, 3, -1, y, None, None)), y
    # codes and scales of h in the buffers of the operand's
    for of in (0, 1):
        for out, out_sf in ((FAR, 4 * FAR), (4 * FAR, 2 * FAR), (FAR, 2 * FAR), (4 * FAR, FAR), (2 * FAR, 4 * FAR)):
            assert refused(L.mxq_gemm_gated(FAR, 2 * FAR, fmt, M, K, w, w, 3, of, out, out_sf, None)), (out, out_sf)


@pytest.mark.parametrize("M", [2, 64, 1000])
def test_a_residual_that_overlaps_the_output_without_being_it(M):
    L, N = _lib.lib(), 512
    w, d = _lib.WDesc(A16, A16, None, N, 512), _lib.WDesc(A16, A16, None, N, N)
    y = 4 * FAR
    for r in (y + 16, y - 16, y + N * 2, y - N * 2, y + M * N * 2 - 16, y - M * N * 2 + 16):
        e = epi(r)
        assert refused(L.mxq_gemm_residual(FAR, 2 * FAR, 0, M, 512, A16, A16, N, None, e, y, None)), r
        assert refused(L.mxq_gemm_bf16_residual(FAR, M, 512, A16, N, None, e, y, None)), r
        assert refused(L.mxq_linear_residual(FAR, M, 512, A16, A16, N, None, 0, e, 2 * FAR, 1 << 23, y, None)), r
        assert refused(L.mxq_gated_ffn(FAR, M, 512, w, w, d, 3, 0, 0, e, 2 * FAR, 1 << 23, y, None)), r
