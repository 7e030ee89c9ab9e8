"""Argument checks of the residual and gated GEMMs (C ABI and binding), without a GPU."""
import ctypes

import pytest
import torch

from fp8_mixed_precision_mxq_b200 import _lib, ops

V = ctypes.c_void_p
A16, A8, WS = 4096, 4096 + 8, 1 << 20


def epi(act=0, dt=1, residual=A16, gate=A16, rpg=128):
    return _lib.Epilogue(act, dt, residual, gate, rpg)


BAD_EPILOGUES = [
    (None, _lib.ERR_INVALID_ARG),
    (epi(act=4), _lib.ERR_INVALID_ARG),
    (epi(act=-1), _lib.ERR_INVALID_ARG),
    (epi(dt=2), _lib.ERR_INVALID_ARG),
    (epi(rpg=0), _lib.ERR_INVALID_ARG),
    (epi(residual=A8), _lib.ERR_ALIGN),
    (epi(gate=A8), _lib.ERR_ALIGN),
]


@pytest.mark.parametrize("e,status", BAD_EPILOGUES)
def test_epilogue_is_checked(e, status):
    L = _lib.lib()
    assert L.mxq_gemm_residual(A16, A16, 0, 128, 256, A16, A16, 256, None, e, A16, None) == status
    assert L.mxq_gemm_bf16_residual(A16, 128, 256, A16, 256, None, e, A16, None) == status
    assert L.mxq_linear_residual(A16, 128, 256, A16, A16, 256, None, 0, e, WS, 1 << 30, A16, None) == status
    w = _lib.WDesc(4096, 4096, None, 256, 256)
    assert L.mxq_gated_ffn(A16, 128, 256, w, w, w, 3, 0, 0, e, WS, 1 << 30, A16, None) == status
    assert _lib.last_error()


def test_residual_gemms_check_their_operands():
    L, e = _lib.lib(), epi()
    bad = [
        ((A16, A16, 0, 128, 256, A16, A16, 250, None, e, A16, None), _lib.ERR_SHAPE),    # N % 8
        ((A16, A16, 1, 128, 96, A16, A16, 256, None, e, A16, None), _lib.ERR_SHAPE),     # W4A8 K % 128
        ((A16, A16, 1, 128, 256, 4096 + 16, A16, 256, None, e, A16, None), _lib.ERR_ALIGN),
        ((A16, A16, 2, 128, 256, A16, A16, 256, None, e, A16, None), _lib.ERR_INVALID_ARG),
        ((A16, A16, 0, 0, 256, A16, A16, 256, None, e, A16, None), _lib.ERR_INVALID_ARG),
        ((A16, A16, 0, 128, 256, A16, A16, 256, None, e, None, None), _lib.ERR_INVALID_ARG),
    ]
    for args, status in bad:
        assert L.mxq_gemm_residual(*args) == status, (args, _lib.last_error())
    assert L.mxq_gemm_bf16_residual(A16, 128, 250, A16, 256, None, e, A16, None) == _lib.ERR_SHAPE
    assert L.mxq_gemm_bf16_residual(A16, 0, 256, A16, 256, None, e, A16, None) == _lib.ERR_INVALID_ARG
    need = L.mxq_workspace_bytes(128, 256, 256, 0, 0)
    assert L.mxq_linear_residual(A16, 128, 256, A16, A16, 256, None, 0, e, WS, need - 1, A16,
                                 None) == _lib.ERR_WORKSPACE
    assert L.mxq_linear_residual(A16, 128, 256, A16, A16, 256, None, 0, e, WS + 16, need, A16,
                                 None) == _lib.ERR_ALIGN


@pytest.mark.parametrize("M", [1, 16, 128])
def test_linear_residual_refuses_an_output_over_its_input(M):
    """Some of the few-row kernel's CTAs still read x while others write y, so no y may overlap it,
    not even the x that is its own residual."""
    L, e = _lib.lib(), epi()
    far = 1 << 24
    for x, y in ((far, far), (far, far + M * 256 * 2 - 16), (far, far - M * 512 * 2 + 16)):
        got = L.mxq_linear_residual(x, M, 256, A16, A16, 512, None, 0, e, WS, 1 << 30, y, None)
        assert got == _lib.ERR_INVALID_ARG and "overlaps" in _lib.last_error(), (x, y, _lib.last_error())


def test_gated_gemms_check_their_operands():
    L = _lib.lib()
    w = _lib.WDesc(4096, 4096, None, 256, 512)
    other = _lib.WDesc(4096, 4096, None, 288, 512)
    odd = _lib.WDesc(4096, 4096, None, 264, 512)
    ragged = _lib.WDesc(4096, 4096, None, 260, 512)
    lost = _lib.WDesc(None, 4096, None, 256, 512)
    bad = [
        ((A16, A16, 0, 128, 512, w, other, 3, -1, A16, None, None), _lib.ERR_SHAPE),      # widths differ
        ((A16, A16, 0, 128, 256, w, w, 3, -1, A16, None, None), _lib.ERR_SHAPE),          # K differs
        ((A16, A16, 0, 128, 512, odd, odd, 3, 0, A16, A16, None), _lib.ERR_SHAPE),        # H % 32 with codes
        ((A16, A16, 0, 128, 512, ragged, ragged, 3, -1, A16, None, None), _lib.ERR_SHAPE),  # H % 8
        ((A16, A16, 0, 128, 512, w, w, 4, -1, A16, None, None), _lib.ERR_INVALID_ARG),    # act
        ((A16, A16, 0, 128, 512, w, w, 3, 2, A16, A16, None), _lib.ERR_INVALID_ARG),      # out_fmt
        ((A16, A16, 0, 128, 512, w, w, 3, -1, A16, A16, None), _lib.ERR_INVALID_ARG),     # scales with bf16
        ((A16, A16, 0, 128, 512, w, w, 3, 1, A16, None, None), _lib.ERR_INVALID_ARG),
        ((A16, A16, 0, 128, 512, w, lost, 3, -1, A16, None, None), _lib.ERR_INVALID_ARG),
        ((A16, A16, 0, 128, 512, None, w, 3, -1, A16, None, None), _lib.ERR_INVALID_ARG),
        ((A16, A16, 0, 128, 512, w, w, 3, -1, A8, None, None), _lib.ERR_ALIGN),
    ]
    for args, status in bad:
        assert L.mxq_gemm_gated(*args) == status, (args, _lib.last_error())
    assert L.mxq_gemm_bf16_gated(A16, 128, 250, A16, None, A16, None, 256, 3, -1, A16, None, None) == _lib.ERR_SHAPE
    assert L.mxq_gemm_bf16_gated(A16, 128, 256, A16, None, None, None, 256, 3, -1, A16, None,
                                 None) == _lib.ERR_INVALID_ARG
    assert L.mxq_gemm_bf16_gated(A16, 128, 256, A16, A8, A16, None, 256, 3, -1, A16, None, None) == _lib.ERR_ALIGN


def test_gated_ffn_checks_its_weights_and_workspace():
    L = _lib.lib()
    up, down = _lib.WDesc(4096, 4096, None, 288, 256), _lib.WDesc(4096, 4096, None, 256, 288)
    wrong = _lib.WDesc(4096, 4096, None, 256, 320)
    none = epi(residual=None, gate=None, rpg=1)
    need = L.mxq_ffn_workspace_bytes(128, 256, 288, 0, 0)

    def call(gate=up, up_=up, dn=down, act=3, uf=0, df=0, e=none, ws=WS, n=need):
        return L.mxq_gated_ffn(A16, 128, 256, gate, up_, dn, act, uf, df, e, ws, n, A16, None)

    assert call(dn=wrong) == _lib.ERR_SHAPE
    assert call(dn=None) == _lib.ERR_INVALID_ARG
    assert call(up_=None) == _lib.ERR_INVALID_ARG
    assert call(df=1, n=1 << 30) == _lib.ERR_SHAPE  # the E4M3 hidden width is not a multiple of 128
    assert call(df=-1) == _lib.ERR_INVALID_ARG
    assert call(act=7) == _lib.ERR_INVALID_ARG
    assert call(e=epi(act=1, residual=None, gate=None, rpg=1)) == _lib.ERR_INVALID_ARG
    assert call(n=need - 1) == _lib.ERR_WORKSPACE
    assert call(ws=None) == _lib.ERR_INVALID_ARG


def test_bindings_reject_host_tensors_and_unknown_names():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = ops.QWeight(x, x, 64, 64)
    with pytest.raises(ValueError):
        ops.linear_residual(x, w)
    with pytest.raises(ValueError):
        ops.gemm_bf16_residual(x, x)
    with pytest.raises(ValueError):
        ops.gated_ffn(x, w, w, w)
    with pytest.raises(ValueError):
        ops._act("relu")
