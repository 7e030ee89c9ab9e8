"""Argument checks of the fused norms (C ABI and binding), without a GPU."""
import ctypes

import pytest
import torch

from fp8_mixed_precision_mxq_b200 import _lib, ops

A16, A8 = 4096, 4096 + 8


def desc(**kw):
    d = dict(x=A16, y=A16, rows=4, K=64, x_dtype=0, vec_dtype=1, norm=1, post_norm=0, weight=None, bias=None,
             post_weight=None, post_bias=None, gate=None, scale=None, shift=None, rows_per_group=4, eps=1e-6)
    d.update(kw)
    return _lib.NormDesc(**d)


BAD = [  # descriptor changes, z, out_fmt, out, sf, status
    (dict(x=None), A16, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(rows=0), A16, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(K=-8), A16, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(K=60), A16, -1, A16, None, _lib.ERR_SHAPE),              # K % 8
    (dict(K=40), A16, 0, A16, A16, _lib.ERR_SHAPE),                # K % 32 with codes
    (dict(K=32768 + 32), A16, -1, A16, None, _lib.ERR_SHAPE),      # longest row
    (dict(rows=2 ** 31), A16, -1, A16, None, _lib.ERR_SHAPE),
    (dict(rows=2 ** 20, K=32768), A16, -1, A16, None, _lib.ERR_SHAPE),
    (dict(x_dtype=2), A16, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(vec_dtype=-1), A16, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(norm=0), A16, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(norm=3), A16, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(post_norm=3), A16, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(eps=-1e-6), A16, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(eps=float("nan")), A16, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(eps=float("inf")), A16, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(rows_per_group=0), A16, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(y=None), A16, -1, A16, None, _lib.ERR_INVALID_ARG),      # z without y
    (dict(y=None, gate=A16), None, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(y=None, post_norm=2), None, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(post_weight=A16), A16, -1, A16, None, _lib.ERR_INVALID_ARG),
    (dict(), None, -1, A16, None, _lib.ERR_INVALID_ARG),           # y without z
    (dict(), A16, -1, None, None, _lib.ERR_INVALID_ARG),
    (dict(), A16, -1, A16, A16, _lib.ERR_INVALID_ARG),             # scales with a bf16 output
    (dict(), A16, 0, A16, None, _lib.ERR_INVALID_ARG),
    (dict(), A16, 2, A16, A16, _lib.ERR_INVALID_ARG),              # unknown format
    (dict(y=A8), A16, -1, A16, None, _lib.ERR_ALIGN),
    (dict(scale=A8), A16, -1, A16, None, _lib.ERR_ALIGN),
    (dict(), A16, 1, A8, A16, _lib.ERR_ALIGN),
]


@pytest.mark.parametrize("change,z,fmt,out,sf,status", BAD)
def test_norm_residual_rejects_bad_arguments(change, z, fmt, out, sf, status):
    L = _lib.lib()
    assert L.mxq_norm_residual(ctypes.byref(desc(**change)), z, fmt, out, sf, None) == status, _lib.last_error()
    assert _lib.last_error()


def test_norm_residual_needs_a_descriptor():
    assert _lib.lib().mxq_norm_residual(None, A16, -1, A16, None, None) == _lib.ERR_INVALID_ARG


def test_binding_rejects_host_tensors():
    with pytest.raises(ValueError):
        ops.norm_residual(torch.zeros(4, 64, dtype=torch.bfloat16))
