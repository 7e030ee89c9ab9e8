"""Tensor-level entry points: the same calls as the C ABI (include/mxq.h), taking torch
tensors for device memory and the current torch stream, or the one given as `stream`.
Nothing here computes: each function checks dtypes and devices, allocates outputs with
torch (on the stream of the call), and calls the library.  As with any work on another
stream, the caller orders a given stream behind whatever wrote the call's tensors, waits
for it before using the result elsewhere, and keeps the tensors it passed until then."""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import FMT_E2M1, FMT_E4M3, MODE_NATIVE, MODE_QDQ, WDesc, check

_FMTS = {"e2m1": FMT_E2M1, "e4m3": FMT_E4M3, FMT_E2M1: FMT_E2M1, FMT_E4M3: FMT_E4M3}
_MODES = {"native": MODE_NATIVE, "qdq": MODE_QDQ, MODE_NATIVE: MODE_NATIVE, MODE_QDQ: MODE_QDQ}


def _fmt(f) -> int:
    return _FMTS[f]


def _mode(m) -> int:
    return _MODES[m]


def _stream(stream=None) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _p(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _empty(shape, dtype, device, stream=None, returned=True) -> torch.Tensor:
    """A new tensor for a call that runs on `stream` (None: the current one).  It comes from that
    stream's memory: a block of the current stream's could still be read by what is queued there
    while the call writes it, or be handed out again there while the call still uses it.  For a
    tensor that is returned the current stream is noted as a user too, since the caller's code
    reads it there after waiting for the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _cuda_bf16(t: torch.Tensor, name: str) -> None:
    if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
        raise ValueError("%s must be a contiguous bf16 CUDA tensor" % name)


def codes_bytes(rows: int, K: int, fmt="e2m1") -> int:
    return int(_lib.lib().mxq_codes_bytes(rows, K, _fmt(fmt)))


def sf_bytes(rows: int, K: int) -> int:
    return int(_lib.lib().mxq_sf_bytes(rows, K))


def workspace_bytes(M: int, N: int, K: int, fmt="e2m1", mode="native") -> int:
    return int(_lib.lib().mxq_workspace_bytes(M, N, K, _fmt(fmt), _mode(mode)))


@dataclass
class QWeight:
    """MXFP4 weight of one linear layer: codes [N, K/2], tiled scales, optional bias."""
    codes: torch.Tensor
    sf: torch.Tensor
    N: int
    K: int
    bias: torch.Tensor | None = None

    def desc(self) -> WDesc:
        return WDesc(self.codes.data_ptr(), self.sf.data_ptr(),
                     0 if self.bias is None else self.bias.data_ptr(), self.N, self.K)


def quantize_act(x: torch.Tensor, fmt="e2m1", codes=None, sf=None, stream=None):
    """x [M, K] bf16 -> (codes, tiled scales) in format fmt."""
    _cuda_bf16(x, "x")
    M, K = x.shape
    f = _fmt(fmt)
    if codes is None:
        codes = _empty(max(1, codes_bytes(M, K, f)), torch.uint8, x.device, stream)
    if sf is None:
        sf = _empty(max(1, sf_bytes(M, K)), torch.uint8, x.device, stream)
    check(_lib.lib().mxq_quantize_act(_p(x), M, K, f, _p(codes), _p(sf), _stream(stream)), "mxq_quantize_act")
    return codes, sf


def quantize_weight(w: torch.Tensor, bias: torch.Tensor | None = None, stream=None) -> QWeight:
    """w [N, K] bf16 -> QWeight (MXFP4 codes [N, K/2] + tiled scales)."""
    _cuda_bf16(w, "w")
    N, K = w.shape
    codes = _empty((N, K // 2), torch.uint8, w.device, stream)
    sf = _empty(max(1, sf_bytes(N, K)), torch.uint8, w.device, stream)
    check(_lib.lib().mxq_quantize_weight(_p(w), N, K, _p(codes), _p(sf), _stream(stream)), "mxq_quantize_weight")
    if bias is not None:
        _cuda_bf16(bias, "bias")
    return QWeight(codes, sf, N, K, bias)


def dequantize(codes: torch.Tensor, sf: torch.Tensor, rows: int, K: int, fmt="e2m1", out=None, stream=None):
    if out is None:
        out = _empty((rows, K), torch.bfloat16, codes.device, stream)
    check(_lib.lib().mxq_dequantize(_p(codes), _p(sf), rows, K, _fmt(fmt), _p(out), _stream(stream)),
          "mxq_dequantize")
    return out


def gemm(a_codes, a_sf, fmt, M: int, K: int, w: QWeight, out=None, stream=None):
    """GEMM on an already-quantized activation: y [M, N] bf16."""
    if out is None:
        out = _empty((M, w.N), torch.bfloat16, a_codes.device, stream)
    check(_lib.lib().mxq_gemm(_p(a_codes), _p(a_sf), _fmt(fmt), M, K, _p(w.codes), _p(w.sf), w.N, _p(w.bias),
                              _p(out), _stream(stream)), "mxq_gemm")
    return out


def gemm_bf16(a: torch.Tensor, b: torch.Tensor, bias: torch.Tensor | None = None, out=None, stream=None):
    """y [M, N] = a [M, K] . b [N, K]^T (+ bias) in bf16 with fp32 accumulation, on the
    library's tcgen05 kernel (kind::f16)."""
    _cuda_bf16(a, "a")
    _cuda_bf16(b, "b")
    if bias is not None:
        _cuda_bf16(bias, "bias")
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError("a is [%d, %d] but b is [%d, %d]" % (M, K, N, b.shape[1]))
    if out is None:
        out = _empty((M, N), torch.bfloat16, a.device, stream)
    check(_lib.lib().mxq_gemm_bf16(_p(a), M, K, _p(b), N, _p(bias), _p(out), _stream(stream)), "mxq_gemm_bf16")
    return out


def gemm_bf16_quant_a(a: torch.Tensor, b: torch.Tensor, fmt="e2m1", bias: torch.Tensor | None = None, out=None,
                      codes=None, sf=None, stream=None):
    """(y, codes, sf): y [M, N] = a [M, K] . b [N, K]^T (+ bias) in bf16 (N <= 128) by the
    bf16 kernel, which also writes a's MX quantization in format fmt (codes, tiled scales:
    the bits quantize_act writes) from the same read of a."""
    _cuda_bf16(a, "a")
    _cuda_bf16(b, "b")
    if bias is not None:
        _cuda_bf16(bias, "bias")
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError("a is [%d, %d] but b is [%d, %d]" % (M, K, N, b.shape[1]))
    f = _fmt(fmt)
    if out is None:
        out = _empty((M, N), torch.bfloat16, a.device, stream)
    if codes is None:
        codes = _empty(max(1, codes_bytes(M, K, f)), torch.uint8, a.device, stream)
    if sf is None:
        sf = _empty(max(1, sf_bytes(M, K)), torch.uint8, a.device, stream)
    check(_lib.lib().mxq_gemm_bf16_quant_a(_p(a), M, K, _p(b), N, _p(bias), _p(out), f, _p(codes), _p(sf),
                                           _stream(stream)), "mxq_gemm_bf16_quant_a")
    return out, codes, sf


def linear(x: torch.Tensor, w: QWeight, fmt="e2m1", mode="native", workspace=None, out=None, stream=None):
    """y = x . deq(w)^T + bias with x quantized on the fly to fmt (E2M1 = W4A4, E4M3 = W4A8)."""
    _cuda_bf16(x, "x")
    M, K = x.shape
    f, m = _fmt(fmt), _mode(mode)
    need = workspace_bytes(M, w.N, K, f, m)
    if workspace is None:
        workspace = _empty(need, torch.uint8, x.device, stream, returned=False)
    if out is None:
        out = _empty((M, w.N), torch.bfloat16, x.device, stream)
    check(_lib.lib().mxq_linear(_p(x), M, K, _p(w.codes), _p(w.sf), w.N, _p(w.bias), f, m, _p(workspace),
                                workspace.numel() * workspace.element_size(), _p(out), _stream(stream)),
          "mxq_linear")
    return out


def linear_noalloc(x: torch.Tensor, w: QWeight, fmt="e2m1", out=None, stream=None):
    """As linear() in native mode, but the library takes its scratch from a fixed static
    device buffer instead of a workspace (for callers that cannot allocate where they run
    a layer; see mxq_linear_noalloc in include/mxq.h for the size limit and the rule that
    calls must not overlap on the GPU).  Only the output is allocated here, and only when
    `out` is not given."""
    _cuda_bf16(x, "x")
    M, K = x.shape
    if out is None:
        out = _empty((M, w.N), torch.bfloat16, x.device, stream)
    check(_lib.lib().mxq_linear_noalloc(_p(x), M, K, _p(w.codes), _p(w.sf), w.N, _p(w.bias), _fmt(fmt), _p(out),
                                        _stream(stream)), "mxq_linear_noalloc")
    return out


def gemm_gelu_quant(a_codes, a_sf, fmt, M: int, K: int, w: QWeight, out_fmt="e2m1", codes=None, sf=None,
                    h=None, stream=None):
    """GEMM whose epilogue applies bias + GELU and writes the result MX-quantized in
    out_fmt (the next layer's input): returns (codes, tiled scales).  Pass a bf16 [M, N]
    tensor as h to also receive the GELU output."""
    f = _fmt(out_fmt)
    if codes is None:
        codes = _empty(max(1, codes_bytes(M, w.N, f)), torch.uint8, a_codes.device, stream)
    if sf is None:
        sf = _empty(max(1, sf_bytes(M, w.N)), torch.uint8, a_codes.device, stream)
    if h is not None:
        _cuda_bf16(h, "h")
    check(_lib.lib().mxq_gemm_gelu_quant(_p(a_codes), _p(a_sf), _fmt(fmt), M, K, _p(w.codes), _p(w.sf), w.N,
                                         _p(w.bias), f, _p(codes), _p(sf), _p(h), _stream(stream)),
          "mxq_gemm_gelu_quant")
    return codes, sf


def gemm_quant(a_codes, a_sf, fmt, M: int, K: int, w: QWeight, act="none", out_fmt="e2m1", codes=None, sf=None,
               h=None, stream=None):
    """GEMM whose epilogue writes its output MX-quantized in out_fmt, after GELU when
    act is "gelu" (mxq_gemm_gelu_quant) or as it is when act is "none": returns (codes,
    tiled scales).  Pass a bf16 [M, N] tensor as h to also receive the quantizer's input."""
    acts = {"none": _lib.ACT_NONE, "gelu": _lib.ACT_GELU}
    if act not in acts:
        raise ValueError("act must be 'none' or 'gelu', got %r" % (act,))
    f = _fmt(out_fmt)
    if codes is None:
        codes = _empty(max(1, codes_bytes(M, w.N, f)), torch.uint8, a_codes.device, stream)
    if sf is None:
        sf = _empty(max(1, sf_bytes(M, w.N)), torch.uint8, a_codes.device, stream)
    if h is not None:
        _cuda_bf16(h, "h")
    check(_lib.lib().mxq_gemm_quant(_p(a_codes), _p(a_sf), _fmt(fmt), M, K, _p(w.codes), _p(w.sf), w.N, _p(w.bias),
                                    acts[act], f, _p(codes), _p(sf), _p(h), _stream(stream)), "mxq_gemm_quant")
    return codes, sf


def gelu_bf16(x: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """GELU of bf16 values as the quantizing epilogue applies it (exact, rounded once to bf16)."""
    _cuda_bf16(x, "x")
    if out is None:
        out = torch.empty_like(x) if stream is None else _empty(x.shape, x.dtype, x.device, stream)
    _cuda_bf16(out, "out")
    if out.numel() != x.numel():
        raise ValueError("out must have as many elements as x")
    check(_lib.lib().mxq_gelu_bf16(_p(x), x.numel(), _p(out), _stream(stream)), "mxq_gelu_bf16")
    return out


def ffn_workspace_bytes(M: int, K: int, H: int, up_fmt="e2m1", down_fmt="e2m1") -> int:
    return int(_lib.lib().mxq_ffn_workspace_bytes(M, K, H, _fmt(up_fmt), _fmt(down_fmt)))


def ffn(x: torch.Tensor, up: QWeight, down: QWeight, up_fmt="e2m1", down_fmt="e2m1", workspace=None, out=None,
        stream=None):
    """y = quant(GELU(x . up^T + b_up)) . down^T + b_down with the hidden activation kept
    MX-quantized between the two linears."""
    _cuda_bf16(x, "x")
    M, K = x.shape
    if workspace is None:
        workspace = _empty(ffn_workspace_bytes(M, K, up.N, up_fmt, down_fmt), torch.uint8, x.device, stream,
                           returned=False)
    if out is None:
        out = _empty((M, down.N), torch.bfloat16, x.device, stream)
    du, dd = up.desc(), down.desc()
    check(_lib.lib().mxq_ffn(_p(x), M, K, ctypes.byref(du), ctypes.byref(dd), _fmt(up_fmt), _fmt(down_fmt),
                             _p(workspace), workspace.numel(), _p(out), _stream(stream)), "mxq_ffn")
    return out


def absmax(x: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """max |x| over a bf16 tensor, as a one-element fp32 CUDA tensor (calibration)."""
    _cuda_bf16(x, "x")
    if out is None:
        out = _empty(1, torch.float32, x.device, stream)
    check(_lib.lib().mxq_absmax(_p(x), x.numel(), _p(out), _stream(stream)), "mxq_absmax")
    return out


def quantize_act_static(x: torch.Tensor, scale: float, codes=None, sf=None, stream=None):
    """x [M, K] bf16 -> static per-tensor E4M3 codes [M, K] and tiled scales (all 127)."""
    _cuda_bf16(x, "x")
    M, K = x.shape
    if codes is None:
        codes = _empty(max(1, codes_bytes(M, K, FMT_E4M3)), torch.uint8, x.device, stream)
    if sf is None:
        sf = _empty(max(1, sf_bytes(M, K)), torch.uint8, x.device, stream)
    check(_lib.lib().mxq_quantize_act_static(_p(x), M, K, float(scale), _p(codes), _p(sf), _stream(stream)),
          "mxq_quantize_act_static")
    return codes, sf


def linear_static(x: torch.Tensor, w: QWeight, act_scale: float, workspace=None, out=None, stream=None):
    """y = act_scale * (static E4M3 codes of x) . deq(w)^T + bias (W4A8, static activations)."""
    _cuda_bf16(x, "x")
    M, K = x.shape
    if workspace is None:
        workspace = _empty(workspace_bytes(M, w.N, K, FMT_E4M3, MODE_NATIVE), torch.uint8, x.device, stream,
                           returned=False)
    if out is None:
        out = _empty((M, w.N), torch.bfloat16, x.device, stream)
    check(_lib.lib().mxq_linear_static(_p(x), M, K, _p(w.codes), _p(w.sf), w.N, _p(w.bias), float(act_scale),
                                       _p(workspace), workspace.numel(), _p(out), _stream(stream)),
          "mxq_linear_static")
    return out


def _f32_or_none(t, name):
    if t is None:
        return None
    if not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()):
        raise ValueError("%s must be a contiguous float32 CUDA tensor" % name)
    return t


def quantize_act_transformed(x: torch.Tensor, fmt="e2m1", block=32, mul=None, codes=None, sf=None, stream=None):
    """x [M, K] bf16 -> MX codes and tiled scales of (x * mul) rotated by the block Hadamard."""
    _cuda_bf16(x, "x")
    M, K = x.shape
    f = _fmt(fmt)
    mul = _f32_or_none(mul, "mul")
    if codes is None:
        codes = _empty(max(1, codes_bytes(M, K, f)), torch.uint8, x.device, stream)
    if sf is None:
        sf = _empty(max(1, sf_bytes(M, K)), torch.uint8, x.device, stream)
    check(_lib.lib().mxq_quantize_act_transformed(_p(x), M, K, f, _p(mul), int(block), _p(codes), _p(sf),
                                                  _stream(stream)), "mxq_quantize_act_transformed")
    return codes, sf


def quantize_weight_transformed(w: torch.Tensor, bias=None, block=32, mul=None, stream=None) -> QWeight:
    """w [N, K] bf16 -> QWeight of (w * mul) rotated by the block Hadamard (mul = s)."""
    _cuda_bf16(w, "w")
    N, K = w.shape
    mul = _f32_or_none(mul, "mul")
    codes = _empty((N, K // 2), torch.uint8, w.device, stream)
    sf = _empty(max(1, sf_bytes(N, K)), torch.uint8, w.device, stream)
    check(_lib.lib().mxq_quantize_weight_transformed(_p(w), N, K, _p(mul), int(block), _p(codes), _p(sf),
                                                     _stream(stream)), "mxq_quantize_weight_transformed")
    if bias is not None:
        _cuda_bf16(bias, "bias")
    return QWeight(codes, sf, N, K, bias)


def linear_transformed(x: torch.Tensor, w: QWeight, fmt="e2m1", block=32, act_mul=None, workspace=None, out=None,
                       stream=None):
    """The linear on the transformed path (w from quantize_weight_transformed, same block)."""
    _cuda_bf16(x, "x")
    M, K = x.shape
    f = _fmt(fmt)
    act_mul = _f32_or_none(act_mul, "act_mul")
    if workspace is None:
        workspace = _empty(workspace_bytes(M, w.N, K, f, MODE_NATIVE), torch.uint8, x.device, stream,
                           returned=False)
    if out is None:
        out = _empty((M, w.N), torch.bfloat16, x.device, stream)
    check(_lib.lib().mxq_linear_transformed(_p(x), M, K, _p(w.codes), _p(w.sf), w.N, _p(w.bias), f, _p(act_mul),
                                            int(block), _p(workspace), workspace.numel(), _p(out), _stream(stream)),
          "mxq_linear_transformed")
    return out


def lowrank_split(w: torch.Tensor, U: torch.Tensor, S: torch.Tensor, Vh: torch.Tensor, rank: int, stream=None):
    """The SVDQuant split of w [N, K] bf16 from its singular triplets (U [N, >= rank],
    S [>= rank], Vh [>= rank, K], fp32 CUDA tensors, the first `rank` used), in the library:
    l2t = bf16(U sqrt(S)) [N, rank], l1t = bf16(sqrt(S) Vh) [rank, K] and the residual
    bf16(w - l2t . l1t) [N, K].  Returns (l1t, l2t, residual)."""
    _cuda_bf16(w, "w")
    N, K = w.shape
    for t, name in ((U, "U"), (S, "S"), (Vh, "Vh")):
        if not (t.is_cuda and t.dtype == torch.float32 and t.stride(-1) == 1):
            raise ValueError("%s must be a float32 CUDA tensor with unit inner stride" % name)
    if U.shape[0] != N or Vh.shape[1] != K or min(U.shape[1], S.shape[0], Vh.shape[0]) < rank:
        raise ValueError("factors of shapes %s, %s, %s do not fit w [%d, %d] at rank %d" % (
            tuple(U.shape), tuple(S.shape), tuple(Vh.shape), N, K, rank))
    l2t = _empty((N, rank), torch.bfloat16, w.device, stream)
    l1t = _empty((rank, K), torch.bfloat16, w.device, stream)
    resid = _empty((N, K), torch.bfloat16, w.device, stream)
    check(_lib.lib().mxq_lowrank_split(_p(U), U.stride(0), _p(S), _p(Vh), Vh.stride(0), _p(w), N, K, rank, _p(l2t),
                                       _p(l1t), _p(resid), _stream(stream)), "mxq_lowrank_split")
    return l1t, l2t, resid


def svd_split(w: torch.Tensor, rank: int, stream=None):
    """Offline weight preparation of the SVDQuant branch (load time, not the layer's path):
    the singular value decomposition of w in fp32 is a library factorization (torch's),
    the split into l2t = U_r sqrt(S_r), l1t = sqrt(S_r) V_r^T and the bf16 residual
    w - l2t . l1t runs in this library (lowrank_split).  Returns (l1t, l2t, residual)."""
    _cuda_bf16(w, "w")
    if stream is not None:  # the decomposition runs there too
        caller = torch.cuda.current_stream(w.device)
        with torch.cuda.stream(stream):
            parts = svd_split(w, rank)
        for t in parts:
            t.record_stream(caller)
        return parts
    U, S, Vh = torch.linalg.svd(w.float(), full_matrices=False)
    return lowrank_split(w, U.contiguous(), S.contiguous(), Vh.contiguous(), rank)


def channel_absmax(x: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """max over rows of |x[:, k]| for a bf16 [rows, K] tensor, as K float32 values."""
    _cuda_bf16(x, "x")
    rows, K = x.shape
    if out is None:
        out = _empty(K, torch.float32, x.device, stream)
    check(_lib.lib().mxq_channel_absmax(_p(x), rows, K, _p(out), _stream(stream)), "mxq_channel_absmax")
    return out


def smooth_scales(amax_x: torch.Tensor, amax_w: torch.Tensor, alpha: float = 0.5, with_inverse: bool = False,
                  stream=None):
    """SmoothQuant's s_k = max(amax_x_k, 1e-5)^alpha / max(amax_w_k, 1e-5)^(1 - alpha);
    with_inverse: also 1 / s_k (the activation's multiplier), returned as (s, 1/s)."""
    amax_x = _f32_or_none(amax_x, "amax_x")
    amax_w = _f32_or_none(amax_w, "amax_w")
    K = amax_x.numel()
    if amax_w.numel() != K:
        raise ValueError("channel counts differ: %d vs %d" % (K, amax_w.numel()))
    s = _empty(K, torch.float32, amax_x.device, stream)
    inv = _empty(K, torch.float32, amax_x.device, stream) if with_inverse else None
    check(_lib.lib().mxq_smooth_scales(_p(amax_x), _p(amax_w), K, float(alpha), _p(s), _p(inv), _stream(stream)),
          "mxq_smooth_scales")
    return (s, inv) if with_inverse else s


def sqnr(refs, tests, out=None, stream=None) -> torch.Tensor:
    """SQNR over pairs of bf16 tensors: a float64 CUDA tensor [sum ref^2, sum (ref - test)^2,
    dB]."""
    refs, tests = list(refs), list(tests)
    if len(refs) != len(tests) or not refs:
        raise ValueError("need as many test tensors as reference tensors, at least one")
    for r, t in zip(refs, tests):
        _cuda_bf16(r, "ref")
        _cuda_bf16(t, "test")
        if r.numel() != t.numel():
            raise ValueError("a reference and its test tensor differ in size")
    if out is None:
        out = _empty(3, torch.float64, refs[0].device, stream)
    n = len(refs)
    rp = (ctypes.c_void_p * n)(*[r.data_ptr() for r in refs])
    tp = (ctypes.c_void_p * n)(*[t.data_ptr() for t in tests])
    ns = (ctypes.c_int64 * n)(*[r.numel() for r in refs])
    check(_lib.lib().mxq_sqnr(rp, tp, ns, n, _p(out), _stream(stream)), "mxq_sqnr")
    return out


_NORMS = {"none": _lib.NORM_NONE, "layer": _lib.NORM_LAYER, "rms": _lib.NORM_RMS}
_OUTS = {"bf16": _lib.OUT_BF16, **_FMTS}
_VEC_DTYPES = {torch.bfloat16: _lib.DTYPE_BF16, torch.float32: _lib.DTYPE_F32}


def _pick(table, key, what):
    if key not in table:
        raise ValueError("%s must be one of %s, got %r" % (what, ", ".join(repr(k) for k in table if isinstance(k, str)),
                                                           key))
    return table[key]


def _tensor(t, name, dtype, shape, device) -> int:
    """The address of t, checked to be a contiguous tensor of that dtype, shape and device."""
    if not (t.dtype == dtype and t.shape == shape and t.is_contiguous() and t.device == device):
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s, got %s %s on %s" % (
            name, dtype, tuple(shape), device, t.dtype, tuple(t.shape), t.device))
    return t.data_ptr()


def _opt(t, name, dtype, shape, device) -> int:
    return 0 if t is None else _tensor(t, name, dtype, shape, device)


def _current_device(x: torch.Tensor) -> torch.device:
    """x's device, which has to be the current one: the library launches there."""
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("expected CUDA tensors, got one on %s" % dev)
    if dev.index != torch.cuda.current_device():
        raise ValueError("tensors are on %s but the current device is cuda:%d" % (dev, torch.cuda.current_device()))
    return dev


def _raw_stream(stream, dev) -> int:
    """The stream's handle: the given stream, or the device's current one."""
    return torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream


def _group_vec(t, name, dtype, rows, K, rows_per_group, device) -> int:
    """The address of per-group vectors [groups, K] ([K] for one group), or 0."""
    if t is None:
        return 0
    groups = -(-rows // rows_per_group)
    shape = t.shape
    ok = len(shape) == 2 and shape[0] >= groups or len(shape) == 1 and groups == 1
    if not ok or shape[-1] != K or t.dtype != dtype or not t.is_contiguous() or t.device != device:
        raise ValueError("%s must be a contiguous %s tensor [%d, %d] on %s, got %s %s on %s" % (
            name, dtype, groups, K, device, t.dtype, tuple(t.shape), t.device))
    return t.data_ptr()


def _rows_per_group(rows_per_group, rows):
    if rows_per_group is None:
        return max(1, rows)
    if rows_per_group <= 0:
        raise ValueError("rows_per_group must be positive, got %r" % (rows_per_group,))
    return int(rows_per_group)


def _mx_bytes(rows: int, K: int, f: int):
    """mxq_codes_bytes and mxq_sf_bytes, at least 1 (the library refuses sizes they do not fit)."""
    return (max(1, rows * K if f == FMT_E4M3 else rows * K // 2),
            max(1, (rows + 127) // 128 * 128 * ((K // 32 + 3) // 4) * 4))


def _codes_out(codes, sf, rows, K, f, dev, stream):
    """The buffers of a quantized [rows, K] output: the caller's, checked, or new ones."""
    nc, ns = _mx_bytes(rows, K, f)
    for t, n, name in ((codes, nc, "codes"), (sf, ns, "sf")):
        if t is not None and not (t.dtype == torch.uint8 and t.is_contiguous() and t.numel() >= n and t.device == dev):
            raise ValueError("%s must be a contiguous uint8 tensor of at least %d bytes on %s" % (name, n, dev))
    codes = _empty(nc, torch.uint8, dev, stream) if codes is None else codes
    sf = _empty(ns, torch.uint8, dev, stream) if sf is None else sf
    return codes, sf


def norm_residual(x: torch.Tensor, y: torch.Tensor | None = None, norm="layer", weight=None, bias=None, gate=None,
                  scale=None, shift=None, rows_per_group=None, post_norm="none", post_weight=None, post_bias=None,
                  eps=1e-6, out_fmt="bf16", z=None, h=None, codes=None, sf=None, stream=None):
    """The norms before and after a block with its gate, residual and modulation, in one pass:
        z = x + gate * post_norm(y),   h = norm(z) * (1 + scale) + shift
    x [rows, K] is the residual stream (bf16 or float32; z has its type), y [rows, K] bf16 the
    block's output (None: z is x, and x is returned as z).  norm "layer" or "rms", post_norm
    also "none".  weight, bias, post_weight, post_bias [K], gate, scale, shift [groups, K] or
    [K] are all bf16 or all float32; row r uses group r // rows_per_group.  Returns (z, h)
    with h bf16, or, for out_fmt "e2m1" / "e4m3", (z, codes, tiled scales): the bits that
    quantize_act writes for that h.  z may be x; no other output may overlap an input."""
    dev = _current_device(x)
    xdt = x.dtype
    if xdt not in _VEC_DTYPES or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 or float32 tensor [rows, K]")
    shape = x.shape
    rows, K = shape
    f = _pick(_OUTS, out_fmt, "out_fmt")
    rpg = _rows_per_group(rows_per_group, rows)
    vdt = torch.float32  # of the channel vectors, unless one of them says otherwise
    for v in (weight, bias, post_weight, post_bias, gate, scale, shift):
        if v is not None:
            vdt = v.dtype
            break
    if vdt not in _VEC_DTYPES:
        raise ValueError("the channel vectors must be bf16 or float32, got %s" % vdt)
    zp = 0
    if y is not None:
        if z is None:
            # (empty_like is 2 us faster than a shape to parse)
            z = torch.empty_like(x) if stream is None else _empty(shape, xdt, dev, stream)
            zp = z.data_ptr()
        else:
            zp = _tensor(z, "z", xdt, shape, dev)
    elif z is not None:
        raise ValueError("z goes with y")
    if f == _lib.OUT_BF16:
        out = _bf16_out(h, rows, K, dev, stream, "h")
    else:
        out, sf = _codes_out(codes, sf, rows, K, f, dev, stream)
    d = _lib.NormDesc(x.data_ptr(), _opt(y, "y", torch.bfloat16, shape, dev), rows, K, _VEC_DTYPES[xdt],
                      _VEC_DTYPES[vdt], _pick(_NORMS, norm, "norm"), _pick(_NORMS, post_norm, "post_norm"),
                      _opt(weight, "weight", vdt, (K,), dev), _opt(bias, "bias", vdt, (K,), dev),
                      _opt(post_weight, "post_weight", vdt, (K,), dev), _opt(post_bias, "post_bias", vdt, (K,), dev),
                      _group_vec(gate, "gate", vdt, rows, K, rpg, dev),
                      _group_vec(scale, "scale", vdt, rows, K, rpg, dev),
                      _group_vec(shift, "shift", vdt, rows, K, rpg, dev), rpg, eps)
    quant = f != _lib.OUT_BF16
    check(_lib.lib().mxq_norm_residual(d, zp, f, out.data_ptr(), sf.data_ptr() if quant else 0,
                                       _raw_stream(stream, dev)), "mxq_norm_residual")
    z = x if y is None else z
    return (z, out, sf) if quant else (z, out)


ROWS_QUANTIZED_IN_KERNEL = 16  # mxq_linear_residual quantizes so few rows inside its GEMM kernel

_ACTS = {"none": _lib.ACT_NONE, "gelu": _lib.ACT_GELU, "gelu_tanh": _lib.ACT_GELU_TANH, "silu": _lib.ACT_SILU}


def _act(a) -> int:
    return _pick(_ACTS, a, "act")


def _epilogue(act, residual, gate, rows_per_group, M, N, dev):
    """The checked mxq_epilogue of an [M, N] output."""
    rpg = _rows_per_group(rows_per_group, M)
    gdt = torch.bfloat16 if gate is None else gate.dtype
    if gdt not in _VEC_DTYPES:
        raise ValueError("gate must be bf16 or float32, got %s" % gdt)
    return _lib.Epilogue(_act(act), _VEC_DTYPES[gdt], _opt(residual, "residual", torch.bfloat16, (M, N), dev),
                         _group_vec(gate, "gate", gdt, M, N, rpg, dev), rpg)


def _operand(codes, sf, M, K, f) -> torch.device:
    """The device of a quantized [M, K] operand, its buffers checked."""
    dev = _current_device(codes)
    nc, ns = _mx_bytes(M, K, f)
    if not (codes.nbytes >= nc and sf.nbytes >= ns and codes.is_contiguous() and sf.is_contiguous() and
            sf.device == dev):
        raise ValueError("a_codes and a_sf must be contiguous tensors of %d and %d bytes on %s" % (nc, ns, dev))
    return dev


def _qweight(w: QWeight, name, dev) -> WDesc:
    """The checked descriptor of a weight."""
    N, K, codes, sf, bias = w.N, w.K, w.codes, w.sf, w.bias
    nc, ns = _mx_bytes(N, K, FMT_E2M1)
    if not (codes.nbytes >= nc and sf.nbytes >= ns and codes.is_contiguous() and sf.is_contiguous() and
            codes.device == dev and sf.device == dev):
        raise ValueError("%s must hold contiguous tensors of %d and %d bytes on %s" % (name, nc, ns, dev))
    return WDesc(codes.data_ptr(), sf.data_ptr(), _opt(bias, "bias", torch.bfloat16, (N,), dev), N, K)


def _bf16_x(x, name) -> torch.device:
    dev = _current_device(x)
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("%s must be a contiguous bf16 tensor [rows, K], got %s %s" % (name, x.dtype, tuple(x.shape)))
    return dev


def _workspace(ws, need, dev, stream):
    """The caller's workspace, or a new one that belongs to the stream its kernels run on (one of
    another stream could be handed out again while they still use it)."""
    if ws is None:
        return _empty(max(1, need), torch.uint8, dev, stream, returned=False)
    if ws.device != dev or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % dev)
    return ws


def _bf16_out(out, M, N, dev, stream, name="out"):
    if out is None:
        return _empty((M, N), torch.bfloat16, dev, stream)
    _tensor(out, name, torch.bfloat16, (M, N), dev)
    return out


def _check_k(w: QWeight, K, name="w"):
    if w.K != K:
        raise ValueError("%s has K=%d but the activation has %d" % (name, w.K, K))


def gemm_residual(a_codes, a_sf, fmt, M: int, K: int, w: QWeight, act="none", residual=None, gate=None,
                  rows_per_group=None, out=None, stream=None):
    """y = residual + gate * act(a . deq(w)^T + bias) [M, N] bf16, rounded once, on an
    already-quantized activation.  act "none", "gelu", "gelu_tanh" or "silu"; residual [M, N]
    bf16 (it may be out; otherwise out must not overlap it, nor the activation: refused); gate [groups, N] or [N], bf16 or float32, row m using group
    m // rows_per_group (default: one group)."""
    f = _fmt(fmt)
    dev = _operand(a_codes, a_sf, M, K, f)
    _check_k(w, K)
    d = _qweight(w, "w", dev)
    e = _epilogue(act, residual, gate, rows_per_group, M, w.N, dev)
    out = _bf16_out(out, M, w.N, dev, stream)
    check(_lib.lib().mxq_gemm_residual(a_codes.data_ptr(), a_sf.data_ptr(), f, M, K, d.codes, d.sf, w.N, d.bias, e,
                                       out.data_ptr(), _raw_stream(stream, dev)), "mxq_gemm_residual")
    return out


def gemm_bf16_residual(a: torch.Tensor, b: torch.Tensor, bias: torch.Tensor | None = None, act="none", residual=None,
                       gate=None, rows_per_group=None, out=None, stream=None):
    """y = residual + gate * act(a . b^T + bias) in bf16 with fp32 accumulation, a [M, K] and
    b [N, K] bf16; the other arguments as for gemm_residual.  out must not overlap a (refused),
    also where a is the residual."""
    dev = _bf16_x(a, "a")
    M, K = a.shape
    N = b.shape[0]
    bp = _tensor(b, "b", torch.bfloat16, (N, K), dev)
    e = _epilogue(act, residual, gate, rows_per_group, M, N, dev)
    out = _bf16_out(out, M, N, dev, stream)
    check(_lib.lib().mxq_gemm_bf16_residual(a.data_ptr(), M, K, bp, N, _opt(bias, "bias", torch.bfloat16, (N,), dev),
                                            e, out.data_ptr(), _raw_stream(stream, dev)), "mxq_gemm_bf16_residual")
    return out


def linear_residual(x: torch.Tensor, w: QWeight, fmt="e2m1", act="none", residual=None, gate=None,
                    rows_per_group=None, workspace=None, out=None, stream=None):
    """linear() with gemm_residual's epilogue: x quantized on the fly to fmt, then
    y = residual + gate * act(x . deq(w)^T + bias).  workspace of
    workspace_bytes(M, N, K, fmt) bytes; up to ROWS_QUANTIZED_IN_KERNEL rows need none.  out
    must not overlap x (refused), also where x is the residual."""
    dev = _bf16_x(x, "x")
    M, K = x.shape
    f = _fmt(fmt)
    _check_k(w, K)
    d = _qweight(w, "w", dev)
    e = _epilogue(act, residual, gate, rows_per_group, M, w.N, dev)
    ws = wsb = 0
    if workspace is not None or M > ROWS_QUANTIZED_IN_KERNEL:
        nc, ns = _mx_bytes(M, K, f)
        workspace = _workspace(workspace, (nc + 255) // 256 * 256 + (ns + 255) // 256 * 256, dev, stream)
        ws, wsb = workspace.data_ptr(), workspace.nbytes
    out = _bf16_out(out, M, w.N, dev, stream)
    check(_lib.lib().mxq_linear_residual(x.data_ptr(), M, K, d.codes, d.sf, w.N, d.bias, f, e, ws, wsb,
                                         out.data_ptr(), _raw_stream(stream, dev)), "mxq_linear_residual")
    return out


def _gated_out(M, H, out_fmt, out, codes, sf, dev, stream):
    """(out_fmt, h or codes, scales or None) of a gated GEMM."""
    f = _pick(_OUTS, out_fmt, "out_fmt")
    if f == _lib.OUT_BF16:
        return f, _bf16_out(out, M, H, dev, stream), None
    codes, sf = _codes_out(codes, sf, M, H, f, dev, stream)
    return f, codes, sf


def gemm_gated(a_codes, a_sf, fmt, M: int, K: int, gate: QWeight, up: QWeight, act="silu", out_fmt="bf16", out=None,
               codes=None, sf=None, stream=None):
    """h = act(a . deq(gate)^T + gate.bias) * (a . deq(up)^T + up.bias) [M, H] in one kernel,
    on an already-quantized activation.  Returns h in bf16, or, for out_fmt "e2m1" / "e4m3",
    (codes, tiled scales): the bits that quantize_act writes for that h.  No output may overlap
    the activation (refused)."""
    f = _fmt(fmt)
    dev = _operand(a_codes, a_sf, M, K, f)
    dg, du = _qweight(gate, "gate", dev), _qweight(up, "up", dev)
    of, o, so = _gated_out(M, gate.N, out_fmt, out, codes, sf, dev, stream)
    check(_lib.lib().mxq_gemm_gated(a_codes.data_ptr(), a_sf.data_ptr(), f, M, K, dg, du, _act(act), of, o.data_ptr(),
                                    0 if so is None else so.data_ptr(), _raw_stream(stream, dev)), "mxq_gemm_gated")
    return o if so is None else (o, so)


def gemm_bf16_gated(a: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, gate_bias=None, up_bias=None, act="silu",
                    out_fmt="bf16", out=None, codes=None, sf=None, stream=None):
    """gemm_gated on bf16 operands: a [M, K], gate and up [H, K]."""
    dev = _bf16_x(a, "a")
    M, K = a.shape
    H = gate.shape[0]
    gp, up_ = _tensor(gate, "gate", torch.bfloat16, (H, K), dev), _tensor(up, "up", torch.bfloat16, (H, K), dev)
    gb, ub = (_opt(b, n, torch.bfloat16, (H,), dev) for b, n in ((gate_bias, "gate_bias"), (up_bias, "up_bias")))
    of, o, so = _gated_out(M, H, out_fmt, out, codes, sf, dev, stream)
    check(_lib.lib().mxq_gemm_bf16_gated(a.data_ptr(), M, K, gp, gb, up_, ub, H, _act(act), of, o.data_ptr(),
                                         0 if so is None else so.data_ptr(), _raw_stream(stream, dev)),
          "mxq_gemm_bf16_gated")
    return o if so is None else (o, so)


def gated_ffn(x: torch.Tensor, gate: QWeight, up: QWeight, down: QWeight, act="silu", up_fmt="e2m1",
              down_fmt="e2m1", residual=None, out_gate=None, rows_per_group=None, workspace=None, out=None,
              stream=None):
    """The gated feed-forward network y = residual + out_gate * (quant(act(x . gate^T) *
    (x . up^T)) . down^T), biases included, with x quantized to up_fmt and the hidden
    activation kept quantized in down_fmt.  residual, out_gate and rows_per_group as
    gemm_residual's residual, gate and rows_per_group; out may be x; workspace of
    ffn_workspace_bytes(M, K, H, up_fmt, down_fmt) bytes."""
    dev = _bf16_x(x, "x")
    M, K = x.shape
    dg, du, dd = _qweight(gate, "gate", dev), _qweight(up, "up", dev), _qweight(down, "down", dev)
    e = _epilogue("none", residual, out_gate, rows_per_group, M, down.N, dev)
    uf, df = _fmt(up_fmt), _fmt(down_fmt)
    need = sum((n + 255) // 256 * 256 for n in _mx_bytes(M, K, uf) + _mx_bytes(M, gate.N, df))
    workspace = _workspace(workspace, need, dev, stream)
    out = _bf16_out(out, M, down.N, dev, stream)
    check(_lib.lib().mxq_gated_ffn(x.data_ptr(), M, K, dg, du, dd, _act(act), uf, df, e, workspace.data_ptr(),
                                   workspace.nbytes, out.data_ptr(),
                                   _raw_stream(stream, dev)), "mxq_gated_ffn")
    return out


def lowrank_workspace_bytes(M: int, N: int, K: int, fmt="e2m1", rank=64) -> int:
    return int(_lib.lib().mxq_lowrank_workspace_bytes(M, N, K, _fmt(fmt), int(rank)))


def linear_lowrank(x: torch.Tensor, residual: QWeight, l1t: torch.Tensor, l2t: torch.Tensor, fmt="e2m1",
                   workspace=None, out=None, stream=None):
    """y = deq(xq) . deq(Rq)^T + bf16(x . l1t^T) . l2t^T + bias (SVDQuant branch in the
    same accumulator)."""
    _cuda_bf16(x, "x")
    _cuda_bf16(l1t, "l1t")
    _cuda_bf16(l2t, "l2t")
    M, K = x.shape
    rank = l1t.shape[0]
    f = _fmt(fmt)
    if workspace is None:
        workspace = _empty(lowrank_workspace_bytes(M, residual.N, K, f, rank), torch.uint8, x.device, stream,
                           returned=False)
    if out is None:
        out = _empty((M, residual.N), torch.bfloat16, x.device, stream)
    check(_lib.lib().mxq_linear_lowrank(_p(x), M, K, _p(residual.codes), _p(residual.sf), residual.N,
                                        _p(residual.bias), f, _p(l1t), _p(l2t), rank, _p(workspace),
                                        workspace.numel(), _p(out), _stream(stream)), "mxq_linear_lowrank")
    return out


def block_workspace_bytes(weights, rows, w4a8_bits: int, mode="native", minimum: bool = False) -> int:
    """Workspace of dit_block_linears: by default the size that lets the quantizers overlap
    the GEMMs (native mode); minimum=True gives the least it accepts."""
    descs = (WDesc * 8)(*[w.desc() for w in weights])
    ms = (ctypes.c_int64 * 8)(*rows)
    fn = _lib.lib().mxq_block_workspace_min_bytes if minimum else _lib.lib().mxq_block_workspace_bytes
    return int(fn(descs, ms, w4a8_bits, _mode(mode)))


def dit_block_linears(weights, xs, w4a8_bits: int, mode="native", workspace=None, outs=None, stream=None):
    """The eight linears of one DiT block (QKV, attn-out, cross-Q/K/V/out, FFN-up,
    FFN-down); bit i of w4a8_bits selects W4A8 for linear i."""
    assert len(weights) == 8 and len(xs) == 8
    rows = [int(x.shape[0]) for x in xs]
    for x in xs:
        _cuda_bf16(x, "block input")
    if outs is None:
        outs = [_empty((r, w.N), torch.bfloat16, xs[0].device, stream) for r, w in zip(rows, weights)]
    need = block_workspace_bytes(weights, rows, w4a8_bits, mode)
    if workspace is None:
        workspace = _empty(need, torch.uint8, xs[0].device, stream, returned=False)
    descs = (WDesc * 8)(*[w.desc() for w in weights])
    xin = (ctypes.c_void_p * 8)(*[x.data_ptr() for x in xs])
    ms = (ctypes.c_int64 * 8)(*rows)
    yout = (ctypes.c_void_p * 8)(*[y.data_ptr() for y in outs])
    check(_lib.lib().mxq_dit_block_linears(descs, xin, ms, yout, w4a8_bits, _mode(mode), _p(workspace),
                                           workspace.numel(), _stream(stream)), "mxq_dit_block_linears")
    return outs


def sf_to_logical(sf: torch.Tensor, rows: int, K: int, stream=None) -> torch.Tensor:
    out = _empty((rows, K // 32), torch.uint8, sf.device, stream)
    check(_lib.lib().mxq_sf_to_logical(_p(sf), rows, K, _p(out), _stream(stream)), "mxq_sf_to_logical")
    return out


def poll_status(stream=None) -> int:
    """Synchronizes the stream and returns the device status word (0 = fine)."""
    return int(_lib.lib().mxq_poll_status(_stream(stream)))


def set_debug(flags: int) -> None:
    _lib.lib().mxq_set_debug(flags)


def last_path() -> str:
    return _lib.last_path()
