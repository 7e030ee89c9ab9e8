"""Memory of calls that are given a stream: what the binding allocates for them comes from that
stream, so that nothing queued on the current stream still reads it or gets it again, and what
they return is noted as used by the current stream.  The library is a stand-in that computes
nothing, torch's streams are stand-ins that note what is allocated under them: no GPU."""
import contextlib

import pytest
import torch

from fp8_mixed_precision_mxq_b200 import _lib, ops

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


class Library:
    """Sizes from the library; calls that note their stream and succeed."""

    def __init__(self, real):
        self.real, self.streams = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*args):
            self.streams.append(getattr(args[-1], "value", args[-1]))
            return 0
        return call


class Stream:
    cuda_stream = 0x5EED


@pytest.fixture
def streams(monkeypatch):
    side, current, log = Stream(), object(), {"under": [], "made": [], "noted": []}

    @contextlib.contextmanager
    def under(s):
        log["under"].append(s)
        yield
        log["under"].pop()

    empty = torch.empty

    def made(*args, **kw):
        t = empty(*args, **kw)
        log["made"].append((t, list(log["under"])))
        return t

    lib = Library(_lib.lib())
    monkeypatch.setattr(_lib, "_lib", lib)
    monkeypatch.setattr(torch, "empty", made)
    monkeypatch.setattr(torch, "empty_like", lambda t: made(t.shape, dtype=t.dtype, device=t.device))
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log["noted"].append((t, s)))
    monkeypatch.setattr(ops, "_current_device", lambda t: t.device)
    monkeypatch.setattr(ops, "_cuda_bf16", lambda t, name: None)
    monkeypatch.setattr(ops, "_f32_or_none", lambda t, name: t)
    return side, current, lib, log


def weight(N, K):
    return ops.QWeight(torch.zeros(N, K // 2, dtype=U8), torch.zeros(ops._mx_bytes(N, K, 0)[1], dtype=U8), N, K)


M, K, H = 80, 256, 384
X = torch.zeros(M, K, dtype=BF16)
XC, XS = (torch.zeros(n, dtype=U8) for n in ops._mx_bytes(M, K, 1))
AROUND = {  # what a transformer block computes between its linears
    "norm_residual": lambda s: ops.norm_residual(X, X, stream=s),
    "norm_residual quantized": lambda s: ops.norm_residual(X.float(), X, out_fmt="e4m3", stream=s),
    "norm_residual without y": lambda s: ops.norm_residual(X, stream=s)[1:],
    "gemm_residual": lambda s: ops.gemm_residual(XC, XS, "e4m3", M, K, weight(H, K), stream=s),
    "gemm_bf16_residual": lambda s: ops.gemm_bf16_residual(X, torch.zeros(H, K, dtype=BF16), stream=s),
    "linear_residual": lambda s: ops.linear_residual(X, weight(H, K), stream=s),
    "gemm_gated": lambda s: ops.gemm_gated(XC, XS, "e4m3", M, K, weight(H, K), weight(H, K), stream=s),
    "gemm_gated quantized": lambda s: ops.gemm_gated(XC, XS, "e4m3", M, K, weight(H, K), weight(H, K),
                                                     out_fmt="e2m1", stream=s),
    "gemm_bf16_gated": lambda s: ops.gemm_bf16_gated(X, torch.zeros(H, K, dtype=BF16), torch.zeros(H, K, dtype=BF16),
                                                     stream=s),
    "gemm_bf16_gated quantized": lambda s: ops.gemm_bf16_gated(X, torch.zeros(H, K, dtype=BF16),
                                                               torch.zeros(H, K, dtype=BF16), out_fmt="e4m3",
                                                               stream=s),
    "gated_ffn": lambda s: ops.gated_ffn(X, weight(H, K), weight(H, K), weight(K, H), stream=s),
}


W, W8 = weight(H, K), [weight(K, K)] * 6 + [weight(H, K), weight(K, H)]
ROWS8 = [X] * 7 + [torch.zeros(M, H, dtype=BF16)]
L1, L2 = torch.zeros(64, K, dtype=BF16), torch.zeros(H, 64, dtype=BF16)
V = torch.zeros(K, dtype=F32)
EARLIER = {  # quantizers, linears and calibration
    "quantize_act": lambda s: ops.quantize_act(X, stream=s),
    "quantize_weight": lambda s: parts(ops.quantize_weight(X, stream=s)),
    "dequantize": lambda s: ops.dequantize(XC, XS, M, K, "e4m3", stream=s),
    "gemm": lambda s: ops.gemm(XC, XS, "e4m3", M, K, W, stream=s),
    "gemm_bf16": lambda s: ops.gemm_bf16(X, torch.zeros(H, K, dtype=BF16), stream=s),
    "gemm_bf16_quant_a": lambda s: ops.gemm_bf16_quant_a(X, L1, stream=s),
    "linear": lambda s: ops.linear(X, W, stream=s),
    "linear qdq": lambda s: ops.linear(X, W, mode="qdq", stream=s),
    "linear_noalloc": lambda s: ops.linear_noalloc(X, W, stream=s),
    "gemm_gelu_quant": lambda s: ops.gemm_gelu_quant(XC, XS, "e4m3", M, K, W, stream=s),
    "gemm_quant": lambda s: ops.gemm_quant(XC, XS, "e4m3", M, K, W, stream=s),
    "gelu_bf16": lambda s: ops.gelu_bf16(X, stream=s),
    "ffn": lambda s: ops.ffn(X, W, weight(K, H), stream=s),
    "absmax": lambda s: ops.absmax(X, stream=s),
    "quantize_act_static": lambda s: ops.quantize_act_static(X, 1.0, stream=s),
    "linear_static": lambda s: ops.linear_static(X, W, 1.0, stream=s),
    "quantize_act_transformed": lambda s: ops.quantize_act_transformed(X, stream=s),
    "quantize_weight_transformed": lambda s: parts(ops.quantize_weight_transformed(X, stream=s)),
    "linear_transformed": lambda s: ops.linear_transformed(X, W, stream=s),
    "channel_absmax": lambda s: ops.channel_absmax(X, stream=s),
    "smooth_scales": lambda s: ops.smooth_scales(V, V, with_inverse=True, stream=s),
    "sqnr": lambda s: ops.sqnr([X], [X], stream=s),
    "linear_lowrank": lambda s: ops.linear_lowrank(X, W, L1, L2, stream=s),
    "dit_block_linears": lambda s: ops.dit_block_linears(W8, ROWS8, 0x0F, stream=s),
    "sf_to_logical": lambda s: ops.sf_to_logical(XS, M, K, stream=s),
}


def parts(w):
    return w.codes, w.sf


def check(call, streams):
    side, current, lib, log = streams
    out = call(side)
    out = out if isinstance(out, (tuple, list)) else (out,)
    assert lib.streams and all(s == side.cuda_stream for s in lib.streams)
    assert log["made"]
    for t, under in log["made"]:
        assert under == [side], "allocated on another stream than the call's"
    noted = [t for t, s in log["noted"] if s is current]
    for t in out:
        assert any(t is n for n in noted), "a returned tensor is not noted on the current stream"


@pytest.mark.parametrize("name", AROUND)
def test_a_call_on_a_stream_allocates_there(name, streams):
    check(AROUND[name], streams)


@pytest.mark.parametrize("name", EARLIER)
def test_a_quantizer_or_linear_on_a_stream_allocates_there(name, streams):
    check(EARLIER[name], streams)


def test_a_split_on_a_stream_is_decomposed_there(streams, monkeypatch):
    side, current, lib, log = streams
    where = []
    svd = lambda w, full_matrices: where.append(list(log["under"])) or (w, w[0], w)  # noqa: E731
    monkeypatch.setattr(torch.linalg, "svd", svd)
    monkeypatch.setattr(ops, "lowrank_split", lambda w, U, S, Vh, rank: where.append(list(log["under"])) or (U, Vh, w))
    out = ops.svd_split(X, 4, stream=side)
    assert where == [[side], [side]]
    assert all(any(t is n and s is current for n, s in log["noted"]) for t in out)
