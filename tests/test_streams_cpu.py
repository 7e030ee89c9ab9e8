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
