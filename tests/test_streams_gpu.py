"""Calls that are given a stream, run while the current stream is busy: outputs that they allocate
are not memory that the current stream still reads or hands out again."""
import pytest
import torch

pytestmark = pytest.mark.gpu

M, K, H = 1000, 1024, 2048


def _ops():
    from fp8_mixed_precision_mxq_b200 import ops
    return ops


def around():
    """The operators between a block's linears, each as a function of its stream."""
    ops = _ops()
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, y = rnd(M, K), rnd(M, K)
    c, s = ops.quantize_act(x, "e4m3")
    wg, wu, wd = ops.quantize_weight(rnd(H, K)), ops.quantize_weight(rnd(H, K)), ops.quantize_weight(rnd(K, H))
    bg, bu = rnd(H, K), rnd(H, K)
    return {
        "norm": lambda st: ops.norm_residual(x, y, stream=st),
        "norm e4m3": lambda st: ops.norm_residual(x, y, out_fmt="e4m3", stream=st),
        "gemm": lambda st: ops.gemm_residual(c, s, "e4m3", M, K, wg, stream=st),
        "gemm bf16": lambda st: ops.gemm_bf16_residual(x, bg, stream=st),
        "linear": lambda st: ops.linear_residual(x, wg, stream=st),
        "gated": lambda st: ops.gemm_gated(c, s, "e4m3", M, K, wg, wu, stream=st),
        "gated e2m1": lambda st: ops.gemm_gated(c, s, "e4m3", M, K, wg, wu, out_fmt="e2m1", stream=st),
        "gated bf16": lambda st: ops.gemm_bf16_gated(x, bg, bu, stream=st),
        "ffn": lambda st: ops.gated_ffn(x, wg, wu, wd, stream=st),
    }


NAMES = ("norm", "norm e4m3", "gemm", "gemm bf16", "linear", "gated", "gated e2m1", "gated bf16", "ffn")


def tensors(out):
    return list(out) if isinstance(out, (tuple, list)) else [out]


def check(call):
    want = [t.clone() for t in tensors(call(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        # blocks of the outputs' sizes, freed while the current stream has yet to read them
        old = [torch.full((t.nbytes,), 0x3C, dtype=torch.uint8, device="cuda") for t in want]
        room = [torch.empty_like(o) for o in old]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        for o, r in zip(old, room):
            r.copy_(o)
        del o, old
        got = tensors(call(side))
        # what the current stream allocates and writes behind the call is other memory too
        junk = [torch.full((t.nbytes,), 0xFF, dtype=torch.uint8, device="cuda") for t in want]
        torch.cuda.synchronize()
        for r in room:
            assert (r == 0x3C).all(), "the call wrote what the current stream still had to read"
        for t, w in zip(got, want):
            assert torch.equal(t, w)
        del got, junk, room


@pytest.mark.parametrize("name", NAMES)
def test_outputs_on_another_stream(name):
    check(around()[name])
    assert _ops().poll_status() == 0


def test_a_chain_on_another_stream_keeps_its_intermediates():
    """Codes and scales that go out of scope while the stream still reads them."""
    ops = _ops()
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, y = rnd(M, K), rnd(M, K)
    wg, wu, wd = ops.quantize_weight(rnd(H, K)), ops.quantize_weight(rnd(H, K)), ops.quantize_weight(rnd(K, H))

    def chain(st):
        z, c, s = ops.norm_residual(x, y, out_fmt="e4m3", stream=st)
        c, s = ops.gemm_gated(c, s, "e4m3", M, K, wg, wu, out_fmt="e2m1", stream=st)
        return ops.gemm_residual(c, s, "e2m1", M, H, wd, residual=z, stream=st)

    want = chain(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = {n for f in ("e4m3", "e2m1") for w in (K, H) for n in ops._mx_bytes(M, w, ops._fmt(f))} | {M * K * 2}
    for _ in range(5):
        with torch.cuda.stream(side):
            torch.cuda._sleep(5_000_000)
        got = chain(side)
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del got, junk
    assert ops.poll_status() == 0


def earlier():
    """Quantizers and linears, each as a function of its stream."""
    ops = _ops()
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x = rnd(M, K)
    c, s = ops.quantize_act(x, "e4m3")
    w, wd = ops.quantize_weight(rnd(H, K)), ops.quantize_weight(rnd(K, H))
    l1, l2 = rnd(64, K), rnd(H, 64)
    return {
        "quantize": lambda st: ops.quantize_act(x, stream=st),
        "dequantize": lambda st: ops.dequantize(c, s, M, K, "e4m3", stream=st),
        "gemm": lambda st: ops.gemm(c, s, "e4m3", M, K, w, stream=st),
        "linear": lambda st: ops.linear(x, w, stream=st),
        "linear qdq": lambda st: ops.linear(x, w, mode="qdq", stream=st),
        "ffn": lambda st: ops.ffn(x, w, wd, stream=st),
        "lowrank": lambda st: ops.linear_lowrank(x, w, l1, l2, stream=st),
        "transformed": lambda st: ops.linear_transformed(x, w, stream=st),
    }


@pytest.mark.parametrize("name", ("quantize", "dequantize", "gemm", "linear", "linear qdq", "ffn", "lowrank",
                                  "transformed"))
def test_quantizers_and_linears_on_another_stream(name):
    check(earlier()[name])
    assert _ops().poll_status() == 0


def test_split_on_another_stream():
    ops = _ops()
    w = torch.randn(96, 128, device="cuda").bfloat16()
    want = ops.svd_split(w, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.svd_split(w, 8, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_on_a_forked_stream():
    """Calls given a stream that joins a capture: their memory is the graph's, and replays repeat."""
    ops = _ops()
    g = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, y = rnd(M, K), rnd(M, K)
    wg, wu, wd = ops.quantize_weight(rnd(H, K)), ops.quantize_weight(rnd(H, K)), ops.quantize_weight(rnd(K, H))
    x1, y1 = rnd(M, K), rnd(M, K)

    def block(a, b, st):
        z, h = ops.norm_residual(a, b, stream=st)
        return ops.gated_ffn(h, wg, wu, wd, residual=z, stream=st)

    want = [block(x, y, None), block(x1, y1, None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = block(x, y, side)
        torch.cuda.current_stream().wait_stream(side)
        out.copy_(got)
        del got
    for a, b, w in ((x1, y1, want[1]), (x.clone(), y.clone(), want[0]), (x1, y1, want[1])):
        x.copy_(a)
        y.copy_(b)
        graph.replay()
        junk = [torch.full((M, K), 9.0, device="cuda").bfloat16() for _ in range(4)]
        assert torch.equal(out, w)
        del junk
    assert ops.poll_status() == 0
