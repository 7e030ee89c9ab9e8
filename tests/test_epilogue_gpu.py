"""The residual and gated GEMMs (ops.gemm_residual, gemm_bf16_residual, linear_residual,
gemm_gated, gemm_bf16_gated, gated_ffn) against the formulas in float64.

Bounds.  The tensor core adds at least 16 products to the binary32 sum at a time, each
addition off by at most 2^-23 of the sums so far (truncation counted), and the few-row kernel
adds at most 8 partial sums: the sum is within (K / 16 + 16) 2^-23 sum|a w| of the exact one.
The activations' slopes stay below 1.2, and their binary32 evaluation (exp, erfc, one quotient)
is within (16 + 4 |v|) 2^-23 of the value; each further step rounds by 2^-24 of its terms and
the result by bf16's half step, 2^-8."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U32, U16, TINY = 2.0 ** -24, 2.0 ** -8, 2.0 ** -133


def _ops():
    from fp8_mixed_precision_mxq_b200 import ops
    return ops


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def deq(codes, sf, rows, K, fmt):
    """The float64 values of packed codes and tiled scales."""
    s = torch.exp2(_ops().sf_to_logical(sf, rows, K).double() - 127)
    if fmt == "e4m3":
        v = codes.reshape(-1)[: rows * K].view(torch.float8_e4m3fn).view(rows, K).double()
    else:
        t = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                         device="cuda")
        c = codes.reshape(-1)[: rows * K // 2].view(rows, K // 2)
        v = t[torch.stack((c & 15, c >> 4), -1).long()].view(rows, K)
    return (v.view(rows, K // 32, 32) * s.unsqueeze(-1)).view(rows, K)


def act64(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def product(a, w, bias):
    """(a . w^T + bias, the bound on its binary32 error) in float64."""
    K = a.shape[1]
    b = torch.zeros((), dtype=torch.float64, device="cuda") if bias is None else bias.double()
    v = a @ w.t() + b
    return v, (K / 16 + 16) * 2 ** -23 * (a.abs() @ w.abs().t()) + U32 * (v.abs() + b.abs())


def act_with_bound(v, tol, act):
    """(act(v), its error bound) of a v known to within tol."""
    r = act64(v, act)
    return r, 1.2 * tol + (0 if act == "none" else (16 + 4 * v.abs()) * 2 ** -23 * r.abs())


def assert_within(got, want, bound, what):
    bound = bound + U16 * (want.abs() + bound) + TINY
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), "%s: %d of %d elements off, worst %.3g (bound there %.3g)" % (
        what, int(bad.sum()), bad.numel(), float((got.double() - want).abs().max()),
        float(bound.flatten()[(got.double() - want).abs().flatten().argmax()]))


def check_residual(y, a, w, bias, act, residual, gate, rpg, what):
    M, N = y.shape
    v, tol = act_with_bound(*product(a, w, bias), act)
    if gate is not None:
        g = gate.double().reshape(-1, N)[torch.arange(M, device="cuda") // rpg]
        v, tol = v * g, tol * g.abs()
    want = v if residual is None else v + residual.double()
    assert_within(y, want, tol + 4 * U32 * (v.abs() + want.abs()), what)


def check_gated(h, a, wg, bg, wu, bu, act, what):
    g, tg = act_with_bound(*product(a, wg, bg), act)
    u, tu = product(a, wu, bu)
    assert_within(h, g * u, tg * u.abs() + tu * g.abs() + tg * tu + 2 * U32 * (g * u).abs(), what)


def operand(g, M, K, fmt):
    """(operand arguments, float64 values) of an activation."""
    ops = _ops()
    x = normal(g, M, K)
    x[:, ::37] *= 20
    c, s = ops.quantize_act(x, fmt)
    return (c, s, fmt, M, K), deq(c, s, M, K, fmt)


def weight(g, N, K, bias=True, std=0.05):
    ops = _ops()
    q = ops.quantize_weight(normal(g, N, K, std=std), bias=normal(g, N, std=0.5) if bias else None)
    return q, deq(q.codes, q.sf, N, K, "e2m1")


def on_few_rows(M, N, fmt, gated=False):
    """The library's choice of kernel: few rows, or an output of at most an SM count of tiles (W4A8:
    two)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return M <= 64 or -(-M // 64) * -(-N // 128) * (2 if gated else 1) <= sms * (2 if fmt == "e4m3" else 1)


# The few-row kernel's widths and both sides of its borders (16, 32 and 64 tokens; several token
# tiles), and the pair kernel, ragged in every direction
RESIDUAL = [  # M, N, K, fmt, act, bias, residual, gate groups, gate dtype
    (1, 8, 32, "e2m1", "none", False, False, 0, None),
    (1, 5120, 5120, "e2m1", "none", True, True, 1, torch.float32),
    (1, 136, 128, "e4m3", "gelu", True, True, 0, None),
    (2, 264, 13824, "e4m3", "silu", False, True, 2, torch.bfloat16),
    (16, 1000, 1056, "e2m1", "gelu_tanh", True, True, 3, torch.float32),
    (17, 640, 1024, "e4m3", "none", True, True, 1, torch.bfloat16),
    (33, 72, 544, "e2m1", "gelu", False, True, 5, torch.float32),
    (64, 4104, 2048, "e2m1", "silu", True, False, 1, torch.float32),
    (64, 512, 5120, "e4m3", "gelu", True, True, 64, torch.float32),
    (65, 256, 512, "e2m1", "none", True, True, 1, torch.float32),
    (130, 520, 5120, "e2m1", "gelu", True, True, 3, torch.bfloat16),
    (200, 2056, 1024, "e4m3", "silu", True, True, 2, torch.float32),
    (1000, 264, 544, "e2m1", "none", True, True, 7, torch.float32),
    (65, 9608, 32, "e2m1", "none", False, True, 0, None),
    (129, 6408, 256, "e4m3", "gelu", True, True, 3, torch.bfloat16),   # groups that end inside a warp's rows
    (129, 12808, 256, "e4m3", "gelu", True, True, 3, torch.bfloat16),   # groups that end inside a warp's rows
    (300, 4104, 1024, "e2m1", "gelu_tanh", True, False, 0, None),
    (513, 2200, 2048, "e4m3", "silu", True, True, 513, torch.float32),  # a group for each row
    (700, 4104, 384, "e4m3", "silu", True, True, 513, torch.float32),  # a group for each row
    (1000, 5120, 1280, "e2m1", "none", True, True, 2, torch.float32),
]


@pytest.mark.parametrize("M,N,K,fmt,act,bias,residual,groups,gdt", RESIDUAL)
def test_gemm_residual_against_float64(M, N, K, fmt, act, bias, residual, groups, gdt):
    ops = _ops()
    g = gen(M + 3 * N + K)
    a, a64 = operand(g, M, K, fmt)
    w, w64 = weight(g, N, K, bias)
    r = normal(g, M, N, std=2.0) if residual else None
    gate = normal(g, groups, N, dtype=gdt) if groups else None
    rpg = -(-M // max(1, groups))
    y = ops.gemm_residual(*a, w, act=act, residual=r, gate=gate, rows_per_group=rpg)
    assert ops.poll_status() == 0
    assert ops.last_path().startswith("rows") == on_few_rows(M, N, fmt) and "+act+residual" in ops.last_path()
    check_residual(y, a64, w64, w.bias, act, r, gate, rpg, "M=%d N=%d K=%d %s %s" % (M, N, K, fmt, act))
    # in place of the residual: the same bits
    if residual:
        y2 = ops.gemm_residual(*a, w, act=act, residual=r, gate=gate, rows_per_group=rpg, out=r)
        assert y2 is r and torch.equal(y2, y)


@pytest.mark.parametrize("M,N,K,act,groups", [
    (1, 8, 8, "none", 1), (5, 136, 72, "gelu", 2), (16, 5120, 4096, "none", 0), (40, 264, 1000, "silu", 1),
    (64, 128, 64, "gelu_tanh", 1), (65, 520, 136, "gelu_tanh", 0), (170, 1032, 264, "gelu", 4),
    (512, 5120, 4096, "gelu_tanh", 0), (300, 4104, 2056, "silu", 7), (129, 6424, 136, "gelu", 0),
])
def test_gemm_bf16_residual_against_float64(M, N, K, act, groups):
    ops = _ops()
    g = gen(M + N + K)
    a, b = normal(g, M, K), normal(g, N, K, std=0.05)
    bias, r = normal(g, N), normal(g, M, N)
    gate = normal(g, groups, N, dtype=torch.float32) if groups else None
    rpg = -(-M // max(1, groups))
    y = ops.gemm_bf16_residual(a, b, bias=bias, act=act, residual=r, gate=gate, rows_per_group=rpg)
    assert ops.poll_status() == 0
    check_residual(y, a.double(), b.double(), bias, act, r, gate, rpg, "bf16 M=%d N=%d K=%d" % (M, N, K))


def test_plain_epilogue_is_the_plain_gemm():
    """Without activation, gate and residual the pair kernel's result is mxq_gemm's, bit for bit."""
    ops = _ops()
    g = gen(1)
    for fmt in ("e2m1", "e4m3"):
        a, _ = operand(g, 300, 1024, fmt)
        w, _ = weight(g, 4104, 1024)
        assert torch.equal(ops.gemm_residual(*a, w), ops.gemm(*a, w))


@pytest.mark.parametrize("M", [1, 48, 200])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_linear_residual_is_quantize_then_gemm(M, fmt):
    ops = _ops()
    g = gen(M)
    x, r, gate = normal(g, M, 640), normal(g, M, 384), normal(g, 384, dtype=torch.float32)
    w, _ = weight(g, 384, 640)
    c, s = ops.quantize_act(x, fmt)
    want = ops.gemm_residual(c, s, fmt, M, 640, w, act="gelu", residual=r, gate=gate)
    ws = torch.full((ops.workspace_bytes(M, 384, 640, fmt),), 0xA5, dtype=torch.uint8, device="cuda")
    assert torch.equal(ops.linear_residual(x, w, fmt, act="gelu", residual=r, gate=gate), want)
    assert torch.equal(ops.linear_residual(x, w, fmt, act="gelu", residual=r, gate=gate, workspace=ws), want)


GATED = [  # M, H, K, fmt, act, bias
    (1, 8, 32, "e2m1", "silu", False),
    (1, 13824, 5120, "e2m1", "silu", True),
    (1, 32, 128, "e4m3", "gelu", True),
    (16, 1056, 544, "e2m1", "gelu_tanh", False),
    (31, 160, 13824, "e4m3", "silu", True),
    (33, 544, 1024, "e2m1", "none", True),
    (64, 2080, 1280, "e4m3", "silu", True),
    (65, 128, 256, "e2m1", "silu", False),
    (100, 8, 32, "e2m1", "gelu", True),
    (200, 1056, 512, "e4m3", "gelu_tanh", True),   # token tiles that share a scale atom
    (65, 4768, 544, "e2m1", "gelu", True),
    (300, 2080, 32, "e2m1", "gelu", True),
    (257, 2088, 512, "e4m3", "gelu_tanh", True),
    (300, 4104, 384, "e4m3", "gelu_tanh", True),
    (777, 5632, 2048, "e4m3", "silu", True),
]


@pytest.mark.parametrize("M,H,K,fmt,act,bias", GATED)
def test_gemm_gated_against_float64(M, H, K, fmt, act, bias):
    ops = _ops()
    g = gen(M + H + K)
    a, a64 = operand(g, M, K, fmt)
    (wg, g64), (wu, u64) = weight(g, H, K, bias), weight(g, H, K, bias)
    h = ops.gemm_gated(*a, wg, wu, act=act)
    assert ops.poll_status() == 0 and "+gated->bf16" in ops.last_path()
    assert ops.last_path().startswith("rows") == on_few_rows(M, H, fmt, gated=True)
    check_gated(h, a64, g64, wg.bias, u64, wu.bias, act, "M=%d H=%d K=%d %s %s" % (M, H, K, fmt, act))
    if H % 32 == 0:
        for of in ("e2m1", "e4m3"):  # the bits of the activation quantizer, padding included
            dirty = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
                     for n in (ops.codes_bytes(M, H, of), ops.sf_bytes(M, H))]
            codes, sf = ops.gemm_gated(*a, wg, wu, act=act, out_fmt=of, codes=dirty[0], sf=dirty[1])
            want_c, want_s = ops.quantize_act(h, of)
            assert torch.equal(codes, want_c) and torch.equal(sf, want_s), of
    assert ops.poll_status() == 0


@pytest.mark.parametrize("M,H,K", [(1, 8, 8), (3, 160, 72), (50, 544, 1000), (64, 128, 2048), (70, 264, 136),
                                   (150, 544, 512), (300, 2080, 512)])
def test_gemm_bf16_gated_against_float64(M, H, K):
    ops = _ops()
    g = gen(M + H + K)
    a, wg, wu = normal(g, M, K), normal(g, H, K, std=0.05), normal(g, H, K, std=0.05)
    bg, bu = normal(g, H), normal(g, H)
    h = ops.gemm_bf16_gated(a, wg, wu, bg, bu)
    assert ops.poll_status() == 0
    check_gated(h, a.double(), wg.double(), bg, wu.double(), bu, "silu", "bf16 gated M=%d H=%d K=%d" % (M, H, K))
    if H % 32 == 0:
        for of in ("e2m1", "e4m3"):
            codes, sf = ops.gemm_bf16_gated(a, wg, wu, bg, bu, out_fmt=of)
            want_c, want_s = ops.quantize_act(h, of)
            assert torch.equal(codes, want_c) and torch.equal(sf, want_s), of


@pytest.mark.parametrize("M", [1, 20, 64, 65, 333, 2100])
@pytest.mark.parametrize("up_fmt,down_fmt", [("e2m1", "e4m3"), ("e4m3", "e2m1")])
def test_gated_ffn_is_its_steps(M, up_fmt, down_fmt):
    ops = _ops()
    g = gen(M)
    K, H = 640, 3200
    x, r, gate = normal(g, M, K), normal(g, M, K), normal(g, 1, K, dtype=torch.float32)
    (wg, _), (wu, _), (wd, d64) = weight(g, H, K), weight(g, H, K), weight(g, K, H)
    c, s = ops.quantize_act(x, up_fmt)
    hc, hs = ops.gemm_gated(c, s, up_fmt, M, K, wg, wu, out_fmt=down_fmt)
    want = ops.gemm_residual(hc, hs, down_fmt, M, H, wd, residual=r, gate=gate)
    y = ops.gated_ffn(x, wg, wu, wd, up_fmt=up_fmt, down_fmt=down_fmt, residual=r, out_gate=gate)
    assert torch.equal(y, want) and ops.poll_status() == 0
    check_residual(y, deq(hc, hs, M, H, down_fmt), d64, wd.bias, "none", r, gate, M, "gated ffn M=%d" % M)


@pytest.mark.parametrize("M", [1, 65, 1500])
def test_block_norm_gated_ffn_residual(M):
    """The operators as a block uses them: the fused norm writes the operand, the gated GEMM
    the hidden operand, and the last linear adds its gated result to the stream, in place."""
    ops = _ops()
    g = gen(M + 5)
    K, H = 1280, 2304
    x, y = normal(g, M, K), normal(g, M, K)
    mods = {k: normal(g, 1, K, std=0.5, dtype=torch.float32) for k in ("gate", "scale", "shift")}
    gate2 = normal(g, 1, K, dtype=torch.float32)
    (wg, _), (wu, _), (wd, _) = weight(g, H, K), weight(g, H, K), weight(g, K, H)
    z, c, s = ops.norm_residual(x, y, out_fmt="e4m3", **mods)
    hc, hs = ops.gemm_gated(c, s, "e4m3", M, K, wg, wu, out_fmt="e2m1")
    out = ops.gemm_residual(hc, hs, "e2m1", M, H, wd, residual=z, gate=gate2, out=z)
    z1, h1 = ops.norm_residual(x, y, **mods)
    want = ops.gated_ffn(h1, wg, wu, wd, up_fmt="e4m3", down_fmt="e2m1", residual=z1, out_gate=gate2)
    assert out is z and torch.equal(out, want) and ops.poll_status() == 0


@pytest.mark.parametrize("M", [3, 200, 9700])
def test_nonfinite_rows_stay_in_their_rows(M):
    """A NaN in one row's input makes that row NaN (E8M0 code 255) and no other."""
    ops = _ops()
    g = gen(9)
    x, r = normal(g, M, 256), normal(g, M, 128)
    w, _ = weight(g, 128, 256)
    clean = ops.linear_residual(x, w, act="silu", residual=r)
    x[1, 3] = float("nan")
    y = ops.linear_residual(x, w, act="silu", residual=r)
    keep = [i for i in range(M) if i != 1]
    assert y[1].isnan().all() and torch.equal(y[keep], clean[keep])
    wu, _ = weight(g, 128, 256)
    c, s = ops.quantize_act(x, "e2m1")
    codes, sf = ops.gemm_gated(c, s, "e2m1", M, 256, w, wu, out_fmt="e4m3")
    logical = ops.sf_to_logical(sf, M, 128)
    assert (logical[1] == 255).all() and (logical[keep] != 255).all()
    assert (codes.view(M, 128)[1] == 0).all()


def test_large_sums_reach_infinity_and_saturated_activations():
    """Sums far out in both tails: silu and both GELUs give v for large v and a (signed) zero
    for far negative v, no NaN."""
    ops = _ops()
    for M in (4, 100, 9700):
        x = torch.full((M, 64), 30.0, device="cuda").bfloat16()
        w = torch.ones((16, 64), device="cuda").bfloat16()
        w[8:] = -1
        for act in ("silu", "gelu", "gelu_tanh"):
            y = ops.gemm_bf16_residual(x, w, act=act).float()
            assert (y[:, :8] == 1920).all() and (y[:, 8:] == 0).all(), act


@pytest.mark.parametrize("M", [8, 300, 3000])
def test_captured_replayed_and_on_two_streams(M):
    ops = _ops()
    g = gen(M)
    K, H = 512, 768
    (wg, _), (wu, _), (wd, _) = weight(g, H, K), weight(g, H, K), weight(g, K, H)
    x, r = normal(g, M, K), normal(g, M, K)
    y = torch.empty_like(x)
    ops.gated_ffn(x, wg, wu, wd, residual=r, out=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.gated_ffn(x, wg, wu, wd, residual=r, out=y)
    x1, r1 = normal(g, M, K), normal(g, M, K)
    x.copy_(x1)
    r.copy_(r1)
    graph.replay()
    want = ops.gated_ffn(x1, wg, wu, wd, residual=r1)
    assert torch.equal(y, want)
    # two calls at once, each with its own workspace
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(ops.gated_ffn(x1, wg, wu, wd, residual=r1))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and ops.poll_status() == 0


@pytest.mark.parametrize("M", [1, 16, 64, 300])
def test_gated_ffn_adds_onto_its_own_input(M):
    """The residual stream updated in place: x is the input, the residual and the output."""
    ops = _ops()
    g = gen(M + 7)
    K, H = 512, 768
    (wg, _), (wu, _), (wd, _) = weight(g, H, K), weight(g, H, K), weight(g, K, H)
    x = normal(g, M, K)
    want = ops.gated_ffn(x, wg, wu, wd, residual=x)
    assert ops.gated_ffn(x, wg, wu, wd, residual=x, out=x) is x
    assert torch.equal(x, want) and ops.poll_status() == 0


@pytest.mark.parametrize("M", [1, 48, 200])
def test_operands_written_right_before_the_call(M):
    """Kernels that start while the one before them ends see what the stream wrote before the call:
    x, the weights and the residual change between calls that follow each other at once."""
    ops = _ops()
    g = gen(M + 11)
    K, H = 1024, 768
    sets = [[weight(g, H, K)[0], weight(g, H, K)[0], weight(g, K, H)[0], weight(g, K, K)[0], normal(g, M, K),
             normal(g, M, K)] for _ in range(2)]
    want = [(ops.linear_residual(s[4], s[3], "e4m3", residual=s[5]), ops.gated_ffn(s[4], *s[:3], residual=s[5]))
            for s in sets]
    cur = [ops.QWeight(w.codes.clone(), w.sf.clone(), w.N, w.K, w.bias.clone()) for w in sets[0][:4]]
    x, r = sets[0][4].clone(), sets[0][5].clone()
    got = []
    for i in range(12):
        s = sets[i % 2]
        for c, w in zip(cur, s[:4]):
            c.codes.copy_(w.codes)
            c.sf.copy_(w.sf)
            c.bias.copy_(w.bias)
        x.copy_(s[4])
        r.copy_(s[5])
        y = ops.linear_residual(x, cur[3], "e4m3", residual=r)
        got.append((y, ops.gated_ffn(x, *cur[:3], residual=r)))
    assert ops.poll_status() == 0
    for i, (y, f) in enumerate(got):
        assert torch.equal(y, want[i % 2][0]) and torch.equal(f, want[i % 2][1]), i


@pytest.mark.parametrize("M", [64, 300])
def test_a_call_on_another_stream_keeps_its_workspace(M):
    """The workspace that a call allocates belongs to the stream it runs on: what the current stream
    allocates and writes right behind it is other memory."""
    ops = _ops()
    g = gen(M + 9)
    K, H = 512, 768
    (wg, _), (wu, _), (wd, _) = weight(g, H, K), weight(g, H, K), weight(g, K, H)
    w, x = weight(g, H, K)[0], normal(g, M, K)
    want_y, want_f = ops.linear_residual(x, w), ops.gated_ffn(x, wg, wu, wd)
    s = torch.cuda.Stream()
    y, f = torch.empty_like(want_y), torch.empty_like(want_f)
    torch.cuda.synchronize()
    sizes = (ops.workspace_bytes(M, H, K, "e2m1"), ops.ffn_workspace_bytes(M, K, H, "e2m1", "e2m1"))
    for _ in range(20):
        ops.linear_residual(x, w, out=y, stream=s)
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes]
        ops.gated_ffn(x, wg, wu, wd, out=f, stream=s)
        junk += [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes]
        del junk
    torch.cuda.synchronize()
    assert torch.equal(y, want_y) and torch.equal(f, want_f) and ops.poll_status() == 0


def test_more_outputs_than_two_grid_dimensions_hold():
    """One token over 65536 weight tiles of 128 outputs."""
    ops = _ops()
    g = gen(3)
    N, K = 65536 * 128 + 8, 32
    block = torch.randn((128, K), generator=g, device="cuda").bfloat16()
    w = block.repeat(65537, 1)[:N].contiguous()
    x = torch.randn((1, K), generator=g, device="cuda").bfloat16()
    y = ops.gemm_bf16_residual(x, w, act="silu")
    want = ops.gemm_bf16_residual(x, block, act="silu")
    assert torch.equal(y, want.repeat(1, 65537)[:, :N]) and ops.poll_status() == 0


@pytest.mark.parametrize("M", [8, 300, 5000])
def test_a_wait_that_runs_out_is_reported(M):
    """Debug bit 0: a stage is never filled; the kernel's wait ends after its limit, the status
    says so, and the next call is right again."""
    from fp8_mixed_precision_mxq_b200 import _lib
    ops = _ops()
    g = gen(M)
    a, a64 = operand(g, M, 512, "e2m1")
    w, w64 = weight(g, 256, 512)
    ops.set_debug(1)
    try:
        ops.gemm_residual(*a, w)
        assert ops.poll_status() == _lib.ERR_TIMEOUT
    finally:
        ops.set_debug(0)
    y = ops.gemm_residual(*a, w)
    assert ops.poll_status() == 0
    check_residual(y, a64, w64, w.bias, "none", None, None, M, "after the time-out")
