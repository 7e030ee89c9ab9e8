"""The fused norms around a block (ops.norm_residual) against the formulas in float64.

Bounds.  u = 2^-24 is binary32's half step, 2^-8 bf16's.  A row sum of K <= 32768 terms is
at most 64 additions in a thread, 5 in a warp and 5 over the warps, so its error is below
80 u sum|v|; the mean is off by at most 80 u mean|v| and 1/sqrt(mean square + eps) by half of
its mean square's relative error (below 90 u) plus its own roundings.  A normalized value n is
therefore off by at most NORM_ULPS u (|n| + mean|v| / std) with NORM_ULPS = 128; the few
elementwise steps after it add at most 4 u of each term; the final rounding adds its half step."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -133
NORM_ULPS = 128


def _ops():
    from fp8_mixed_precision_mxq_b200 import ops
    return ops


def ref_norm(v, kind, w, b, eps):
    """(norm(v) * w + b, its error bound) in float64."""
    if kind == "none":
        return v, torch.zeros_like(v)
    d = v - v.mean(-1, keepdim=True) if kind == "layer" else v
    rstd = (d.square().mean(-1, keepdim=True) + eps).rsqrt()
    n = d * rstd
    off = v.abs().mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(rstd)
    # the mean's own error also shifts the centered squares: (80 u mean|v|)^2 / var, second order
    tol = NORM_ULPS * U32 * (n.abs() + off * rstd)
    w = torch.ones_like(v[0]) if w is None else w.double()
    b = torch.zeros_like(v[0]) if b is None else b.double()
    return n * w + b, tol * w.abs() + 4 * U32 * ((n * w).abs() + b.abs())


def per_row(v, rows, rpg, default, K, device):
    if v is None:
        return torch.full((rows, K), default, dtype=torch.float64, device=device)
    return v.double().reshape(-1, K)[torch.arange(rows, device=device) // rpg]


def check(x, y, z, h, norm, post, vecs, rpg, eps=1e-6):
    """z against the formula, and h against the formula on the z that was stored."""
    rows, K = x.shape
    if y is not None:
        u, tol = ref_norm(y.double(), post, vecs.get("post_weight"), vecs.get("post_bias"), eps)
        g = per_row(vecs.get("gate"), rows, rpg, 1.0, K, x.device)
        want = x.double() + g * u
        step = U32 if x.dtype == torch.float32 else U16
        bound = g.abs() * tol + 4 * U32 * (x.double().abs() + (g * u).abs())
        bound = bound + step * (want.abs() + bound) + TINY
        bad = (z.double() - want).abs() > bound
        assert not bad.any(), "z: %d elements off, worst %.3g" % (int(bad.sum()), float((z.double() - want).abs().max()))
    n, tol = ref_norm(z.double(), norm, vecs.get("weight"), vecs.get("bias"), eps)
    s = 1 + per_row(vecs.get("scale"), rows, rpg, 0.0, K, x.device)
    t = per_row(vecs.get("shift"), rows, rpg, 0.0, K, x.device)
    want = n * s + t
    bound = tol * s.abs() + 4 * U32 * ((n * s).abs() + n.abs() + t.abs())
    bound = bound + U16 * (want.abs() + bound) + TINY
    bad = (h.double() - want).abs() > bound
    assert not bad.any(), "h: %d elements off, worst %.3g" % (int(bad.sum()), float((h.double() - want).abs().max()))


def make(rows, K, seed, stream=torch.bfloat16, vec=torch.float32, groups=1, norm="layer", post="none", affine=False,
         mod=True, offset=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (rnd(rows, K) * 2 + offset).to(stream)
    y = (rnd(rows, K) + offset / 2).to(torch.bfloat16)
    vecs = {}
    if affine:
        vecs["weight"], vecs["bias"] = (1 + 0.3 * rnd(K)).to(vec), (0.3 * rnd(K)).to(vec)
    if post != "none":
        vecs["post_weight"], vecs["post_bias"] = (1 + 0.3 * rnd(K)).to(vec), (0.3 * rnd(K)).to(vec)
    if mod:
        for k in ("gate", "scale", "shift"):
            vecs[k] = (0.5 * rnd(groups, K)).to(vec)
    return x, y, vecs


CASES = [  # rows, K, stream, vec, groups, norm, post, affine, mod
    (1, 8, torch.bfloat16, torch.float32, 1, "layer", "none", False, True),      # one chunk of one row
    (1, 5120, torch.bfloat16, torch.bfloat16, 1, "rms", "none", True, False),    # one token
    (3, 40, torch.float32, torch.float32, 3, "rms", "layer", True, True),        # one row per group
    (37, 1056, torch.bfloat16, torch.bfloat16, 2, "layer", "rms", True, True),   # ragged last group
    (129, 4096, torch.float32, torch.bfloat16, 1, "layer", "layer", False, True),
    (300, 5120, torch.bfloat16, torch.float32, 2, "layer", "none", False, True),  # four chunks a thread
    (300, 5120, torch.float32, torch.float32, 1, "rms", "rms", True, False),
    (513, 96, torch.bfloat16, torch.float32, 5, "layer", "none", True, True),
    (5, 16384, torch.bfloat16, torch.float32, 1, "rms", "rms", True, True),
    (4, 32768, torch.float32, torch.float32, 1, "layer", "layer", True, True),   # the longest row
    (311, 32736, torch.bfloat16, torch.bfloat16, 2, "layer", "rms", True, True),
]


@pytest.mark.parametrize("rows,K,stream,vec,groups,norm,post,affine,mod", CASES)
def test_norm_residual_against_float64(rows, K, stream, vec, groups, norm, post, affine, mod):
    ops = _ops()
    x, y, vecs = make(rows, K, rows + K, stream, vec, groups, norm, post, affine, mod)
    rpg = -(-rows // groups)
    x0, y0 = x.clone(), y.clone()
    z, h = ops.norm_residual(x, y, norm=norm, post_norm=post, rows_per_group=rpg, **vecs)
    assert z.dtype == stream and h.dtype == torch.bfloat16
    assert torch.equal(x, x0) and torch.equal(y, y0)
    check(x, y, z, h, norm, post, vecs, rpg)
    if K % 32 == 0:
        for fmt in ("e2m1", "e4m3"):  # the bits of the activation quantizer, padding included
            zq, codes, sf = ops.norm_residual(x, y, norm=norm, post_norm=post, rows_per_group=rpg, out_fmt=fmt,
                                              codes=torch.full((ops.codes_bytes(rows, K, fmt),), 0xA5,
                                                               dtype=torch.uint8, device="cuda"),
                                              sf=torch.full((ops.sf_bytes(rows, K),), 0xA5, dtype=torch.uint8,
                                                            device="cuda"), **vecs)
            want_c, want_s = ops.quantize_act(h, fmt)
            assert torch.equal(zq, z) and torch.equal(codes, want_c) and torch.equal(sf, want_s)
    assert ops.poll_status() == 0


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_without_a_block_output_x_is_the_stream(norm):
    ops = _ops()
    x, _, vecs = make(70, 320, 1)
    del vecs["gate"]
    z, h = ops.norm_residual(x, norm=norm, **vecs)
    assert z is x
    check(x, None, x, h, norm, "none", vecs, 70)


def test_large_common_offset_keeps_its_digits():
    """Rows of mean 1000 and deviation 2 on an fp32 stream: two passes lose nothing of the
    deviations beyond the bound."""
    ops = _ops()
    x, y, vecs = make(200, 5120, 2, torch.float32, offset=1000.0)
    z, h = ops.norm_residual(x, y, **vecs)
    check(x, y, z, h, "layer", "none", vecs, 200)


def test_constant_zero_and_nonfinite_rows():
    """A zero row and a constant row normalize to zero (eps > 0), so h is the shift; a NaN or
    Inf reaches its own row's h and no other row."""
    ops = _ops()
    x, _, _ = make(6, 512, 3)
    x[0] = 0
    x[1] = 7.5
    x[3, 5] = float("nan")
    x[4, 100] = float("inf")
    shift = torch.randn(512, device="cuda")
    _, h = ops.norm_residual(x, norm="layer", shift=shift)
    assert torch.equal(h[0], shift.bfloat16()) and torch.equal(h[1], shift.bfloat16())
    assert h[3].isnan().all() and h[4].isnan().all()
    check(x[[2, 5]], None, x[[2, 5]], h[[2, 5]], "layer", "none", {"shift": shift}, 2)
    _, r = ops.norm_residual(x, norm="rms")
    assert torch.equal(r[0], torch.zeros_like(r[0])) and r[3].isnan().all()
    _, codes, sf = ops.norm_residual(x, norm="layer", shift=shift, out_fmt="e2m1")
    s = ops.sf_to_logical(sf, 6, 512)
    assert (s[3] == 255).all() and (s[4] == 255).all() and (s[[0, 1, 2, 5]] != 255).all()
    assert (codes.view(6, 256)[3] == 0).all()


def test_in_place_stream_and_given_buffers():
    """z may be x; given buffers receive the results; a call on a side stream follows that
    stream's earlier work."""
    ops = _ops()
    x, y, vecs = make(333, 2048, 4)
    z, h = ops.norm_residual(x, y, **vecs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x2 = x.clone()
        h2 = torch.empty_like(h)
        z2, h3 = ops.norm_residual(x2, y, z=x2, h=h2, **vecs)
    torch.cuda.current_stream().wait_stream(s)
    assert z2 is x2 and h3 is h2 and torch.equal(x2, z) and torch.equal(h2, h)


def test_captured_and_replayed():
    ops = _ops()
    x, y, vecs = make(64, 1024, 5)
    z, h = torch.empty_like(x), torch.empty_like(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.norm_residual(x, y, z=z, h=h, **vecs)
    for seed in (6, 7):
        x1, y1, _ = make(64, 1024, seed)
        x.copy_(x1)
        y.copy_(y1)
        g.replay()
        zr, hr = ops.norm_residual(x1, y1, **vecs)
        assert torch.equal(z, zr) and torch.equal(h, hr)


def test_offsets_past_32_bits():
    """A stream of more than 2^32 bytes: the last rows are computed from their own data."""
    ops = _ops()
    rows, K = 70000, 32768  # 4.6e9 bytes of bf16, 2.3e9 elements
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(8))
    _, h = ops.norm_residual(x, norm="rms")
    check(x[-3:], None, x[-3:], h[-3:], "rms", "none", {}, 3)
    _, codes, sf = ops.norm_residual(x, norm="rms", out_fmt="e4m3", h=None)
    want, ws = ops.quantize_act(h[-(rows % 128):].contiguous(), "e4m3")
    assert torch.equal(codes[(rows - rows % 128) * K: rows * K], want[: (rows % 128) * K])
    assert torch.equal(sf[-ws.numel():], ws)
