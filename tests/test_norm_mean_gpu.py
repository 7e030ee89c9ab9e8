"""LayerNorm of rows far from zero (ops.norm_residual): the mean's error must not be blown up by
1 / sqrt(variance + eps).

Bounds.  A constant row's mean is that value (for a bf16 row the sum is exact, K values of eight
bits, and its division is rounded once; for an fp32 row the mean of the centered values, small
multiples of one ulp, is exact), so the centered values are zeros and h is the shift, exactly.  For
an fp32 row of any mean, the mean of the centered values d is off by at most 80 u mean|d| <= 80 u
std (u = 2^-24: 64 additions in a thread, 5 in a warp, 5 over the warps, the division), v - mean
is exact within a binade, 1/sqrt of the variance off by 90 u / 2 and the product by 2 u: n is
within 128 u (1 + |n|) of the formula's, and bf16's half step is 2^-8 |n|."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
WIDTHS = [896, 1792, 2816, 3584, 5120, 7168, 10752, 28672]  # 1 / K is rounded at each


def _ops():
    from fp8_mixed_precision_mxq_b200 import ops
    return ops


@pytest.mark.parametrize("rows", [2, 301])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", WIDTHS)
def test_constant_rows_normalize_to_zero(K, stream, rows):
    ops = _ops()
    value = torch.tensor([896.0, 1.75, -0.3, 896.123, 1e-3, -65000.0], device="cuda").to(stream)
    x = value[torch.arange(rows, device="cuda") % 6].unsqueeze(1).expand(rows, K).contiguous()
    shift = torch.randn(K, device="cuda")
    _, h = ops.norm_residual(x, norm="layer")
    assert torch.equal(h, torch.zeros_like(h))
    _, h = ops.norm_residual(x, norm="layer", shift=shift)
    assert torch.equal(h, shift.bfloat16().expand(rows, K))
    for fmt in ("e2m1", "e4m3"):
        _, codes, sf = ops.norm_residual(x, norm="layer", out_fmt=fmt)
        assert (codes & (0x77 if fmt == "e2m1" else 0x7F) == 0).all() and (sf == 0).all()
    assert ops.poll_status() == 0


@pytest.mark.parametrize("rows", [2, 301])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", WIDTHS)
def test_constant_rows_normalize_to_zero_after_the_block(K, stream, rows):
    ops = _ops()
    value = torch.tensor([896.0, 1.75, -0.3, 1e-3, -65000.0], device="cuda").bfloat16()
    y = value[torch.arange(rows, device="cuda") % 5].unsqueeze(1).expand(rows, K).contiguous()
    x = torch.randn(rows, K, device="cuda").to(stream)
    z, _ = ops.norm_residual(x, y, norm="rms", post_norm="layer")
    assert torch.equal(z, x)
    bias = torch.randn(K, device="cuda")
    z, _ = ops.norm_residual(x, y, norm="rms", post_norm="layer", post_bias=bias)
    assert torch.equal(z, (x.float() + bias).to(stream)) and ops.poll_status() == 0


@pytest.mark.parametrize("rows", [3, 301])
@pytest.mark.parametrize("K", WIDTHS)
def test_fp32_rows_far_from_zero_keep_their_deviations(K, rows):
    """Means of 1000 deviations and more, beside a row near zero; every row for itself."""
    ops = _ops()
    g = torch.Generator(device="cuda").manual_seed(K + rows)
    x = torch.randn(rows, K, generator=g, device="cuda")
    kind = torch.arange(rows, device="cuda").unsqueeze(1) % 3
    x = torch.where(kind == 0, 1000 + 0.02 * x, torch.where(kind == 1, -7 + 0.001 * x, x))
    _, h = ops.norm_residual(x, norm="layer", eps=1e-12)
    v = x.double()
    var, mean = torch.var_mean(v, -1, correction=0, keepdim=True)
    n = (v - mean) / torch.sqrt(var + 1e-12)
    # a row near zero takes the plain mean: 128 u mean|v| / std more
    far = mean.square() > 256 * var
    bound = 128 * U32 * (1 + n.abs() + torch.where(far, 0.0, (v.abs().mean(-1, keepdim=True) / var.sqrt())))
    bound = bound + U16 * (n.abs() + bound)
    bad = (h.double() - n).abs() > bound
    assert far[0] and far[1] and not far[2]
    assert not bad.any(), "%d elements off, worst %.3g" % (int(bad.sum()), float((h.double() - n).abs().max()))
    # a row's result does not depend on its neighbours
    _, h0 = ops.norm_residual(x[2::3].contiguous(), norm="layer", eps=1e-12)
    if rows < 297 or h0.shape[0] > 296:
        assert torch.equal(h0, h[2::3])
    assert ops.poll_status() == 0
