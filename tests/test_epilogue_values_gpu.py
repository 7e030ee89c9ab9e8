"""The epilogues' arithmetic over all of bf16: an operand of zeros leaves the bias as the sum, so
that every value reaches the activation and the MX quantizer, on both kernels (one row and many).

Bounds.  A sum v that is exact; the activations' exponent is below 128 and carries three half
steps, which exp turns into 128 * 3 * 2^-24 ln 2 < 134 * 2^-23 of the value, polynomial, quotient and
products another 16 * 2^-23; bf16's half step is 2^-8.  Where 1 + exp passes 2^126 the quotient is 0:
the value is then below 90 * 2^-126 < 2^-119."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _ops():
    from fp8_mixed_precision_mxq_b200 import ops
    return ops


def all_bf16():
    return torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.uint16).view(torch.bfloat16)


def act64(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * 0.5 * torch.special.erfc(v * -math.sqrt(0.5))  # ndtr loses v < -7 to cancellation
    if act == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3))
    return v


@pytest.mark.parametrize("M", [1, 64, 65])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh"])
def test_activation_of_every_bf16_value(act, M):
    ops = _ops()
    v = all_bf16()
    a = torch.zeros(M, 8, dtype=torch.bfloat16, device="cuda")
    y = ops.gemm_bf16_residual(a, torch.zeros(65536, 8, dtype=torch.bfloat16, device="cuda"), bias=v, act=act)
    assert ops.poll_status() == 0 and ops.last_path().startswith("rows") == (M <= 64)
    want = act64(v.double(), act)
    assert torch.equal(y.isnan().any(0), want.isnan()) and torch.equal(y.isnan().all(0), want.isnan())
    fine = ~want.isnan()
    got, want = y.double()[:, fine], want[fine].expand(M, -1)
    big = want.abs() > torch.finfo(torch.bfloat16).max
    assert torch.equal(got[big], want[big])
    off = (got[~big] - want[~big]).abs()
    bound = (2.0 ** -8 + 150 * 2.0 ** -23) * want[~big].abs() + 2.0 ** -119 * (act != "none")
    assert (off <= bound).all(), "worst %.3g" % float((off / (want[~big].abs() + 1e-300)).max())


@pytest.mark.parametrize("M", [1, 64, 65, 300])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_codes_of_extreme_magnitudes(M, fmt):
    """h = gate bias * up bias over every size bf16 holds: the bits that the quantizer writes for it."""
    ops = _ops()
    g = torch.Generator(device="cuda").manual_seed(M)
    H = 32 * 520
    size = torch.exp2((torch.arange(520, device="cuda", dtype=torch.float64) - 260) / 2).float()
    bg = torch.randn(H, generator=g, device="cuda").bfloat16()
    bg = (bg.float().view(520, 32) * size[:, None]).view(H).bfloat16()
    bu = (torch.rand(520, 32, generator=g, device="cuda") * size[:, None]).view(H).bfloat16()
    bg[77], bu[3000], bu[4000] = float("nan"), float("inf"), -0.0
    a, w = (torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda") for n in (M, H))
    h = ops.gemm_bf16_gated(a, w, w, bg, bu, act="none")
    want = bg.float() * bu.float()
    assert torch.equal(h.nan_to_num(7), want.bfloat16().nan_to_num(7).expand(M, H))
    codes, sf = ops.gemm_bf16_gated(a, w, w, bg, bu, act="none", out_fmt=fmt)
    want_c, want_s = ops.quantize_act(h, fmt)
    assert torch.equal(codes, want_c) and torch.equal(sf, want_s) and ops.poll_status() == 0


def test_results_repeat_bit_for_bit():
    ops = _ops()
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    K, H = 1024, 2048
    wg, wu, wd = ops.quantize_weight(rnd(H, K)), ops.quantize_weight(rnd(H, K)), ops.quantize_weight(rnd(K, H))
    for M in (1, 48, 200, 3000):
        x, r = rnd(M, K), rnd(M, K)
        first = ops.gated_ffn(x, wg, wu, wd, up_fmt="e4m3", residual=r)
        lin = ops.linear_residual(x, wg, act="gelu")
        for _ in range(5):
            assert torch.equal(ops.gated_ffn(x, wg, wu, wd, up_fmt="e4m3", residual=r), first)
            assert torch.equal(ops.linear_residual(x, wg, act="gelu"), lin)
    assert ops.poll_status() == 0
