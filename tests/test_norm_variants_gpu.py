"""Every kernel that the fused norms choose for many rows (more than 296), against float64: one,
two and four chunks a thread, rows that fill the CTA's spans and ragged ones, each stream, vector
type, output and kind of group.  Formulas and bounds are those of test_norm_gpu.py."""
import pytest
import torch

from tests.test_norm_gpu import check, make

pytestmark = pytest.mark.gpu


def _ops():
    from fp8_mixed_precision_mxq_b200 import ops
    return ops


WIDTHS = [
    2048,   # one chunk a thread, eight full spans
    2016,   # one chunk, the last span ragged
    5120,   # two chunks, twenty full spans
    4000,   # two chunks, the last span ragged
    2816,   # two chunks, eleven spans: the last warp's second chunk is past the row
    7168,   # four chunks, full
    5376,   # four chunks, 21 spans
    6176,   # four chunks, the last span ragged
]


@pytest.mark.parametrize("vec", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", WIDTHS)
def test_many_rows(K, stream, vec):
    ops = _ops()
    for i, (rows, rpg, norm, post) in enumerate(((301, 301, "layer", "none"), (300, 101, "rms", "layer"),
                                                 (298, 1, "layer", "rms"), (299, 3, "layer", "layer"))):
        groups = -(-rows // rpg)
        x, y, vecs = make(rows, K, K + i, stream, vec, groups, norm, post, affine=i % 2 == 1)
        z, h = ops.norm_residual(x, y, norm=norm, post_norm=post, rows_per_group=rpg, **vecs)
        check(x, y, z, h, norm, post, vecs, rpg)
        for fmt in ("e2m1", "e4m3"):
            dirty = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
                     for n in ops._mx_bytes(rows, K, ops._fmt(fmt))]
            zq, codes, sf = ops.norm_residual(x, y, norm=norm, post_norm=post, rows_per_group=rpg, out_fmt=fmt,
                                              codes=dirty[0], sf=dirty[1], **vecs)
            want_c, want_s = ops.quantize_act(h, fmt)
            assert torch.equal(zq, z) and torch.equal(codes, want_c) and torch.equal(sf, want_s), (rows, rpg, fmt)
    assert ops.poll_status() == 0


@pytest.mark.parametrize("K", [2048, 4000, 7168])
def test_rows_past_the_last_and_next_to_it_stay(K):
    """Buffers longer than the call's rows keep what lies behind them."""
    ops = _ops()
    rows, more = 299, 40
    x, y, vecs = make(rows + more, K, K)
    z = torch.full_like(x, 7.0)
    h = torch.full_like(y, 7.0)
    ops.norm_residual(x[:rows], y[:rows], z=z[:rows], h=h[:rows], **vecs)
    assert (z[rows:] == 7).all() and (h[rows:] == 7).all()
    check(x[:rows], y[:rows], z[:rows], h[:rows], "layer", "none", vecs, rows)


def test_results_repeat_bit_for_bit():
    ops = _ops()
    for rows, K in ((3, 5120), (300, 2048), (5000, 5120), (700, 7168)):
        x, y, vecs = make(rows, K, rows)
        first = ops.norm_residual(x, y, out_fmt="e4m3", **vecs)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, ops.norm_residual(x, y, out_fmt="e4m3", **vecs)))


@pytest.mark.parametrize("rows", [2, 301])
def test_codes_of_extreme_magnitudes(rows):
    """Blocks of every size bf16 holds, subnormal and infinite ones too: the quantizer's bits."""
    ops = _ops()
    K = 32 * 288
    x, _, _ = make(rows, K, rows)
    weight = torch.exp2(torch.arange(288, device="cuda", dtype=torch.float64) - 150).clamp(max=2.0 ** 127).float()
    weight = weight.repeat_interleave(32)
    _, h = ops.norm_residual(x, norm="rms", weight=weight)
    assert h.isinf().any() and (h == 0).any()
    for fmt in ("e2m1", "e4m3"):
        _, codes, sf = ops.norm_residual(x, norm="rms", weight=weight, out_fmt=fmt)
        want_c, want_s = ops.quantize_act(h, fmt)
        assert torch.equal(codes, want_c) and torch.equal(sf, want_s), fmt
    assert ops.poll_status() == 0
