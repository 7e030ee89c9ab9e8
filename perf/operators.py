"""The operators around a block's quantized linears, as they are timed: the fused norm and
residual, the linear with activation and residual in its epilogue, and the gated
feed-forward network.  `run` computes them in plain torch operations, or, with `own` set,
by the library's calls; `exact` in 64 bits."""
import math

import torch

own = False

# Sizes of the repository's workloads: model width 5120, FFN 13824, 32760 tokens (480p) and
# 75600 tokens (720p), text context 512 of width 4096.
DIM, FFN, TOKENS_480P, TOKENS_720P = 5120, 13824, 32760, 75600


def _norm(name, rows, K, **kw):
    c = dict(op="norm", rows=rows, K=K, norm="layer", post="none", affine=False, mod=True, groups=1, stream="bf16",
             vec="f32", out="bf16")
    return {"name": name, **c, **kw} if name else {**c, **kw}


def _linear(name, M, N, K, fmt, **kw):
    c = dict(op="linear", M=M, N=N, K=K, fmt=fmt, act="none", bias=True, residual=True, gate_groups=0)
    return {"name": name, **c, **kw} if name else {**c, **kw}


def _gated(name, M, K, H, fmt, h_fmt, **kw):
    c = dict(op="gated", M=M, K=K, H=H, fmt=fmt, h_fmt=h_fmt, act="silu", bias=False, residual=True)
    return {"name": name, **c, **kw} if name else {**c, **kw}


def listed():
    return [
        # one token of a decoder: residual add, RMSNorm with weight, E4M3 operand of the next linear
        _norm("norm_token", 1, DIM, norm="rms", affine=True, mod=False, vec="bf16", out="e4m3"),
        # a ragged chunk with norms before and after the block (RMS both) on an fp32 residual stream
        _norm("norm_sandwich_chunk", 1023, 4096, norm="rms", post="rms", affine=True, mod=False, stream="f32"),
        # a 480p video block: gated residual, LayerNorm and modulation of two clips, bf16 out
        _norm("norm_adaln_480p", TOKENS_480P, DIM, groups=2),
        # a 720p video block whose next linear is W4A8: the operand is written quantized
        _norm("norm_adaln_720p_e4m3", TOKENS_720P, DIM, out="e4m3"),
        # one token through an output projection: bias and residual, W4A4
        _linear("linear_token", 1, DIM, DIM, "e2m1"),
        # a batch of 48 decoding sequences through the second FFN linear, W4A8
        _linear("linear_batch", 48, DIM, FFN, "e4m3"),
        # the text embedding's first linear with its tanh GELU, kept in bf16
        _linear("linear_text_bf16", 512, DIM, 4096, "bf16", act="gelu_tanh", residual=False),
        # FFN-down of a 480p block with its gate and residual, W4A8
        _linear("linear_ffn_down_480p", TOKENS_480P, DIM, FFN, "e4m3", gate_groups=1),
        # one token through a gated FFN, W4A4 up and W4A8 down
        _gated("gated_token", 1, DIM, FFN, "e2m1", "e4m3"),
        # a ragged prefill chunk: the two projections and their product alone, bf16 out
        _gated("gated_up_chunk", 777, 2048, 5632, "e4m3", "bf16", bias=True, residual=False),
        # a ragged chunk through the fused norm, the gated FFN and its residual, one after the other
        _gated("gated_block_chunk", 2049, DIM, 8192, "e4m3", "e2m1", residual=True, chain=True),
        # a 480p block's tokens through a gated FFN, W4A4
        _gated("gated_ffn_480p", TOKENS_480P, DIM, FFN, "e2m1", "e2m1"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "gated"])
    if op == "norm":
        rows = _log(rng, 1, TOKENS_720P)
        K = 32 * rng.randint(8, 256)
        while rows * K > TOKENS_720P * DIM:
            rows = _log(rng, 1, TOKENS_720P)
        return _norm(None, rows, K, norm=rng.choice(["layer", "rms"]), post=rng.choice(["none", "rms", "layer"]),
                     affine=rng.random() < 0.5, mod=rng.random() < 0.5, groups=rng.randint(1, min(3, rows)),
                     stream=rng.choice(["bf16", "bf16", "f32"]), vec=rng.choice(["f32", "bf16"]),
                     out=rng.choice(["bf16", "e4m3"]))
    fmt = rng.choice(["e2m1", "e4m3"])
    M = _log(rng, 1, 16384)
    if op == "linear":
        fmt = rng.choice([fmt, fmt, "bf16"])
        K = 128 * rng.randint(4, 64) if fmt == "e4m3" else 32 * rng.randint(16, 256)
        return _linear(None, M, 8 * rng.randint(64, 1024), K, fmt,
                       act=rng.choice(["none", "gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.7,
                       residual=rng.random() < 0.8, gate_groups=rng.randint(0, min(2, M)))
    chain = rng.random() < 0.3
    return _gated(None, M, 128 * rng.randint(4, 48), 128 * rng.randint(8, 80), fmt,
                  rng.choice(["e2m1", "e4m3"]) if chain else rng.choice(["e2m1", "e4m3", "bf16"]),
                  act=rng.choice(["silu", "gelu", "gelu_tanh"]), bias=rng.random() < 0.5, chain=chain)


def _rows_per_group(rows, groups):
    return -(-rows // groups)


# ---------------------------------------------------------------------------- inputs

_EMAX = {"e2m1": 2, "e4m3": 8}


def _mx_round(x, fmt):
    """(element values, E8M0 scale codes) of the MX quantization of a bf16-valued x [R, K]:
    blocks of 32 along K, scale 2^(floor(log2 amax) - emax), round to nearest even, saturating."""
    R, K = x.shape
    b = x.float().view(R, K // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    code = torch.where(amax > 0, torch.frexp(amax)[1] - 1 - _EMAX[fmt] + 127, torch.zeros_like(amax).int()).clamp(0, 254)
    v = torch.ldexp(b, 127 - code)
    a = v.abs()
    if fmt == "e2m1":
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        q = (torch.round(a / step) * step).clamp(max=6.0)
    else:
        step = torch.ldexp(torch.ones_like(a), (torch.frexp(a)[1] - 1).clamp(min=-6) - 3)
        q = (torch.round(a / step) * step).clamp(max=448.0)
    return torch.copysign(q, b).view(R, K), code.view(R, K // 32)


def _tiled(code):
    """Scale codes [R, K/32] in the tiled layout (atoms of 128 rows x 4 k-blocks, zero-padded)."""
    R, KB = code.shape
    rb, kb = -(-R // 128), -(-KB // 4)
    full = torch.zeros(rb * 128, kb * 4, dtype=torch.uint8, device=code.device)
    full[:R, :KB] = code.to(torch.uint8)
    return full.view(rb, 4, 32, kb, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untiled(sf, R, K):
    rb, kb = -(-R // 128), -(-(K // 32) // 4)
    return sf.view(rb, kb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, kb * 4)[:R, : K // 32]


def _codes(x, fmt):
    """Packed MX codes and tiled scales of a bf16 tensor."""
    q, code = _mx_round(x, fmt)
    if fmt == "e4m3":
        return q.to(torch.float8_e4m3fn).view(torch.uint8), _tiled(code)
    m = q.abs()
    c = torch.where(m < 4, torch.where(m < 2, m * 2, m + 2), m / 2 + 4).to(torch.uint8)
    c = torch.where(torch.signbit(q), c + 8, c)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous(), _tiled(code)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _decode(codes, sf, R, K, fmt, dtype):
    """The values that packed codes and tiled scales stand for."""
    if fmt == "e4m3":
        v = codes.view(torch.float8_e4m3fn).view(R, K).to(dtype)
    else:
        table = torch.tensor(_E2M1 + tuple(-t for t in _E2M1), dtype=dtype, device=codes.device)
        c = codes.view(R, K // 2)
        v = table[torch.stack((c & 15, c >> 4), -1).int()].view(R, K)
    e = _untiled(sf, R, K).int() - 127
    s = torch.ldexp(torch.ones_like(e, dtype=dtype), e)
    return (v.view(R, K // 32, 32) * s.unsqueeze(-1)).view(R, K)


class _Make:
    """Seeded draws on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(int(seed))

    def normal(self, *shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=self.g, device="cuda") * std).to(dtype)

    def activation(self, R, K, dtype=torch.bfloat16):
        """N(0, 1) with about one channel in a hundred 20 times larger."""
        big = torch.rand(K, generator=self.g, device="cuda") < 0.01
        x = torch.randn(R, K, generator=self.g, device="cuda")
        return x.mul_(torch.where(big, 20.0, 1.0)).to(dtype)

    def weight(self, N, K, fmt="e2m1"):
        w = self.normal(N, K, std=0.02)
        return w if fmt == "bf16" else _codes(w, "e2m1")


_VEC = {"f32": torch.float32, "bf16": torch.bfloat16}


def _norm_inputs(m, c):
    rows, K = c["rows"], c["K"]
    stream = torch.float32 if c["stream"] == "f32" else torch.bfloat16
    vec = _VEC[c["vec"]]
    s = dict(x=m.activation(rows, K, stream), y=m.activation(rows, K))
    s["weight"] = (m.normal(K, std=0.3, dtype=torch.float32) + 1).to(vec) if c["affine"] else None
    s["bias"] = m.normal(K, std=0.3, dtype=vec) if c["affine"] and c["norm"] == "layer" else None
    s["post_weight"] = (m.normal(K, std=0.3, dtype=torch.float32) + 1).to(vec) if c["post"] != "none" else None
    s["post_bias"] = m.normal(K, std=0.3, dtype=vec) if c["post"] == "layer" else None
    for name in ("gate", "scale", "shift"):
        s[name] = m.normal(c["groups"], K, std=0.5, dtype=vec) if c["mod"] else None
    return s


def prepare(case, seed):
    m, c = _Make(seed), dict(case)
    s = dict(case=c)
    if c["op"] == "norm":
        s.update(_norm_inputs(m, c))
        return s
    M, K = c["M"], c["K"]
    if c["op"] == "linear":
        s["w"] = m.weight(c["N"], K, c["fmt"])
        s["bias"] = m.normal(c["N"], std=0.1) if c["bias"] else None
        s["x"] = m.activation(M, K)
        s["residual"] = m.normal(M, c["N"]) if c["residual"] else None
        s["gate"] = m.normal(c["gate_groups"], c["N"], std=0.5, dtype=torch.float32) if c["gate_groups"] else None
        return s
    H = c["H"]
    s["gate_w"], s["up_w"] = m.weight(H, K), m.weight(H, K)
    s["gate_b"], s["up_b"] = (m.normal(H, std=0.1), m.normal(H, std=0.1)) if c["bias"] else (None, None)
    if c["h_fmt"] == "bf16":  # the projections alone, on an operand that a norm or quantizer wrote
        s["a"] = _codes(m.activation(M, K), c["fmt"])
        return s
    s["down_w"] = m.weight(K, H)
    s["down_b"] = m.normal(K, std=0.1) if c["bias"] else None
    if c.get("chain"):
        s["norm"] = _norm_inputs(m, _norm(None, M, K))
        s["out_gate"] = m.normal(1, K, std=0.5, dtype=torch.float32)
    else:
        s["x"] = m.activation(M, K)
        s["residual"] = m.normal(M, K) if c["residual"] else None
    return s


# ---------------------------------------------------------------------------- the plain forms

EPS = 1e-6


def _groups(v, rows):
    """[G, K] per-group vectors, one row for each of `rows` rows."""
    if v.shape[0] == 1:
        return v.float()
    rpg = _rows_per_group(rows, v.shape[0])
    return v.float()[torch.arange(rows, device=v.device) // rpg]


def _plain_norm(v, kind, weight, bias):
    if kind == "none":
        return v
    d = v - v.mean(-1, keepdim=True) if kind == "layer" else v
    n = d * torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    n = n if weight is None else n * weight.float()
    return n if bias is None else n + bias.float()


def _plain_norm_residual(s, c):
    rows = c["rows"]
    u = _plain_norm(s["y"].float(), c["post"], s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        u = u * _groups(s["gate"], rows)
    z = (s["x"].float() + u).to(s["x"].dtype)
    n = _plain_norm(z.float(), c["norm"], s["weight"], s["bias"])
    if s["scale"] is not None:
        n = n * (1 + _groups(s["scale"], rows)) + _groups(s["shift"], rows)
    return z, n.to(torch.bfloat16)


def _act(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(v * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _qdq(x, fmt):
    q, code = _mx_round(x, fmt)
    R, K = x.shape
    return torch.ldexp(q.view(R, K // 32, 32), (code - 127).unsqueeze(-1)).view(R, K)


def _matmul(a, w, b):
    y = a @ w.t()
    return y if b is None else y + b.float()


def _plain_weight(w, N, K):
    return _decode(w[0], w[1], N, K, "e2m1", torch.float32) if isinstance(w, tuple) else w.float()


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        z, h = _plain_norm_residual(s, c)
        if c["out"] == "bf16":
            return {"z": z, "h": h}
        q, code = _mx_round(h, c["out"])
        return {"z": z, "codes": q.to(torch.float8_e4m3fn), "scales": _tiled(code).view(torch.float8_e8m0fnu)}
    M, K = c["M"], c["K"]
    if c["op"] == "linear":
        x = s["x"].float() if c["fmt"] == "bf16" else _qdq(s["x"], c["fmt"])
        y = _act(_matmul(x, _plain_weight(s["w"], c["N"], K), s["bias"]), c["act"])
        y = y if s["gate"] is None else y * _groups(s["gate"], M)
        return (y if s["residual"] is None else y + s["residual"].float()).to(torch.bfloat16)
    H = c["H"]
    z = None
    if c["h_fmt"] == "bf16":
        x = _decode(*s["a"], M, K, c["fmt"], torch.float32)
    elif c.get("chain"):
        z, x = _plain_norm_residual(s["norm"], _norm(None, M, K))
        x = _qdq(x, c["fmt"])
    else:
        x = _qdq(s["x"], c["fmt"])
    g = _act(_matmul(x, _plain_weight(s["gate_w"], H, K), s["gate_b"]), c["act"])
    h = (g * _matmul(x, _plain_weight(s["up_w"], H, K), s["up_b"])).to(torch.bfloat16)
    if c["h_fmt"] == "bf16":
        return h
    y = _matmul(_qdq(h, c["h_fmt"]), _plain_weight(s["down_w"], K, H), s["down_b"])
    if z is not None:
        return {"z": z, "y": (z.float() + y * s["out_gate"]).to(torch.bfloat16)}
    return (y if s["residual"] is None else y + s["residual"].float()).to(torch.bfloat16)


# ---------------------------------------------------------------------------- the library's calls


def _own_norm(ops, s, c, out):
    return ops.norm_residual(s["x"], s["y"], norm=c["norm"], weight=s["weight"], bias=s["bias"], gate=s["gate"],
                             scale=s["scale"], shift=s["shift"],
                             rows_per_group=_rows_per_group(c["rows"], c["groups"]), post_norm=c["post"],
                             post_weight=s["post_weight"], post_bias=s["post_bias"], eps=EPS, out_fmt=out)


def _own(s):
    from fp8_mixed_precision_mxq_b200 import ops
    c = s["case"]
    if c["op"] == "norm":
        if c["out"] == "bf16":
            z, h = _own_norm(ops, s, c, "bf16")
            return {"z": z, "h": h}
        z, codes, sf = _own_norm(ops, s, c, c["out"])
        return {"z": z, "codes": codes.view(torch.float8_e4m3fn).view(z.shape), "scales": sf.view(torch.float8_e8m0fnu)}
    M, K = c["M"], c["K"]
    if c["op"] == "linear":
        rpg = _rows_per_group(M, max(1, c["gate_groups"]))
        if c["fmt"] == "bf16":
            return ops.gemm_bf16_residual(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"],
                                          gate=s["gate"], rows_per_group=rpg)
        return ops.linear_residual(s["x"], ops.QWeight(*s["w"], c["N"], K, s["bias"]), c["fmt"], act=c["act"],
                                   residual=s["residual"], gate=s["gate"], rows_per_group=rpg)
    H = c["H"]
    gate, up = ops.QWeight(*s["gate_w"], H, K, s["gate_b"]), ops.QWeight(*s["up_w"], H, K, s["up_b"])
    if c["h_fmt"] == "bf16":
        return ops.gemm_gated(*s["a"], c["fmt"], M, K, gate, up, act=c["act"], out_fmt="bf16")
    down = ops.QWeight(*s["down_w"], K, H, s["down_b"])
    if c.get("chain"):
        z, codes, sf = _own_norm(ops, s["norm"], _norm(None, M, K), c["fmt"])
        codes, sf = ops.gemm_gated(codes, sf, c["fmt"], M, K, gate, up, act=c["act"], out_fmt=c["h_fmt"])
        return {"z": z, "y": ops.gemm_residual(codes, sf, c["h_fmt"], M, H, down, residual=z, gate=s["out_gate"])}
    return ops.gated_ffn(s["x"], gate, up, down, act=c["act"], up_fmt=c["fmt"], down_fmt=c["h_fmt"],
                         residual=s["residual"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------- what a pass cannot do without


def work(case):
    c = case
    per = {"e2m1": 0.5 + 1 / 32, "e4m3": 1 + 1 / 32, "bf16": 2.0}
    if c["op"] == "norm":
        n, st = c["rows"] * c["K"], 4 if c["stream"] == "f32" else 2
        vec = (3 * c["groups"] if c["mod"] else 0) + 2 * c["affine"] + (c["post"] != "none")
        return {"bytes": n * (2 * st + 2 + per[c["out"]]) + vec * c["K"] * (4 if c["vec"] == "f32" else 2), "flops": 12 * n}
    M, K = c["M"], c["K"]
    if c["op"] == "linear":
        N = c["N"]
        return {"bytes": M * K * 2 + N * K * per["bf16" if c["fmt"] == "bf16" else "e2m1"] +
                M * N * 2 * (1 + c["residual"]) + N * (2 * c["bias"] + 4 * c["gate_groups"]), "flops": 2 * M * N * K}
    H = c["H"]
    if c["h_fmt"] == "bf16":
        return {"bytes": M * K * per[c["fmt"]] + 2 * H * K * per["e2m1"] + M * H * 2, "flops": 4 * M * H * K}
    rows = (2 + 2 + 2 + 2) if c.get("chain") else 2 + 2 + 2 * c["residual"]
    return {"bytes": M * K * rows + 3 * H * K * per["e2m1"], "flops": 6 * M * H * K}


# ---------------------------------------------------------------------------- in 64 bits

_GRID = {}


def _grid(fmt):
    """Magnitudes of a format, ascending by code, and the midpoints between neighbours."""
    if fmt not in _GRID:
        if fmt == "e2m1":
            v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        else:
            v = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
            v = v[:-1]  # the last code is NaN
        v = torch.tensor(v, dtype=torch.float64, device="cuda")
        _GRID[fmt] = v, (v[1:] + v[:-1]) / 2
    return _GRID[fmt]


def _exact_mx(h, fmt):
    """(element values, scale values, codes of the scales) of bf16 values h, in 64 bits."""
    grid, mid = _grid(fmt)
    R, K = h.shape
    b = h.to(torch.float64).reshape(R, K // 32, 32)
    amax = b.abs().amax(-1)
    e = torch.floor(torch.log2(amax))
    e = torch.where(torch.exp2(e) > amax, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
    e = torch.where(amax == 0, torch.full_like(e, -127.0), (e - (2 if fmt == "e2m1" else 8)).clamp(min=-127))
    t = (b / torch.exp2(e).unsqueeze(-1)).contiguous()
    a = t.abs()
    low, high = torch.searchsorted(mid, a), torch.searchsorted(mid, a, right=True)
    q = grid[torch.where((low != high) & (low % 2 == 1), high, low)]
    return torch.where(t < 0, -q, q).reshape(R, K), e


def _exact_qdq(h, fmt):
    q, e = _exact_mx(h, fmt)
    R, K = q.shape
    return (q.view(R, -1, 32) * torch.exp2(e).unsqueeze(-1)).view(R, K)


def _exact_norm(v, kind, weight, bias):
    if kind == "none":
        return v
    var, mean = torch.var_mean(v, -1, correction=0, keepdim=True)
    n = (v - mean) / torch.sqrt(var + EPS) if kind == "layer" else v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)
    if weight is not None:
        n = n * weight.double()
    return n if bias is None else n + bias.double()


def _expand(v, rows):
    return v.double().repeat_interleave(-(-rows // v.shape[0]), 0)[:rows]


def _exact_norm_residual(s, c):
    """z and h in 64 bits, h from z in the type it is stored in."""
    u = _exact_norm(s["y"].double(), c["post"], s["post_weight"], s["post_bias"])
    z = s["x"].double() + (u if s["gate"] is None else u * _expand(s["gate"], c["rows"]))
    n = _exact_norm(z.to(s["x"].dtype).double(), c["norm"], s["weight"], s["bias"])
    if s["scale"] is not None:
        n = n + n * _expand(s["scale"], c["rows"]) + _expand(s["shift"], c["rows"])
    return z, n


def _exact_act(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def _exact_linear(x, w, N, b):
    w = _decode(w[0], w[1], N, x.shape[1], "e2m1", torch.float64) if isinstance(w, tuple) else w.double()
    y = torch.mm(x, w.t())
    return y if b is None else y + b.double()


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        z, h = _exact_norm_residual(s, c)
        if c["out"] == "bf16":
            return {"z": z, "h": h}
        q, e = _exact_mx(h.to(torch.bfloat16), c["out"])
        return {"z": z, "codes": q, "scales": torch.exp2(_tiled((e + 127).int()).double() - 127)}
    M, K = c["M"], c["K"]
    if c["op"] == "linear":
        x = s["x"].double() if c["fmt"] == "bf16" else _exact_qdq(s["x"], c["fmt"])
        y = _exact_act(_exact_linear(x, s["w"], c["N"], s["bias"]), c["act"])
        y = y if s["gate"] is None else y * _expand(s["gate"], M)
        return y if s["residual"] is None else y + s["residual"].double()
    H, z = c["H"], None
    if c["h_fmt"] == "bf16":
        x = _decode(*s["a"], M, K, c["fmt"], torch.float64)
    elif c.get("chain"):
        z, h = _exact_norm_residual(s["norm"], _norm(None, M, K))
        x = _exact_qdq(h.to(torch.bfloat16), c["fmt"])
    else:
        x = _exact_qdq(s["x"], c["fmt"])
    h = _exact_act(_exact_linear(x, s["gate_w"], H, s["gate_b"]), c["act"])
    h = h * _exact_linear(x, s["up_w"], H, s["up_b"])
    if c["h_fmt"] == "bf16":
        return h
    y = _exact_linear(_exact_qdq(h.to(torch.bfloat16), c["h_fmt"]), s["down_w"], K, s["down_b"])
    if z is not None:
        return {"z": z, "y": z.to(torch.bfloat16).double() + y * s["out_gate"].double()}
    return y if s["residual"] is None else y + s["residual"].double()
