"""The operators around retention in a RetNet layer, as cases to measure: the rotary prologue (`rotary` and its
gradient), layer norm (forward, with the residual sum, and backward with the weights' gradients) and the backward
of the output epilogue (per-head RMSNorm times a swish gate).

`run` computes a case either in its plain form (elementary torch operations in 32 bits, angles in 64) or, with
`own` set, by the library's entry points. `exact` gives the same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CAP = 340_000_000  # bytes of one pass of the largest case


def listed():
    return [
        # layer norm before the retention sub-layer of the 1.3B-shaped layer: 4 x 2048 tokens, 8 heads of 256
        dict(name="ln_1p3b", op="ln", rows=8192, D=2048, dtype="bf16", weights="same", residual=False),
        # one decode step of 64 sequences at a model width of 16 x 256, residual added: launch latency
        dict(name="ln_decode_residual", op="ln", rows=64, D=4096, dtype="bf16", weights="f32", residual=True),
        # fp32 activations at a width that leaves no 16-byte rows
        dict(name="ln_odd_f32", op="ln", rows=9189, D=1023, dtype="f32", weights="same", residual=True),
        # training step of the 6.7B-shaped layer: 8192 tokens, width 4096, gradient of the residual stream added
        dict(name="ln_bwd_6p7b", op="ln_bwd", rows=8192, D=4096, dtype="bf16", weights="f32", residual=True),
        # a ragged batch at an odd width
        dict(name="ln_bwd_odd", op="ln_bwd", rows=3885, D=771, dtype="bf16", weights="same", residual=False),
        # q and k of the 1.3B-shaped layer, interleaved pairs over the whole head, k pre-scaled
        dict(name="rotary_1p3b", op="rotary", B=4, N=2048, H=8, d=256, rot=256, layout="interleaved",
             where="offset", fused=True, amplitude=1.0, dtype="bf16"),
        # one decode step of 64 sequences, each at a position of its own in a long context
        dict(name="rotary_decode", op="rotary", B=64, N=1, H=16, d=256, rot=256, layout="interleaved",
             where="starts", fused=True, amplitude=1.0, dtype="bf16"),
        # gradient at the gated layer's shapes: half layout, half of the head rotated, packed documents' positions
        dict(name="rotary_bwd_gated", op="rotary_bwd", B=2, N=16384, H=8, d=128, rot=64, layout="half",
             where="positions", fused=False, amplitude=1.0, dtype="bf16"),
        # fp32, odd sizes, frequencies and amplitude scaled for a long context
        dict(name="rotary_odd_f32", op="rotary", B=3, N=1001, H=5, d=72, rot=36, layout="half",
             where="starts", fused=False, amplitude=1.2, dtype="f32"),
        # backward of the epilogue at the 1.3B-shaped retention output
        dict(name="gate_bwd_1p3b", op="gate_bwd", B=4, H=8, N=2048, d=512, dtype="bf16"),
        # and at the gated layer's long sequence: the largest case
        dict(name="gate_bwd_gated", op="gate_bwd", B=2, H=8, N=16384, d=128, dtype="bf16"),
        # fp32, odd sizes
        dict(name="gate_bwd_odd_f32", op="gate_bwd", B=3, H=5, N=333, d=99, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: sizes spread over the logarithm of their ranges, widths either whole 16-byte rows or not."""
    op = rng.choice(["ln", "ln_bwd", "rotary", "rotary_bwd", "gate_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    odd = rng.random() < 0.35
    if op in ("ln", "ln_bwd"):
        D = _log(rng, 32, 16384)
        D = D if odd else max(32, D // 32 * 32)
        case = dict(op=op, rows=_log(rng, 1, 65536), D=D, dtype=dtype, weights=rng.choice(["same", "f32", "none"]),
                    residual=rng.random() < 0.5)
        key = "rows"
    elif op in ("rotary", "rotary_bwd"):
        d = rng.randrange(8, 257) if odd else rng.choice([32, 64, 96, 128, 192, 256])
        rot = 2 * rng.randrange(1, d // 2 + 1) if odd else rng.choice([d, d, d // 2])
        case = dict(op=op, B=_log(rng, 1, 64), N=_log(rng, 1, 16384), H=rng.randrange(1, 33), d=d, rot=rot,
                    layout=rng.choice(["interleaved", "half"]), where=rng.choice(["offset", "starts", "positions"]),
                    fused=rng.random() < 0.5 and op == "rotary", amplitude=rng.choice([1.0, 1.0, 1.1]), dtype=dtype)
        key = "N"
    else:
        d = rng.randrange(16, 1025) if odd else rng.choice([32, 64, 128, 256, 512, 1024])
        case = dict(op=op, B=_log(rng, 1, 64), H=rng.randrange(1, 33), N=_log(rng, 1, 16384), d=d, dtype=dtype)
        key = "N"
    while work(case)["bytes"] > 0.95 * CAP:
        if case[key] > 1:
            case[key] = max(1, case[key] * 2 // 3)
        else:
            case["B"] = max(1, case["B"] // 2)
    return case


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("ln", "ln_bwd"):
        M, D = case["rows"], case["D"]
        back, res = case["op"] == "ln_bwd", case["residual"]
        we = 0 if case["weights"] == "none" else 4 if case["weights"] == "f32" else e
        if back:  # dy, x (, dsum) and the statistics in, dx and the weights' gradients out
            return {"bytes": M * D * e * (4 if res else 3) + 8 * M + D * we * 3, "flops": 16 * M * D}
        return {"bytes": M * D * e * (4 if res else 2) + D * we * 2, "flops": 8 * M * D}
    if case["op"] in ("rotary", "rotary_bwd"):
        n = case["B"] * case["N"]
        pos = {"offset": 0, "starts": 8 * case["B"], "positions": 8 * n}[case["where"]]
        return {"bytes": 2 * 2 * n * case["H"] * case["d"] * e + 4 * case["rot"] + pos,
                "flops": 2 * n * case["H"] * (3 * case["rot"] + case["d"])}
    n = case["B"] * case["H"] * case["N"] * case["d"]
    return {"bytes": 5 * n * e, "flops": 24 * n}


def _frequencies(rot, scaled):
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if scaled:  # interpolated where a period is longer than an 8192-token context, ramped between 1 and 32 turns
        turns = 8192.0 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / 8.0
    return f.to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    s = {"case": case}
    if case["op"] in ("ln", "ln_bwd"):
        M, D = case["rows"], case["D"]
        # a residual stream: rows of different size, channels with offsets of their own
        x = (normal(M, D) * torch.exp(0.5 * normal(M, 1)) + 0.5 * normal(D)).to(t)
        wt = torch.float32 if case["weights"] == "f32" else t
        none = case["weights"] == "none"
        s["x"] = x
        s["weight"] = None if none else (1.0 + 0.2 * normal(D)).to(wt)
        s["bias"] = None if none else (0.1 * normal(D)).to(wt)
        if case["op"] == "ln":
            s["residual"] = normal(M, D).to(t) if case["residual"] else None
        else:
            x64 = x.double()
            s["mean"] = x64.mean(-1).float()
            s["rstd"] = (x64.var(-1, unbiased=False) + EPS).rsqrt().float()
            s["dy"] = normal(M, D).to(t)
            s["dsum"] = normal(M, D).to(t) if case["residual"] else None
        return s
    if case["op"] in ("rotary", "rotary_bwd"):
        B, N, H, d = case["B"], case["N"], case["H"], case["d"]
        s["freqs"] = _frequencies(case["rot"], case["amplitude"] != 1.0)
        s["k_scale"] = d ** -0.5
        s["offset"], s["starts"], s["positions"] = 0, None, None
        if case["where"] == "offset":
            s["offset"] = 4096
        elif case["where"] == "starts":
            s["starts"] = torch.randint(0, 1_000_000, (B,), generator=g, device=DEV)
        else:  # documents of different lengths packed into each row
            first = torch.rand(B, N, generator=g, device=DEV) < 8.0 / N
            first[:, 0] = True
            at = torch.arange(N, device=DEV).expand(B, N)
            s["positions"] = at - torch.where(first, at, 0).cummax(1).values
        if case["op"] == "rotary":
            if case["fused"]:  # q, k and v side by side in one projection's output
                x = normal(B, N, 3 * H * d).to(t)
                s["q"], s["k"] = x[..., :H * d].unflatten(-1, (H, d)), x[..., H * d:2 * H * d].unflatten(-1, (H, d))
            else:
                s["q"], s["k"] = normal(B, N, H, d).to(t), normal(B, N, H, d).to(t)
        else:
            s["dq"], s["dk"] = normal(B, H, N, d).to(t), normal(B, H, N, d).to(t)
        return s
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    s["o"] = (normal(B, H, N, d) * torch.exp(normal(B, H, N, 1))).to(t)  # the decays give rows of different size
    s["gate"] = normal(B, N, H, d).to(t)
    s["dy"] = (normal(B, N, H, d) / math.sqrt(d)).to(t)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"ln": _own_ln, "ln_bwd": _own_ln_bwd, "rotary": _own_rotary, "rotary_bwd": _own_rotary_bwd,
                "gate_bwd": _own_gate_bwd}[op](state)
    return {"ln": _plain_ln, "ln_bwd": _plain_ln_bwd, "rotary": _plain_rotary, "rotary_bwd": _plain_rotary_bwd,
            "gate_bwd": _plain_gate_bwd}[op](state)


# ---------------------------------------------------------------- the library's calls

def _own_ln(s):
    from linear_attention_ret_b200 import ret
    if s["residual"] is None:
        return [ret.layer_norm(s["x"], s["weight"], s["bias"], EPS)]
    return list(ret.layer_norm(s["x"], s["weight"], s["bias"], EPS, residual=s["residual"]))


def _own_ln_bwd(s):
    from linear_attention_ret_b200 import ret
    return list(ret.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], dsum=s["dsum"],
                                        dbias=s["bias"] is not None))


def _own_rotary(s):
    from linear_attention_ret_b200 import ret
    c = s["case"]
    return list(ret.rotary(s["q"], s["k"], s["freqs"], positions=s["positions"], starts=s["starts"],
                           offset=s["offset"], layout=c["layout"], amplitude=c["amplitude"], k_scale=s["k_scale"]))


def _own_rotary_bwd(s):
    from linear_attention_ret_b200 import ret
    c = s["case"]
    return list(ret.rotary_backward(s["dq"], s["dk"], s["freqs"], positions=s["positions"], starts=s["starts"],
                                    offset=s["offset"], layout=c["layout"], amplitude=c["amplitude"],
                                    k_scale=s["k_scale"]))


def _own_gate_bwd(s):
    from linear_attention_ret_b200 import ret
    return list(ret.msr_norm_gate_backward(s["dy"], s["o"], s["gate"], EPS))


# ---------------------------------------------------------------- plain forms

def _plain_ln(s):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    c = x - x.mean(-1, keepdim=True)
    y = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
    if s["weight"] is not None:
        y = y * s["weight"].float() + s["bias"].float()
    y = y.to(s["x"].dtype)
    return [y] if s["residual"] is None else [y, x.to(s["x"].dtype)]


def _plain_ln_bwd(s):
    dy, t = s["dy"].float(), s["x"].dtype
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    w = s["weight"]
    u = dy if w is None else dy * w.float()
    dx = s["rstd"][:, None] * (u - u.mean(-1, keepdim=True) - xh * (u * xh).mean(-1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    if w is None:
        return [dx.to(t), None, None]
    return [dx.to(t), (dy * xh).sum(0).to(w.dtype), dy.sum(0).to(w.dtype)]


def _plain_turn(x, s, scale, sign):
    """x [B, N, H, d] rotated by sign times its positions' angles."""
    c = s["case"]
    rot, t = c["rot"], x.dtype
    x = x.float()
    B, N = x.shape[:2]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(N, device=x.device)[None, :].expand(B, N)
        if s["starts"] is not None:
            pos = pos + s["starts"][:, None]
    ang = (pos + s["offset"]).double()[:, :, None, None] * s["freqs"]
    cos, sin = ang.cos().float() * c["amplitude"], sign * ang.sin().float() * c["amplitude"]
    if c["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return (torch.cat([r, x[..., rot:]], -1) * scale).to(t)


def _plain_rotary(s):
    return [_plain_turn(s["q"], s, 1.0, 1.0).transpose(1, 2).contiguous(),
            _plain_turn(s["k"], s, s["k_scale"], 1.0).transpose(1, 2).contiguous()]


def _plain_rotary_bwd(s):
    return [_plain_turn(s["dq"].transpose(1, 2), s, 1.0, -1.0).contiguous(),
            _plain_turn(s["dk"].transpose(1, 2), s, s["k_scale"], -1.0).contiguous()]


def _plain_gate_bwd(s):
    t = s["o"].dtype
    o, g, dy = s["o"].float(), s["gate"].float().transpose(1, 2), s["dy"].float().transpose(1, 2)
    r = torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS)
    sig = 1.0 / (1.0 + torch.exp(-g))
    u = dy * g * sig
    do = r * u - o * (r * r * r) * (u * o).mean(-1, keepdim=True)
    dg = dy * o * r * (sig + g * sig * (1.0 - sig))
    return [do.to(t), dg.to(t).transpose(1, 2).contiguous()]


# ---------------------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ln":
        x = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        y = _define_ln(x, s["weight"], s["bias"])
        return [y] if s["residual"] is None else [y, x]
    if case["op"] == "ln_bwd":
        leaves = [None if v is None else v.double().requires_grad_() for v in (s["x"], s["weight"], s["bias"])]
        x, w, b = leaves
        total = (_define_ln(x, w, b) * s["dy"].double()).sum()
        if s["dsum"] is not None:
            total = total + (x * s["dsum"].double()).sum()
        grads = iter(torch.autograd.grad(total, [v for v in leaves if v is not None]))
        return [None if v is None else next(grads) for v in leaves]
    if case["op"] in ("rotary", "rotary_bwd"):
        back = case["op"] == "rotary_bwd"
        names = ("dq", "dk") if back else ("q", "k")
        return [_define_turn(s[n].transpose(1, 2) if back else s[n], s, 1.0 if n[-1] == "q" else s["k_scale"], back)
                for n in names]
    o, g = s["o"].double().requires_grad_(), s["gate"].double().requires_grad_()
    y = g * torch.sigmoid(g) * (o / torch.sqrt(o.pow(2).sum(-1, keepdim=True) / case["d"] + EPS)).transpose(1, 2)
    return list(torch.autograd.grad((y * s["dy"].double()).sum(), [o, g]))


def _define_ln(x, w, b):
    D = x.shape[-1]
    mu = x.sum(-1, keepdim=True) / D
    var = ((x - mu) ** 2).sum(-1, keepdim=True) / D
    y = (x - mu) / torch.sqrt(var + EPS)
    return y if w is None else y * w.double() + b.double()


def _define_turn(x, s, scale, back):
    """Pairs as complex numbers times m e^(i t); back: times the conjugate. [B, N, H, d] in, heads moved as `run` does."""
    c = s["case"]
    rot = c["rot"]
    B, N, H, d = x.shape
    n = torch.arange(N, dtype=torch.float64, device=x.device)
    pos = s["positions"].double() if s["positions"] is not None else n.expand(B, N)
    if s["starts"] is not None:
        pos = pos + s["starts"].double().unsqueeze(1)
    t = torch.einsum("bn,f->bnf", pos + float(s["offset"]), s["freqs"]).unsqueeze(2)
    z = torch.polar(torch.full_like(t, c["amplitude"]), -t if back else t)
    x = x.double()
    head = x[..., :rot]
    pairs = head.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if c["layout"] == "half" else head.unflatten(-1, (-1, 2))
    w = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    y = x.clone()
    y[..., :rot] = (w.transpose(-1, -2) if c["layout"] == "half" else w).reshape(B, N, H, rot)
    y = y * scale
    return y.contiguous() if back else y.transpose(1, 2).contiguous()
