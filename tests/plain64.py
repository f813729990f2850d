"""Plain 64-bit forms of the operators around retention (rotary prologue, layer norm, the output
epilogue's gradients), for the tests: torch float64 on the CPU, from the formulas, with no code of
the library. Also the bounds that the tests allow, counted in rounding steps.

u(t) = torch.finfo(t).eps / 2 is the relative error of one rounding to t. An fp32 sum of n terms
held as runs of at most L terms and joined in pairs is off by at most (L + log2 n) u(f32) of the
sum of magnitudes.
"""
import torch

U32 = torch.finfo(torch.float32).eps / 2


def run(D):
    """Longest serial run of an fp32 sum over a row of D, plus the joins."""
    return 80 if D <= 16384 else D // 256 + 16


def u(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def positions(B, N, positions=None, starts=None, offset=0):
    if positions is not None:
        return offset + positions.cpu()
    n = offset + torch.arange(N)[None, :].expand(B, N)
    return n if starts is None else n + starts.cpu()[:, None]


def rotate(x, freqs, pos, layout="interleaved", amplitude=1.0, scale=1.0, inverse=False):
    """x [B, N, H, d] turned by pos [B, N] * freqs [rot/2]; also the size |a| + |b| behind each output."""
    x = f64(x)
    y, size = x.clone(), x.abs()
    if freqs is not None and len(freqs):
        f = f64(freqs)
        r = 2 * len(f)
        t = (pos.to(torch.float64)[..., None] * f)[:, :, None, :]
        c, s = amplitude * t.cos(), amplitude * t.sin() * (-1.0 if inverse else 1.0)
        i = slice(0, r // 2) if layout == "half" else slice(0, r, 2)
        j = slice(r // 2, r) if layout == "half" else slice(1, r, 2)
        a, b = x[..., i], x[..., j]
        y[..., i], y[..., j] = a * c - b * s, a * s + b * c
        size[..., i] = size[..., j] = (a.abs() + b.abs()) * abs(amplitude)
    return y * scale, size * abs(scale)


def rotate_bound(y, size, dtype):
    """cos and sin within 2^-21, three fp32 products and a sum, one rounding to dtype."""
    return u(dtype) * y.abs() + (2.0 ** -21 + 6 * U32) * size + 1e-37


def layer_norm(x, w, b, eps, residual=None):
    """(y, s, mean, rstd)"""
    s = f64(x) if residual is None else f64(x) + f64(residual)
    mu = s.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt(((s - mu) ** 2).mean(-1, keepdim=True) + eps)
    y = (s - mu) * r * (1.0 if w is None else f64(w)) + (0.0 if b is None else f64(b))
    return y, s, mu[..., 0], r[..., 0]


def layer_norm_bound(s, w, b, eps, dtype):
    """Of y: the mean is off by RUN u of the mean magnitude, the centred value by u of |s| more; the
    variance by (RUN + 2) u and by twice the centred values' errors, the fp32 rsqrt by 2 u."""
    RUN = run(s.shape[-1])
    mu = s.mean(-1, keepdim=True)
    v = ((s - mu) ** 2).mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt(v + eps)
    aw = 1.0 if w is None else f64(w).abs()
    ab = 0.0 if b is None else f64(b).abs()
    xh = ((s - mu) * r).abs()
    centre = U32 * (2 * s.abs() + 2 * mu.abs() + RUN * s.abs().mean(-1, keepdim=True))
    # the variance's centred values carry `centre` too: relative error of r at most r^2 mean(|c| centre)
    rel = U32 * (RUN / 2 + 6) + r * r * ((s - mu).abs() * centre).mean(-1, keepdim=True)
    y32 = aw * (r * centre + xh * rel) + U32 * (2 * aw * xh + ab)
    y = (aw * xh + ab)
    return u(dtype) * y + (1 + u(dtype)) * y32 + 1e-37


def layer_norm_backward(dy, x, w, mean, rstd, dsum=None):
    """(dx, dw, db) from given statistics; dw for weight 1 too."""
    dy, x, mean, rstd = f64(dy), f64(x), f64(mean)[..., None], f64(rstd)[..., None]
    xh = (x - mean) * rstd
    g = dy if w is None else dy * f64(w)
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    if dsum is not None:
        dx = dx + f64(dsum)
    D = x.shape[-1]
    return dx, (dy * xh).reshape(-1, D).sum(0), dy.reshape(-1, D).sum(0)


def layer_norm_backward_bounds(dy, x, w, mean, rstd, dsum, dtype, wdtype, rows_run):
    """Bounds of (dx, dw, db). rows_run: longest serial run of the sums over rows, plus the joins."""
    RUN = run(x.shape[-1])
    dy, x, mean, rstd = f64(dy), f64(x), f64(mean)[..., None], f64(rstd)[..., None]
    xh = ((x - mean) * rstd).abs()
    exh = 2 * U32 * (xh + (x.abs() + mean.abs()) * rstd)  # of xh: a difference and a product in fp32
    g = dy.abs() * (1.0 if w is None else f64(w).abs())
    m1, m2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    em2 = (g * exh).mean(-1, keepdim=True) + (RUN + 4) * U32 * m2
    e = rstd * (U32 * (2 * g + (RUN + 4) * m1) + xh * em2 + exh * m2 + 4 * U32 * (g + m1 + xh * m2))
    size = rstd * (g + m1 + xh * m2)
    d = 0.0 if dsum is None else f64(dsum).abs()
    dx, dw, db = layer_norm_backward(dy, x, w, mean[..., 0], rstd[..., 0], dsum)
    D = x.shape[-1]
    bx = u(dtype) * dx.abs() + (1 + u(dtype)) * (e + U32 * (size + d)) + 1e-37
    sw = (dy.abs() * xh).reshape(-1, D).sum(0)
    bw = u(wdtype) * dw.abs() + (rows_run + 2) * U32 * sw + (dy.abs() * exh).reshape(-1, D).sum(0) + 1e-37
    bb = u(wdtype) * db.abs() + (rows_run + 2) * U32 * dy.abs().reshape(-1, D).sum(0) + 1e-37
    return bx, bw, bb


def norm_gate_backward(dy, o, gate, eps):
    """(do [B, H, N, dv], dgate [B, N, H, dv])"""
    dy, o, g = f64(dy).transpose(1, 2), f64(o), f64(gate).transpose(1, 2)
    r = 1.0 / torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
    sig = torch.sigmoid(g)
    t = dy * g * sig
    do = r * t - o * r ** 3 * (t * o).mean(-1, keepdim=True)
    dg = dy * o * r * (sig + g * sig * (1 - sig))
    return do, dg.transpose(1, 2)


def norm_gate_backward_bounds(dy, o, gate, eps, dtype):
    """The sigmoid is within 2^-21 (hardware exponential and reciprocal, |g| up to 16 counted in the
    exponent's rounding: |g| log2(e) u(f32) of it); the rest are fp32 products and row sums."""
    RUN = run(o.shape[-1])
    do, dg = norm_gate_backward(dy, o, gate, eps)
    dy, o, g = f64(dy).transpose(1, 2), f64(o).abs(), f64(gate).transpose(1, 2)
    r = 1.0 / torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
    sig = torch.sigmoid(g)
    es = 2.0 ** -21 + 2 * g.abs() * U32  # relative, of sig
    t = (dy * g * sig).abs()
    m = (t * o).mean(-1, keepdim=True)
    em = (t * o * es).mean(-1, keepdim=True) + (RUN + 4) * U32 * m
    rr = (RUN / 2 + 6) * U32  # relative, of r
    e = r * t * (es + rr + 4 * U32) + o * r ** 3 * (em + m * (3 * rr + 8 * U32))
    bo = u(dtype) * do.abs() + (1 + u(dtype)) * e + 1e-37
    # sig (1 - sig): 1 - sig is off by es sig + u
    ds = es * sig + g.abs() * (es * sig * (1 - sig) + sig * (es * sig + U32)) + 6 * U32 * (sig + g.abs() * sig)
    eg = dy.abs() * o * r * (ds + (rr + 4 * U32) * (sig + g.abs() * sig))
    bg = (u(dtype) * dg.abs().transpose(1, 2) + (1 + u(dtype)) * eg + 1e-37).transpose(1, 2)
    return bo, bg


def assert_within(got, want, bound, what=""):
    got = f64(got)
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}, want {tuple(want.shape)}"
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got - want).abs() / bound).max().item() if got.numel() else 0.0
    assert over <= 1.0, f"{what}: {over:.3f} of the bound"
