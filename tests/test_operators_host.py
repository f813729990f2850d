"""The operators around retention on the CPU: the plain 64-bit forms against differences and
identities, the frequency tables, the refusals of the binding and of the C ABI (nothing is
launched), and the autograd wrappers' routing with the plain forms in the library's place."""
import ctypes

import pytest
import torch

from linear_attention_ret_b200 import autograd as A
from linear_attention_ret_b200 import ret
from linear_attention_ret_b200.rotary import frequencies
from tests import plain64 as P

bf, f32, f64 = torch.bfloat16, torch.float32, torch.float64


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=f64)


# ---------------------------------------------------------------- the plain forms

def _differences(fn, x, dy, h=1e-6):
    """d sum(dy * fn(x)) / dx by central differences."""
    g = torch.empty_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        up = (dy * fn(x)).sum()
        flat[i] = keep - h
        out[i] = (up - (dy * fn(x)).sum()) / (2 * h)
        flat[i] = keep
    return g


def test_plain_gradients_agree_with_differences():
    x, w, b, dy = randn(3, 7), 1 + 0.2 * randn(7, seed=1), randn(7, seed=2), randn(3, 7, seed=3)
    eps = 1e-3
    _, _, mean, rstd = P.layer_norm(x, w, b, eps)
    got = P.layer_norm_backward(dy, x, w, mean, rstd)
    want = (_differences(lambda t: P.layer_norm(t, w, b, eps)[0], x.clone(), dy),
            _differences(lambda t: P.layer_norm(x, t, b, eps)[0], w.clone(), dy),
            _differences(lambda t: P.layer_norm(x, w, t, eps)[0], b.clone(), dy))
    for g, ref in zip(got, want):
        assert torch.allclose(g, ref, rtol=1e-7, atol=1e-8)

    o, gate, dy = randn(2, 2, 3, 5), randn(2, 3, 2, 5, seed=4), randn(2, 3, 2, 5, seed=5)

    def fwd(o, gate):
        r = 1 / torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
        return gate * torch.sigmoid(gate) * (o * r).transpose(1, 2)

    do, dg = P.norm_gate_backward(dy, o, gate, eps)
    assert torch.allclose(do, _differences(lambda t: fwd(t, gate), o.clone(), dy), rtol=1e-7, atol=1e-8)
    assert torch.allclose(dg, _differences(lambda t: fwd(o, t), gate.clone(), dy), rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_plain_rotation(layout):
    freqs, _ = frequencies(6)
    pos = torch.tensor([[0, 5, -3, 1000]])
    x = randn(1, 4, 2, 9)
    y, _ = P.rotate(x, freqs, pos, layout, 1.0, 0.5)
    assert torch.equal(y[:, 0], 0.5 * x[:, 0])                # position 0
    assert torch.equal(y[..., 6:], 0.5 * x[..., 6:])          # behind the rotated part
    assert torch.allclose(P.rotate(2 * y, freqs, pos, layout, inverse=True)[0], x, atol=1e-12)
    dy = randn(1, 4, 2, 9, seed=1)
    want = _differences(lambda t: P.rotate(t, freqs, pos, layout, 1.3, 0.5)[0], x.clone(), dy)
    assert torch.allclose(P.rotate(dy, freqs, pos, layout, 1.3, 0.5, True)[0], want, atol=1e-7)
    # scores depend on the distance alone
    q, k = randn(1, 1, 1, 6), randn(1, 1, 1, 6, seed=2)
    s = [(P.rotate(q, freqs, torch.tensor([[n]]), layout)[0] * P.rotate(k, freqs, torch.tensor([[n - 4]]), layout)[0])
         .sum().item() for n in (4, 90, 5000)]
    assert s[1] == pytest.approx(s[0], abs=1e-10) and s[2] == pytest.approx(s[0], abs=1e-10)


def test_plain_layer_norm_is_torchs():
    x, r, w, b = randn(4, 11), randn(4, 11, seed=1), randn(11, seed=2), randn(11, seed=3)
    y, s, _, _ = P.layer_norm(x, w, b, 1e-5, r)
    assert torch.allclose(y, torch.nn.functional.layer_norm(x + r, (11,), w, b, 1e-5), atol=1e-12)
    assert torch.equal(s, x + r)


# ---------------------------------------------------------------- frequency tables

def test_frequencies():
    f, m = frequencies(8, 100.0)
    assert m == 1.0 and f.dtype == f64
    assert torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75], dtype=f64))
    f, _ = frequencies(8, 100.0, schedule="retnet")
    assert torch.allclose(f, torch.tensor([1.0, 100 ** (-1 / 3), 100 ** (-2 / 3), 0.01], dtype=f64))
    assert frequencies(2, schedule="retnet")[0].tolist() == [1.0]
    base, _ = frequencies(64)
    assert torch.allclose(frequencies(64, scaling="linear", factor=4.0)[0], base / 4)
    ntk, _ = frequencies(64, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and ntk[-1].item() == pytest.approx(base[-1].item() / 4)
    yarn, m = frequencies(64, scaling="yarn", factor=4.0, length=2048)
    turns = 2048 * base / (2 * torch.pi)
    assert torch.equal(yarn[turns >= 32], base[turns >= 32])
    assert torch.allclose(yarn[turns <= 1], base[turns <= 1] / 4) and (turns <= 1).any()
    mid = (turns > 1) & (turns < 32)
    assert ((yarn < base) & (yarn > base / 4))[mid].all()
    assert m == pytest.approx(0.1 * 1.3862943611198906 + 1)


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=0), dict(rot=4, base=0.0), dict(rot=4, factor=0.5),
                                dict(rot=4, schedule="x"), dict(rot=4, scaling="x"), dict(rot=4, scaling="yarn"),
                                dict(rot=2, scaling="ntk", factor=2.0),
                                dict(rot=8, schedule="retnet", scaling="ntk", factor=2.0)])
def test_frequencies_refusals(kw):
    with pytest.raises(ValueError):
        frequencies(**kw)


# ---------------------------------------------------------------- refusals of the binding

def _refused(match, fn, *args, **kw):
    with pytest.raises((ValueError, TypeError), match=match):
        fn(*args, **kw)


def test_binding_refusals():
    B, N, H, d = 2, 5, 3, 8
    q, k, f = torch.zeros(B, N, H, d, dtype=bf), torch.zeros(B, N, 2, d, dtype=bf), torch.ones(4, dtype=f64)
    at, st = torch.zeros(B, N, dtype=torch.int64), torch.zeros(B, dtype=torch.int64)
    for kw in (dict(), dict(positions=at), dict(starts=st, layout="half"), dict(q_out=q.transpose(1, 2))):
        _refused("CUDA tensors", ret.rotary, q, k, f, **kw)      # valid but for the device
    _refused("CUDA tensors", ret.rotary, q[:, :, :, :], None, None)
    _refused("CUDA tensors", ret.rotary_backward, q.transpose(1, 2), k.transpose(1, 2), f, dq_out=q)
    _refused("4 dimensions", ret.rotary, q[0], k, f)
    _refused("k must have shape", ret.rotary, q, k[:, :4], f)
    _refused("k must be", ret.rotary, q, k.float(), f)
    _refused("freqs must be", ret.rotary, q, k, f.float())
    _refused("rotates 10", ret.rotary, q, k, torch.ones(5, dtype=f64))
    _refused("positions must have shape", ret.rotary, q, k, f, positions=at[:, :3])
    _refused("positions must be", ret.rotary, q, k, f, positions=at.int())
    _refused("starts must have shape", ret.rotary, q, k, f, starts=at)
    _refused("not both", ret.rotary, q, k, f, starts=st, positions=at)
    _refused("layout", ret.rotary, q, k, f, layout="pairs")
    _refused("without k", ret.rotary, q, None, f, k_out=k.transpose(1, 2))
    _refused("output of q must have shape", ret.rotary, q, k, f, q_out=q)
    _refused("contiguous", ret.rotary, torch.zeros(B, N, H, 2 * d, dtype=bf)[..., ::2], k, f)
    _refused("unsupported dtype", ret.rotary, q.half(), k.half(), f)

    x, w = torch.zeros(4, 6, dtype=bf), torch.ones(6)
    m = torch.zeros(4)
    _refused("CUDA tensors", ret.layer_norm, x, w, w)
    _refused("CUDA tensors", ret.layer_norm, x, w.to(bf), None, residual=x, mean=m, rstd=m)
    _refused("CUDA tensors", ret.layer_norm_backward, x, x, w, m, m, dsum=x)
    _refused("one element", ret.layer_norm, torch.zeros(4, 0))
    _refused("one dimension", ret.layer_norm, torch.zeros(()))
    _refused("weight must have shape", ret.layer_norm, x, w[:5])
    _refused("weight and bias must be", ret.layer_norm, x, w.double())
    _refused("weight and bias must be", ret.layer_norm, x.float(), w.to(bf))
    _refused("share one dtype", ret.layer_norm, x, w, w.to(bf))
    _refused("residual must have shape", ret.layer_norm, x, w, residual=x[:3])
    _refused("residual must be", ret.layer_norm, x, w, residual=x.float())
    _refused("mean must have shape", ret.layer_norm, x, w, mean=m[:3])
    _refused("without a residual", ret.layer_norm, x, w, sum_out=x)
    _refused("unsupported dtype", ret.layer_norm, x.half(), w)
    _refused("dy must have shape", ret.layer_norm_backward, x[:2], x, w, m, m)
    _refused("rstd must be", ret.layer_norm_backward, x, x, w, m, m.double())
    _refused("wdtype", ret.layer_norm_backward, x, x, None, m, m, wdtype=f64)

    o, g = torch.zeros(B, H, N, d), torch.zeros(B, N, H, d)
    _refused("CUDA tensors", ret.msr_norm_gate_backward, g, o, g)
    _refused("gate must have shape", ret.msr_norm_gate_backward, g, o, o)
    _refused("dy must be", ret.msr_norm_gate_backward, g.to(bf), o, g)
    _refused("dout must have shape", ret.msr_norm_gate_backward, g, o, g, dout=g)


# ---------------------------------------------------------------- refusals of the C ABI

@pytest.fixture(scope="module")
def lib():
    from linear_attention_ret_b200 import build
    build.build()
    return ret.load()


BASE = 1 << 40  # addresses that are never dereferenced
OK, NULL, SHAPE, DTYPE, UNSUPPORTED, ALIGN = 0, 1, 2, 3, 4, 7


def p(at):
    return None if at is None else ctypes.c_void_p(at)


def _rot(lib, q=BASE, k=None, qo=2 * BASE, ko=None, sq=(640, 64, 16), sk=None, sqo=(640, 64, 16), sko=None,
         freqs=3 * BASE, positions=None, starts=None, B=2, N=10, Hq=4, Hk=0, d=16, rot=16, layout=0, amplitude=1.0,
         q_scale=1.0, dt=1):
    arr = lambda s: None if s is None else (ctypes.c_longlong * 3)(*s)
    return lib.ret_rotary(p(q), p(k), p(qo), p(ko), arr(sq), arr(sk), arr(sqo), arr(sko), p(freqs), p(positions),
                          p(starts), 0, B, N, Hq, Hk, d, rot, layout, 0, amplitude, q_scale, 1.0, dt, None)


def test_rotary_abi_refusals(lib):
    assert _rot(lib, dt=3) == DTYPE
    for bad in (dict(B=0), dict(N=-1), dict(Hq=0), dict(Hk=-1), dict(d=0), dict(rot=3), dict(rot=18), dict(rot=-2),
                dict(amplitude=float("inf")), dict(q_scale=float("nan")), dict(sq=(640, -64, 16))):
        assert _rot(lib, **bad) == SHAPE, bad
    assert _rot(lib, layout=2) == UNSUPPORTED
    assert _rot(lib, N=0, q=None) == OK
    for bad in (dict(q=None), dict(qo=None), dict(sq=None), dict(sqo=None), dict(freqs=None), dict(Hk=4)):
        assert _rot(lib, **bad) == NULL, bad
    assert _rot(lib, positions=4 * BASE, starts=5 * BASE) == UNSUPPORTED
    assert _rot(lib, q=BASE + 1) == ALIGN
    assert _rot(lib, sq=(1 << 60, 64, 16)) == UNSUPPORTED
    # outputs that write an element twice, or lie over an input, the other output or the tables
    for bad in (dict(sqo=(640, 64, 8)), dict(sqo=(0, 64, 16)), dict(sqo=(600, 64, 16)), dict(qo=BASE + 2),
                dict(qo=BASE, sqo=(640, 16, 160)), dict(qo=3 * BASE - 8), dict(positions=2 * BASE + 16),
                dict(starts=2 * BASE)):
        assert _rot(lib, **bad) == UNSUPPORTED, bad
    two = dict(k=4 * BASE, Hk=4, sk=(640, 64, 16), sko=(640, 64, 16))
    for bad in (dict(ko=2 * BASE), dict(ko=2 * BASE + 32), dict(ko=BASE), dict(ko=BASE + 64)):
        assert _rot(lib, **two, **bad) == UNSUPPORTED, bad
    # interleaved head-major views of one buffer are not seen to be disjoint
    assert _rot(lib, k=4 * BASE, Hk=4, sk=(640, 64, 16), sqo=(1280, 16, 320), sko=(1280, 16, 320),
                ko=2 * BASE + 320) == UNSUPPORTED


def test_layer_norm_abi_refusals(lib):
    def ln(x=BASE, res=None, w=None, b=None, y=2 * BASE, s=None, mean=None, rstd=None, rows=4, D=8, eps=1e-5, dt=1,
           wdt=0):
        return lib.ret_layer_norm(p(x), p(res), p(w), p(b), p(y), p(s), p(mean), p(rstd), rows, D, eps, dt, wdt, None)

    for bad in (dict(dt=2), dict(wdt=5), dict(dt=0, wdt=1)):
        assert ln(**bad) == DTYPE
    for bad in (dict(rows=-1), dict(D=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert ln(**bad) == SHAPE
    assert ln(rows=1 << 60) == UNSUPPORTED
    assert ln(rows=0, x=None) == OK
    assert ln(x=None) == NULL and ln(y=None) == NULL
    assert ln(x=BASE + 1) == ALIGN and ln(w=3 * BASE + 2) == ALIGN and ln(mean=3 * BASE + 1) == ALIGN
    for bad in (dict(y=BASE + 2), dict(s=2 * BASE), dict(s=BASE + 16), dict(res=3 * BASE, y=3 * BASE + 4),
                dict(w=2 * BASE), dict(mean=2 * BASE + 4), dict(mean=3 * BASE, rstd=3 * BASE), dict(mean=BASE)):
        assert ln(**bad) == UNSUPPORTED, bad

    def back(dy=BASE, x=2 * BASE, w=None, mean=3 * BASE, rstd=4 * BASE, dsum=None, dx=5 * BASE, dw=None, db=None,
             rows=4, D=8, dt=1, wdt=0):
        return lib.ret_layer_norm_backward(p(dy), p(x), p(w), p(mean), p(rstd), p(dsum), p(dx), p(dw), p(db), rows, D,
                                           dt, wdt, None)

    assert back(dt=2) == DTYPE and back(dt=0, wdt=1) == DTYPE
    assert back(rows=-1) == SHAPE and back(D=0) == SHAPE
    assert back(rows=0) == OK
    for name in ("dy", "x", "mean", "rstd", "dx"):
        assert back(**{name: None}) == NULL, name
    assert back(dw=6 * BASE + 2) == ALIGN
    for bad in (dict(dx=BASE + 2), dict(dx=2 * BASE + 32), dict(dx=3 * BASE), dict(dw=5 * BASE), dict(dw=BASE),
                dict(dw=6 * BASE, db=6 * BASE), dict(w=6 * BASE, dw=6 * BASE), dict(db=4 * BASE)):
        assert back(**bad) == UNSUPPORTED, bad


def test_norm_gate_backward_abi_refusals(lib):
    def f(dy=BASE, o=2 * BASE, g=3 * BASE, do=4 * BASE, dg=5 * BASE, B=1, H=2, N=8, dv=64, eps=1e-5, dt=1):
        return lib.ret_msr_norm_gate_backward(p(dy), p(o), p(g), p(do), p(dg), B, H, N, dv, eps, dt, None)

    assert f(dt=2) == DTYPE
    for bad in (dict(B=0), dict(H=0), dict(N=-1), dict(dv=0), dict(eps=-1.0), dict(eps=float("inf"))):
        assert f(**bad) == SHAPE
    assert f(N=0, dy=None) == OK
    for name in ("dy", "o", "g", "do", "dg"):
        assert f(**{name: None}) == NULL
    assert f(o=2 * BASE + 1) == ALIGN
    for bad in (dict(do=BASE), dict(do=3 * BASE), dict(do=2 * BASE + 2), dict(dg=2 * BASE), dict(dg=4 * BASE + 8),
                dict(dg=3 * BASE + 2), dict(dg=BASE + 2)):
        assert f(**bad) == UNSUPPORTED, bad


# ---------------------------------------------------------------- autograd routing

@pytest.fixture
def plain_library(monkeypatch):
    """The library's calls replaced by the plain forms, inside the test only."""
    def rotary(q, k, freqs, positions=None, starts=None, offset=0, layout="interleaved", amplitude=1.0, q_scale=1.0,
               k_scale=1.0):
        pos = P.positions(*q.shape[:2], positions, starts, offset)
        return tuple(None if t is None else P.rotate(t, freqs, pos, layout, amplitude, s)[0].transpose(1, 2)
                     for t, s in ((q, q_scale), (k, k_scale)))

    def rotary_backward(dq, dk, freqs, positions=None, starts=None, offset=0, layout="interleaved", amplitude=1.0,
                        q_scale=1.0, k_scale=1.0):
        pos = P.positions(dq.shape[0], dq.shape[2], positions, starts, offset)
        return tuple(None if t is None else P.rotate(t.transpose(1, 2), freqs, pos, layout, amplitude, s, True)[0]
                     for t, s in ((dq, q_scale), (dk, k_scale)))

    def layer_norm(x, weight=None, bias=None, eps=1e-5, residual=None, mean=None, rstd=None):
        y, s, m, r = P.layer_norm(x, weight, bias, eps, residual)
        mean.copy_(m)
        rstd.copy_(r)
        return y if residual is None else (y, s)

    def layer_norm_backward(dy, x, weight, mean, rstd, dsum=None, dweight=True, dbias=True, wdtype=None):
        assert weight is not None or wdtype in (None, f64)
        dx, dw, db = P.layer_norm_backward(dy, x, weight, mean, rstd, dsum)
        return dx, dw if dweight and weight is not None else None, db if dbias else None

    def norm_gate(o, gate, eps):
        r = 1 / torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
        return gate * torch.sigmoid(gate) * (o * r).transpose(1, 2)

    def chunkwise(q, k, v, decay, chunk, **_):
        n = torch.arange(q.shape[2])
        D = torch.where(n[:, None] >= n, decay[:, None, None] ** (n[:, None] - n).clamp(min=0), 0.0)
        return ((q @ k.transpose(-1, -2)) * D) @ v

    def chunkwise_backward(q, k, v, decay, do, chunk, gated=False, ddecay=True):
        with torch.enable_grad():
            leaves = [t.detach().requires_grad_() for t in (q, k, v, decay)]
            return torch.autograd.grad((chunkwise(*leaves, chunk) * do).sum(), leaves)

    for f in (rotary, rotary_backward, layer_norm, layer_norm_backward, chunkwise_backward):
        monkeypatch.setattr(ret, f.__name__, f)
    monkeypatch.setattr(ret, "msr_norm_gate", norm_gate)
    monkeypatch.setattr(ret, "msr_norm_gate_backward", P.norm_gate_backward)
    monkeypatch.setattr(ret, "ret_chunkwise", chunkwise)
    monkeypatch.setattr(ret, "empty_like", torch.empty_like, raising=False)


def _grads(fn, leaves):
    leaves = [t.clone().requires_grad_() for t in leaves]
    out = fn(*leaves)
    out = out if isinstance(out, tuple) else (out,)
    total = sum((o * randn(*o.shape, seed=50 + i)).sum() for i, o in enumerate(out) if o is not None)
    return torch.autograd.grad(total, leaves)


def _check_grads(fn, leaves, atol=1e-6):
    """The wrapper's gradients against central differences of its own forward."""
    got = _grads(fn, leaves)
    for i, g in enumerate(got):
        def scalar_fn(t):
            args = [l.clone() for l in leaves]
            args[i] = t
            with torch.no_grad():
                out = fn(*args)
            out = out if isinstance(out, tuple) else (out,)
            return sum((o * randn(*o.shape, seed=50 + j)).sum() for j, o in enumerate(out) if o is not None)
        want = _differences(scalar_fn, leaves[i].clone(), torch.ones((), dtype=f64))
        assert torch.allclose(g, want, rtol=1e-5, atol=atol), i


def test_rotary_routes_gradients(plain_library):
    freqs, _ = frequencies(4)
    q, k = randn(2, 3, 2, 6), randn(2, 3, 1, 6, seed=1)
    kw = dict(starts=torch.tensor([4, 9]), layout="half", amplitude=1.2, q_scale=0.5, k_scale=0.25)
    _check_grads(lambda q, k: A.rotary(q, k, freqs, **kw), [q, k])
    _check_grads(lambda q: A.rotary(q, None, freqs, **kw), [q])
    _check_grads(lambda q, k: A.rotary(q, k, freqs, **kw)[1] + 0 * q.sum(), [q, k])  # k's output alone
    _check_grads(lambda q, k: A.rotary(q, k, freqs, **kw)[0] + 0 * k.sum(), [q, k])  # q's output alone


def test_layer_norm_routes_gradients(plain_library):
    x, r, w, b = randn(2, 3, 5), randn(2, 3, 5, seed=1), randn(5, seed=2), randn(5, seed=3)
    _check_grads(lambda x, w, b: A.layer_norm(x, w, b, 1e-2), [x, w, b])
    _check_grads(lambda x, b: A.layer_norm(x, None, b, 1e-2), [x, b])
    _check_grads(lambda x: A.layer_norm(x, w, b, 1e-2), [x])
    _check_grads(lambda x, r, w: A.layer_norm(x, w, None, 1e-2, residual=r), [x, r, w])
    _check_grads(lambda x, r: A.layer_norm(x, w, None, 1e-2, residual=r)[1], [x, r])      # the sum alone
    _check_grads(lambda x, r: A.layer_norm(x, w, None, 1e-2, residual=r)[0], [x, r])      # y alone


def test_path_routes_gradients(plain_library):
    B, N, H, dk, dv = 1, 4, 2, 4, 3
    freqs, _ = frequencies(dk, schedule="retnet")
    leaves = [randn(B, N, H, dk), randn(B, N, H, dk, seed=1), randn(B, N, H, dv, seed=2), randn(B, N, H, dv, seed=3),
              torch.tensor([0.9, 0.5], dtype=f64)]
    _check_grads(lambda q, k, v, g, decay: A.multi_scale_retention(q, k, v, g, decay, freqs, eps=1e-2, k_scale=0.5),
                 leaves)


def test_second_backward_raises(plain_library):
    x = randn(2, 5).requires_grad_()
    g, = torch.autograd.grad(A.layer_norm(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


# ---------------------------------------------------------------- devices and streams

def test_calls_enter_the_tensors_device_and_the_given_stream(monkeypatch):
    class Stream:
        def __init__(self, device):
            self.device = device

    one, two = torch.device("cuda", 0), torch.device("cuda", 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda d: ("device", d))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: ("stream", s))
    assert ret._elsewhere(one, None) is None
    assert ret._elsewhere(two, None) == ("device", two)
    s = Stream(two)
    assert ret._elsewhere(two, s) == ("stream", s)
    with pytest.raises(ValueError, match="stream is on"):
        ret._elsewhere(one, s)
