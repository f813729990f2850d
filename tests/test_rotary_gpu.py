"""The rotary prologue on the GPU against its plain 64-bit form: pair layouts, partly rotated heads,
odd sizes, strided views (slices of a fused projection, head-major, expanded), positions, in-place
calls, and its inverse as gradient."""
import pytest
import torch

from linear_attention_ret_b200.rotary import frequencies
from tests import plain64 as P

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
bf, f32 = torch.bfloat16, torch.float32


def randn(*shape, dtype=f32, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def check(ret, q, k, rot, kw, dtype, back=False, call=None, what=""):
    """One call against the plain form; q, k are token-major (back: head-major) device views."""
    freqs = frequencies(rot)[0].to(DEV) if rot else None
    tok = (lambda t: t.transpose(1, 2)) if back else (lambda t: t)
    B, N = tok(q).shape[:2]
    got = (call or (ret.rotary_backward if back else ret.rotary))(q, k, freqs, **kw)
    pos = P.positions(B, N, kw.get("positions"), kw.get("starts"), kw.get("offset", 0))
    for name, t, o in (("q", q, got[0]), ("k", k, got[1])):
        if t is None:
            assert o is None
            continue
        y, size = P.rotate(tok(t), freqs, pos, kw.get("layout", "interleaved"), kw.get("amplitude", 1.0),
                           kw.get(name + "_scale", 1.0), back)
        o = o if back else o.transpose(1, 2)
        P.assert_within(o, y, P.rotate_bound(y, size, dtype), f"{what} {name}")
    return got


CASES = [
    # B, N, Hq, Hk, d, rot
    (2, 37, 8, 8, 256, 256),    # the 1.3B-shaped heads
    (1, 1, 16, 16, 256, 256),   # one token
    (3, 5, 4, 2, 128, 64),      # half of the head, fewer key heads
    (2, 9, 3, 3, 72, 36),       # a half of 18: no whole vectors in the half layout
    (1, 7, 2, 5, 66, 2),        # one pair, then 64 elements as they are
    (2, 3, 1, 1, 7, 6),         # odd head: rows of every alignment
    (1, 4, 2, 0, 33, 32),       # no k
    (1, 3, 2, 2, 1, 0),         # nothing to rotate, one element
    (1, 2, 3, 3, 264, 200),     # wider than retention's heads; a half of 100
    (70, 1, 5, 5, 64, 64),      # many sequences of one token
    (1, 1500, 1, 1, 32, 32),    # long and narrow
]


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("B,N,Hq,Hk,d,rot", CASES)
def test_rotary_matches_plain(cuda_lib, B, N, Hq, Hk, d, rot, dtype, layout):
    q = randn(B, N, Hq, d, dtype=dtype)
    k = randn(B, N, Hk, d, dtype=dtype, seed=1) if Hk else None
    kw = dict(layout=layout, q_scale=0.75, k_scale=d ** -0.5, amplitude=1.1, offset=3)
    out = check(cuda_lib, q, k, rot, kw, dtype)
    assert all(t is None or t.is_contiguous() for t in out)
    hq, hk = (None if t is None else t.transpose(1, 2).contiguous() for t in (q, k))
    out = check(cuda_lib, hq, hk, rot, kw, dtype, back=True)
    assert all(t is None or t.is_contiguous() for t in out)
    assert cuda_lib.last_device_error() == 0


@pytest.mark.parametrize("dtype", [bf, f32])
def test_positions(cuda_lib, dtype):
    B, N, H, d = 3, 11, 2, 64
    q, k = randn(B, N, H, d, dtype=dtype), randn(B, N, H, d, dtype=dtype, seed=1)
    g = torch.Generator().manual_seed(2)
    starts = torch.tensor([0, 1 << 20, (1 << 24) - 5], device=DEV)
    at = torch.randint(-(1 << 20), 1 << 24, (B, N), generator=g).to(DEV)
    for kw in (dict(), dict(offset=1 << 22), dict(starts=starts), dict(starts=starts, offset=-7), dict(positions=at),
               dict(positions=at, offset=12)):
        check(cuda_lib, q, k, d, kw, dtype, what=str(list(kw)))
        check(cuda_lib, q.transpose(1, 2).contiguous(), k.transpose(1, 2).contiguous(), d, kw, dtype, back=True)


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("pad", [0, 1, 4, 8])
def test_views(cuda_lib, dtype, layout, pad):
    """q and k inside a fused projection whose rows start at every alignment; outputs inside one buffer too."""
    B, N, H, d = 2, 6, 3, 64
    buf = randn(B, N, 3 * H * d + 2 * pad, dtype=dtype)
    q = buf[..., pad:pad + H * d].unflatten(-1, (H, d))
    k = buf[..., pad + H * d:pad + 2 * H * d].unflatten(-1, (H, d))
    kw = dict(layout=layout)
    check(cuda_lib, q, k, d, kw, dtype)
    # head-major inputs as views, and an expanded input: one row for all batches and heads
    hq = randn(B, H, N, d, dtype=dtype, seed=3)
    row = randn(1, N, 1, d, dtype=dtype, seed=4).expand(B, N, H, d)
    check(cuda_lib, hq.transpose(1, 2), row, d, kw, dtype)
    # the gradient into slices of a fused gradient; what lies beside them stays
    dq, dk = randn(B, H, N, d, dtype=dtype, seed=5), randn(B, H, N, d, dtype=dtype, seed=6)
    fused = torch.full_like(buf, 7.0)
    oq = fused[..., pad:pad + H * d].unflatten(-1, (H, d))
    ok = fused[..., pad + H * d:pad + 2 * H * d].unflatten(-1, (H, d))
    check(cuda_lib, dq, dk, d, kw, dtype, back=True,
          call=lambda *a, **w: cuda_lib.rotary_backward(*a, dq_out=oq, dk_out=ok, **w))
    assert (fused[..., :pad] == 7).all() and (fused[..., pad + 2 * H * d:] == 7).all()


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_in_place(cuda_lib, layout):
    B, N, H, d = 2, 6, 3, 64
    freqs = frequencies(48)[0].to(DEV)
    buf = randn(B, N, 2 * H * d, dtype=bf)
    want = cuda_lib.rotary(buf[..., :H * d].unflatten(-1, (H, d)), buf[..., H * d:].unflatten(-1, (H, d)), freqs,
                           layout=layout)
    q, k = buf[..., :H * d].unflatten(-1, (H, d)), buf[..., H * d:].unflatten(-1, (H, d))
    got = cuda_lib.rotary(q, k, freqs, layout=layout, q_out=q.transpose(1, 2), k_out=k.transpose(1, 2))
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0].transpose(1, 2)) and torch.equal(k, want[1].transpose(1, 2))


def test_layout_only_and_empty(cuda_lib):
    v = randn(2, 5, 3, 40, dtype=bf)
    out, none = cuda_lib.rotary(v, None, None)
    assert none is None and torch.equal(out, v.transpose(1, 2))
    back, _ = cuda_lib.rotary_backward(out, None, None)
    assert torch.equal(back, v)
    e = torch.empty(2, 0, 3, 40, dtype=bf, device=DEV)
    q, k = cuda_lib.rotary(e, e, frequencies(40)[0].to(DEV))
    assert q.shape == (2, 3, 0, 40) and k.shape == (2, 3, 0, 40)


def test_non_finite_values_stay_in_their_pairs(cuda_lib):
    q = randn(1, 2, 2, 64, dtype=bf)
    q[0, 1, 0, 6] = float("inf")
    q[0, 0, 1, 9] = float("nan")
    out, _ = cuda_lib.rotary(q, None, frequencies(64)[0].to(DEV), offset=1)
    bad = ~torch.isfinite(out.transpose(1, 2))
    want = torch.zeros_like(bad)
    want[0, 1, 0, 6:8] = True
    want[0, 0, 1, 8:10] = True
    assert torch.equal(bad, want)


def test_overlaps_are_refused(cuda_lib):
    q = randn(1, 6, 2, 32, dtype=bf)
    f = frequencies(32)[0].to(DEV)
    for kw in (dict(q_out=q.view(1, 2, 6, 32)),                  # the input's memory in another order
               dict(q_out=torch.empty(1, 1, 6, 32, dtype=bf, device=DEV).expand(1, 2, 6, 32))):
        with pytest.raises(cuda_lib.RetError) as e:
            cuda_lib.rotary(q, None, f, **kw)
        assert e.value.code == 4
    out = torch.empty(1, 2, 6, 32, dtype=bf, device=DEV)
    with pytest.raises(cuda_lib.RetError):
        cuda_lib.rotary(q, q, f, q_out=out, k_out=out)


def test_64_bit_offsets(cuda_lib):
    """Elements behind 2^32 bytes and 2^31 elements of a strided buffer."""
    N, d, row = 3, 64, 1 << 30
    buf = torch.zeros(2 * row + row // 2, dtype=bf, device=DEV)
    q = torch.as_strided(buf, (1, N, 1, d), (d, row, d, 1))
    q.copy_(randn(1, N, 1, d, dtype=bf))
    check(cuda_lib, q, None, d, dict(offset=5), bf)
