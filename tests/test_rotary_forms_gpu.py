"""The rotary prologue's kernels for few heads over many tokens (a thread's rows are of several tokens) and for
heads wider than a block's units (a thread per pair), against the plain 64-bit form."""
import pytest
import torch

from linear_attention_ret_b200.rotary import frequencies
from tests.test_rotary_gpu import DEV, bf, check, f32, randn

pytestmark = pytest.mark.gpu

KW = dict(q_scale=0.75, amplitude=1.1, offset=3)

# B, N, Hq, Hk, d, rot: one to three heads and more tokens than two blocks per SM of 4 (256 / (heads x units))
# tokens each take, no whole number of blocks
FEW_HEADS = [
    (1, 9475, 1, 1, 128, 128),
    (2, 4801, 2, 2, 64, 64),
    (1, 9501, 3, 1, 40, 24),    # fewer key heads, partly rotated
    (1, 9501, 1, 3, 40, 24),    # more key heads
    (3, 3301, 2, 0, 33, 32),    # no k, single elements
    (1, 2401, 2, 1, 99, 64),
    (1, 1203, 3, 3, 256, 256),
    (1, 37891, 1, 1, 32, 32),
    (1, 9501, 1, 2, 100, 50),   # pairs of bf16
    (1, 14301, 1, 2, 40, 24),
]

# heads of more units than a block has threads, for q and k together
WIDE_HEADS = [
    (2, 13, 2, 1, 515, 300),
    (1, 7, 3, 0, 1031, 514),
    (1, 3, 1, 2, 517, 2),
    (2, 3, 2, 2, 513, 0),       # nothing to rotate
    (1, 700, 1, 1, 259, 258),
]


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("B,N,Hq,Hk,d,rot", FEW_HEADS + WIDE_HEADS)
def test_matches_plain(cuda_lib, B, N, Hq, Hk, d, rot, dtype, layout):
    q = randn(B, N, Hq, d, dtype=dtype)
    k = randn(B, N, Hk, d, dtype=dtype, seed=1) if Hk else None
    kw = dict(KW, layout=layout, k_scale=d ** -0.5)
    check(cuda_lib, q, k, rot, kw, dtype)
    hq, hk = (None if t is None else t.transpose(1, 2).contiguous() for t in (q, k))
    check(cuda_lib, hq, hk, rot, kw, dtype, back=True)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("N,d,rot,shift", [(9501, 64, 32, 0), (9501, 33, 20, 0), (11, 515, 300, 0), (9, 300, 200, 1)])
def test_in_place_and_positions(cuda_lib, N, d, rot, shift, dtype, layout):
    """Slices of a fused buffer turned in place, one start per sequence; shift: off 16 bytes, so that 300 elements
    too take a thread per pair."""
    B, Hq, Hk = 2, 2, 1
    buf = randn(B, N, (Hq + Hk) * d + shift, dtype=dtype)
    q = buf[..., shift:shift + Hq * d].unflatten(-1, (Hq, d))
    k = buf[..., shift + Hq * d:].unflatten(-1, (Hk, d))
    edge = buf[..., :shift].clone()
    starts = torch.tensor([7, 1 << 20], device=DEV)
    kw = dict(layout=layout, starts=starts)
    want = check(cuda_lib, q, k, rot, kw, dtype)
    got = cuda_lib.rotary(q, k, frequencies(rot)[0].to(DEV), q_out=q.transpose(1, 2), k_out=k.transpose(1, 2), **kw)
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0].transpose(1, 2)) and torch.equal(k, want[1].transpose(1, 2))
    assert torch.equal(buf[..., :shift], edge)
