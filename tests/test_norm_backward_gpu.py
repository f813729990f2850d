"""The gradients of the output epilogue on the GPU against the plain 64-bit forms."""
import pytest
import torch

from linear_attention_ret_b200 import inputs as I
from tests import plain64 as P

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
bf, f32 = torch.bfloat16, torch.float32
EPS = 1e-5

CASES = [
    # B, H, N, dv
    (2, 8, 37, 512),   # 1.3B-shaped heads
    (1, 1, 1, 512),    # one row
    (3, 2, 41, 128),
    (2, 3, 9, 64),
    (1, 5, 7, 8),
    (1, 2, 6, 2048),
    (1, 2, 5, 4096),
    (2, 3, 11, 99),    # odd rows
    (1, 2, 13, 100),
    (1, 3, 4, 40),
    (2, 1, 3, 1),
    (1, 2, 3, 1023),
]


def inputs(B, H, N, dv, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + 1)
    o = I.retention_output(B, H, N, dv, dtype, seed=seed).to(DEV)
    gate = (2 * I.gate_projection(B, H, N, dv, torch.float32, seed=seed)).to(dtype).to(DEV)
    dy = torch.randn(B, N, H, dv, generator=g).to(dtype).to(DEV)
    return dy, o, gate


def check(ret, dy, o, gate, eps=EPS):
    got = ret.msr_norm_gate_backward(dy, o, gate, eps)
    want = P.norm_gate_backward(dy, o, gate, eps)
    for name, g, w, b in zip(("do", "dgate"), got, want, P.norm_gate_backward_bounds(dy, o, gate, eps, o.dtype)):
        P.assert_within(g, w, b, name)
    return got


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("B,H,N,dv", CASES)
def test_matches_plain(cuda_lib, B, H, N, dv, dtype):
    check(cuda_lib, *inputs(B, H, N, dv, dtype))


def test_eps_and_zero_rows(cuda_lib):
    dy, o, gate = inputs(1, 2, 5, 64, f32)
    check(cuda_lib, dy, o, gate, 0.0)
    check(cuda_lib, dy, o, gate, 10.0)
    o[0, 1, 3] = 0.0  # u / sqrt(eps), no gradient of the gate
    do, dg = check(cuda_lib, dy, o, gate)
    assert not dg[0, 3, 1].any() and do[0, 1, 3].any()


def test_saturated_gates(cuda_lib):
    dy, o, gate = inputs(1, 1, 4, 64, f32)
    gate[0, 0], gate[0, 1] = 200.0, -200.0
    do, dg = cuda_lib.msr_norm_gate_backward(dy, o, gate, EPS)
    want_o, want_g = P.norm_gate_backward(dy, o, gate, EPS)
    assert torch.isfinite(do).all() and torch.isfinite(dg).all()
    # swish(200) = 200 and swish'(200) = 1 to fp32; at -200 both vanish
    assert torch.allclose(do.double().cpu()[0, 0, 0], want_o[0, 0, 0], rtol=1e-4, atol=1e-4)
    assert torch.allclose(dg.double().cpu()[0, 0], want_g[0, 0], rtol=1e-5, atol=1e-6)
    assert not do[0, 0, 1].any() and not dg[0, 1].any()


def test_non_finite_rows_stay_alone(cuda_lib):
    for dv in (64, 99):
        dy, o, gate = inputs(1, 2, 6, dv, bf)
        do, dg = cuda_lib.msr_norm_gate_backward(dy, o, gate, EPS)
        dy[0, 2, 1, 3] = float("nan")
        do2, dg2 = cuda_lib.msr_norm_gate_backward(dy, o, gate, EPS)
        keep = torch.ones(1, 2, 6, dtype=torch.bool, device=DEV)
        keep[0, 1, 2] = False
        assert torch.equal(do2[keep], do[keep]) and torch.isnan(do2[0, 1, 2]).all()
        assert torch.equal(dg2.transpose(1, 2)[keep], dg.transpose(1, 2)[keep])


@pytest.mark.parametrize("dv", [256, 99])
def test_in_place(cuda_lib, dv):
    dy, o, gate = inputs(2, 3, 7, dv, bf)
    do, dg = cuda_lib.msr_norm_gate_backward(dy, o, gate, EPS)
    for place in ("dy", "gate"):
        t = dict(dy=dy.clone(), gate=gate.clone(), o=o.clone())
        a, b = cuda_lib.msr_norm_gate_backward(t["dy"], t["o"], t["gate"], EPS, dout=t["o"], dgate=t[place])
        assert torch.equal(a, do) and torch.equal(b, dg) and b.data_ptr() == t[place].data_ptr()


def test_views_off_vector_alignment(cuda_lib):
    dy, o, gate = inputs(1, 2, 5, 64, bf)
    n = o.numel()

    def shifted(t):
        buf = torch.empty(n + 1, dtype=bf, device=DEV)
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)

    want = cuda_lib.msr_norm_gate_backward(dy, o, gate, EPS)
    got = check(cuda_lib, shifted(dy), shifted(o), shifted(gate))
    for g, w, b in zip(got, want, P.norm_gate_backward_bounds(dy, o, gate, EPS, bf)):
        assert ((g.double() - w.double()).abs().cpu() <= 2 * b).all()


def test_no_tokens(cuda_lib):
    o, g = torch.empty(1, 2, 0, 64, device=DEV), torch.empty(1, 0, 2, 64, device=DEV)
    do, dg = cuda_lib.msr_norm_gate_backward(g, o, g)
    assert do.shape == o.shape and dg.shape == g.shape


def test_64_bit_offsets(cuda_lib):
    """Rows behind 2^31 elements: token-major and head-major."""
    B, H, N, dv = 2, 1, (1 << 21) + 3, 512
    o = torch.zeros(B, H, N, dv, dtype=bf, device=DEV)
    gate, dy = torch.zeros(B, N, H, dv, dtype=bf, device=DEV), torch.zeros(B, N, H, dv, dtype=bf, device=DEV)
    tdy, to, tg = inputs(1, H, 3, dv, bf)
    o[1, :, -3:], gate[1, -3:], dy[1, -3:] = to[0], tg[0], tdy[0]
    do, dg = cuda_lib.msr_norm_gate_backward(dy, o, gate, EPS, dout=o, dgate=gate)
    want = cuda_lib.msr_norm_gate_backward(tdy, to, tg, EPS)
    assert torch.equal(do[1:, :, -3:], want[0]) and torch.equal(dg[1:, -3:], want[1])
    assert not do[0].any() and not dg[0].any()
