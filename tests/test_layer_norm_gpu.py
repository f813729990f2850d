"""Layer norm, its residual form and its gradients on the GPU against the plain 64-bit forms."""
import pytest
import torch

from tests import plain64 as P

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
bf, f32 = torch.bfloat16, torch.float32
EPS = 1e-5


def randn(*shape, dtype=f32, seed=0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g)
    if len(shape) > 1:  # rows of different size
        x = x * torch.exp(torch.randn(*shape[:-1], 1, generator=g)) + shift
    return x.to(dtype).to(DEV)


# rows, D: one row, few rows, many; widths of one vector, below and above each kernel's reach, and odd ones
SIZES = [(1, 1), (20, 1), (3, 2), (21, 3), (2, 7), (5, 8), (1, 64), (7, 100), (65, 127), (9, 256), (300, 512), (33, 771), (17, 1023), (64, 1024),
         (1000, 1280), (40, 2048), (13, 2050), (129, 4096), (5, 5000), (37, 8192), (3, 8191), (4, 16384), (2, 16380)]
TYPES = [(bf, bf), (bf, f32), (f32, f32)]


def ids(v):
    return str(v).replace("torch.", "")


def forward_check(ret, rows, D, dtype, wdtype, affine=3, residual=False, shift=0.0, seed=0):
    x = randn(rows, D, dtype=dtype, seed=seed, shift=shift)
    w = (1 + 0.3 * randn(D, seed=seed + 1)).to(wdtype) if affine & 1 else None
    b = randn(D, dtype=wdtype, seed=seed + 2) if affine & 2 else None
    r = randn(rows, D, dtype=dtype, seed=seed + 3) if residual else None
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    out = ret.layer_norm(x, w, b, EPS, residual=r, mean=mean, rstd=rstd)
    y, s = out if residual else (out, None)
    want, total, mu, rs = P.layer_norm(x, w, b, EPS, r)
    P.assert_within(y, want, P.layer_norm_bound(total, w, b, EPS, dtype), "y")
    if residual:
        P.assert_within(s, total, P.u(dtype) * total.abs() + P.U32 * (1 + P.u(dtype)) * total.abs() + 1e-37, "sum")
    run, c = P.run(D), total.abs()
    bm = P.U32 * (2 * mu.abs() + run * c.mean(-1)) + 1e-37
    P.assert_within(mean, mu, bm, "mean")
    cen = (total - mu[:, None]).abs()
    ec = P.U32 * 2 * c + bm[:, None]
    br = rs * (P.U32 * (run / 2 + 6) + rs ** 2 * (cen * ec + ec ** 2).mean(-1))
    P.assert_within(rstd, rs, br, "rstd")
    return x, w, b, mean, rstd


@pytest.mark.parametrize("dtype,wdtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,D", SIZES)
def test_forward_matches_plain(cuda_lib, rows, D, dtype, wdtype):
    forward_check(cuda_lib, rows, D, dtype, wdtype)
    forward_check(cuda_lib, rows, D, dtype, wdtype, residual=True, seed=10)


@pytest.mark.parametrize("affine", [0, 1, 2])
@pytest.mark.parametrize("rows,D", [(5, 96), (3, 771), (6, 4096)])
def test_forward_without_weight_or_bias(cuda_lib, rows, D, affine):
    forward_check(cuda_lib, rows, D, bf, f32, affine=affine)
    forward_check(cuda_lib, rows, D, f32, f32, affine=affine, residual=True)


@pytest.mark.parametrize("rows,D", [(5, 128), (4, 1023), (3, 4096)])
def test_mean_far_from_zero(cuda_lib, rows, D):
    forward_check(cuda_lib, rows, D, f32, f32, shift=1000.0)


def test_constant_and_zero_rows(cuda_lib):
    x = torch.tensor([[0.0] * 64, [3.0] * 64, [1.0] + [0.0] * 63], device=DEV)
    b = randn(64)
    y = cuda_lib.layer_norm(x, None, b, EPS)
    assert torch.equal(y[0], b) and torch.equal(y[1], b)
    P.assert_within(y, P.layer_norm(x, None, b, EPS)[0], P.layer_norm_bound(P.f64(x), None, b, EPS, f32))
    one = cuda_lib.layer_norm(torch.tensor([[5.0], [-2.0]], device=DEV), eps=0.5)
    assert torch.equal(one, torch.zeros_like(one))


def test_non_finite_rows_stay_alone(cuda_lib):
    for D in (64, 1023, 4096):
        x = randn(9, D, dtype=bf)
        want = cuda_lib.layer_norm(x)
        x[3, 5], x[7, 0] = float("inf"), float("nan")
        got = cuda_lib.layer_norm(x)
        rest = [0, 1, 2, 4, 5, 6, 8]
        assert torch.equal(got[rest], want[rest])
        assert torch.isnan(got[7]).all() and not torch.isfinite(got[3]).any()


@pytest.mark.parametrize("rows,D", [(5, 96), (3, 771), (6, 4096), (2, 40000)])
def test_forward_in_place(cuda_lib, rows, D):
    x, r, w = randn(rows, D, dtype=bf), randn(rows, D, dtype=bf, seed=1), randn(D, seed=2)
    y, s = cuda_lib.layer_norm(x, w, residual=r)
    a, c = x.clone(), r.clone()
    cuda_lib.layer_norm(a, w, residual=c, y=a, sum_out=c)
    assert torch.equal(a, y) and torch.equal(c, s)
    a, c = x.clone(), r.clone()
    cuda_lib.layer_norm(a, w, residual=c, y=c, sum_out=a)
    assert torch.equal(c, y) and torch.equal(a, s)


@pytest.mark.parametrize("shift", [1, 2, 4])
def test_views_off_vector_alignment(cuda_lib, shift):
    """Contiguous tensors that do not start on 16 bytes."""
    rows, D = 6, 512
    buf = randn(rows * D + shift, dtype=bf)
    x = buf[shift:].view(rows, D)
    w = randn(D + shift, seed=1)[shift:]
    y = cuda_lib.layer_norm(x, w)
    want, total, mean, rstd = P.layer_norm(x, w, None, EPS)
    P.assert_within(y, want, P.layer_norm_bound(total, w, None, EPS, bf))
    m, r = mean.float().to(DEV), rstd.float().to(DEV)
    dy = randn(rows * D + shift, dtype=bf, seed=2)[shift:].view(rows, D)
    got = cuda_lib.layer_norm_backward(dy, x, w, m, r)
    bounds = P.layer_norm_backward_bounds(dy, x, w, m, r, None, bf, f32, rows)
    for g, ref, bound in zip(got, P.layer_norm_backward(dy, x, w, m, r), bounds):
        P.assert_within(g, ref, bound)


def backward_check(ret, rows, D, dtype, wdtype, weight=True, residual=False, seed=0):
    x, w, b, mean, rstd = forward_check(ret, rows, D, dtype, wdtype, affine=3 if weight else 2, seed=seed)
    dy = randn(rows, D, dtype=dtype, seed=seed + 5)
    dsum = randn(rows, D, dtype=dtype, seed=seed + 6) if residual else None
    got = ret.layer_norm_backward(dy, x, w, mean, rstd, dsum=dsum, wdtype=None if weight else wdtype)
    want = P.layer_norm_backward(dy, x, w, mean, rstd, dsum)
    # any order of the sums over rows: at most 1184 partial sums joined one after another, or rows of them
    bounds = P.layer_norm_backward_bounds(dy, x, w, mean, rstd, dsum, dtype, wdtype, min(rows, 1300))
    for name, g, ref, bound in zip(("dx", "dweight", "dbias"), got, want, bounds):
        if name == "dweight" and not weight:
            assert g is None
        else:
            P.assert_within(g, ref, bound, name)
    return dy, x, w, mean, rstd, dsum, got


@pytest.mark.parametrize("dtype,wdtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,D", SIZES)
def test_backward_matches_plain(cuda_lib, rows, D, dtype, wdtype):
    backward_check(cuda_lib, rows, D, dtype, wdtype)
    dy, x, w, mean, rstd, dsum, got = backward_check(cuda_lib, rows, D, dtype, wdtype, residual=True, seed=20)
    again = cuda_lib.layer_norm_backward(dy, x, w, mean, rstd, dsum=dsum)
    assert all(torch.equal(a, g) for a, g in zip(again, got))  # fixed order: bit for bit


@pytest.mark.parametrize("rows,D", [(4000, 64), (3000, 257), (2500, 1024), (1500, 770), (700, 9000), (300, 12289)])
def test_backward_of_many_rows(cuda_lib, rows, D):
    backward_check(cuda_lib, rows, D, bf, f32)
    backward_check(cuda_lib, rows, D, bf, f32, weight=False, residual=True)


def test_backward_parts_on_request(cuda_lib):
    dy, x, w, mean, rstd, _, (dx, dw, db) = backward_check(cuda_lib, 40, 512, bf, f32)
    a, none_w, none_b = cuda_lib.layer_norm_backward(dy, x, w, mean, rstd, dweight=False, dbias=False)
    assert none_w is None and none_b is None and torch.equal(a, dx)
    a, b, none_b = cuda_lib.layer_norm_backward(dy, x, w, mean, rstd, dbias=False)
    assert none_b is None and torch.equal(a, dx) and torch.equal(b, dw)
    a, none_w, c = cuda_lib.layer_norm_backward(dy, x, w, mean, rstd, dweight=False)
    assert none_w is None and torch.equal(a, dx) and torch.equal(c, db)


@pytest.mark.parametrize("rows,D", [(5, 96), (7, 771), (200, 2048), (2, 40000)])
def test_backward_in_place(cuda_lib, rows, D):
    dy, x, w, mean, rstd, dsum, got = backward_check(cuda_lib, rows, D, bf, f32, residual=True)
    for place in ("dy", "x", "dsum"):
        t = dict(dy=dy.clone(), x=x.clone(), dsum=dsum.clone())
        out = cuda_lib.layer_norm_backward(t["dy"], t["x"], w, mean, rstd, dsum=t["dsum"], dx=t[place])
        assert out[0].data_ptr() == t[place].data_ptr()
        assert all(torch.equal(a, g) for a, g in zip(out, got)), place


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("rows,D", [(300, 1023), (40, 5), (150, 6001)])
def test_in_place_at_odd_widths(cuda_lib, rows, D, dtype):
    """Rows that start on no 16 bytes share units of memory with their neighbours."""
    dy, x, w, mean, rstd, dsum, got = backward_check(cuda_lib, rows, D, dtype, f32, residual=True)
    out = cuda_lib.layer_norm_backward(dy, x, w, mean, rstd, dsum=dsum, dx=dy)
    assert all(torch.equal(a, g) for a, g in zip(out, got))
    y, s = cuda_lib.layer_norm(x, w, residual=dsum)
    a, c = x.clone(), dsum.clone()
    cuda_lib.layer_norm(a, w, residual=c, y=a, sum_out=c)
    assert torch.equal(a, y) and torch.equal(c, s)


def test_no_rows(cuda_lib):
    x, w = torch.empty(0, 64, dtype=bf, device=DEV), randn(64)
    m = torch.empty(0, device=DEV)
    assert cuda_lib.layer_norm(x, w).shape == (0, 64)
    dx, dw, db = cuda_lib.layer_norm_backward(x, x, w, m, m)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_leading_shape(cuda_lib):
    x, w = randn(2, 3, 4, 64, dtype=bf), randn(64)
    mean, rstd = torch.empty(2, 3, 4, device=DEV), torch.empty(2, 3, 4, device=DEV)
    y = cuda_lib.layer_norm(x, w, mean=mean, rstd=rstd)
    assert torch.equal(y.view(24, 64), cuda_lib.layer_norm(x.view(24, 64), w))
    dx, _, _ = cuda_lib.layer_norm_backward(y, x, w, mean, rstd)
    assert dx.shape == x.shape


def test_64_bit_offsets(cuda_lib):
    """Rows behind 2^32 bytes and 2^31 elements."""
    rows, D = (1 << 19) + 9, 4096
    x = torch.zeros(rows, D, dtype=bf, device=DEV)
    last = randn(9, D, dtype=bf)
    x[-9:] = last
    w = randn(D)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    y = cuda_lib.layer_norm(x, w, mean=mean, rstd=rstd)
    assert torch.equal(y[-9:], cuda_lib.layer_norm(last, w)) and not y[:100].any()
    dx, dw, db = cuda_lib.layer_norm_backward(x, x, w, mean, rstd, dx=y)
    want = P.layer_norm_backward(last, last, w, mean[-9:], rstd[-9:])
    bounds = P.layer_norm_backward_bounds(last, last, w, mean[-9:], rstd[-9:], None, bf, f32, 1300)
    for g, ref, bound in zip((dx[-9:], dw, db), want, bounds):
        P.assert_within(g, ref, bound)
