"""Layer norm on the GPU beyond test_layer_norm_gpu.py: the sum without a residual through the C ABI, and the
backward of rows whose mean is far from zero, and sizes at which every block takes many rows."""
import ctypes

import pytest
import torch

from tests import plain64 as P
from tests.test_layer_norm_gpu import DEV, EPS, backward_check, bf, f32, forward_check, randn

pytestmark = pytest.mark.gpu


def abi_forward(ret, x, y, sum_out):
    """ret_layer_norm without residual, weight, bias and statistics, as a C caller makes it."""
    p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())
    rows, D = x.shape
    dt = 1 if x.dtype == bf else 0
    return ret.load().ret_layer_norm(p(x), None, None, None, p(y), p(sum_out), None, None, rows, D, EPS, dt, dt,
                                     ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("rows,D", [(5, 3), (4000, 96), (70, 500), (9, 771), (1300, 1024), (33, 4098), (3, 9361),
                                    (5, 16384), (2, 20000)])
def test_sum_without_residual_is_x(cuda_lib, rows, D, dtype):
    x = randn(rows, D, dtype=dtype)
    want, total, _, _ = P.layer_norm(x, None, None, EPS)
    bound = P.layer_norm_bound(total, None, None, EPS, dtype)
    y, s = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    assert abi_forward(cuda_lib, x, y, s) == 0
    assert torch.equal(s, x)
    P.assert_within(y, want, bound)
    # in place: y over x, the sum beside it; and the sum over x itself
    a, s = x.clone(), torch.full_like(x, 7.0)
    assert abi_forward(cuda_lib, a, a, s) == 0
    assert torch.equal(s, x) and torch.equal(a, y)
    a, z = x.clone(), torch.full_like(x, 7.0)
    assert abi_forward(cuda_lib, a, z, a) == 0
    assert torch.equal(a, x) and torch.equal(z, y)


# ---------------------------------------------------------------- the backward's centred values

def centred_check(ret, dy, x, w, mean, rstd, dsum, dtype, wdtype):
    """The bounds of plain64 with x - mean for x and 0 for the mean: xh is then held to roundings of itself (the
    difference and the product with rstd), whatever the mean's size."""
    got = ret.layer_norm_backward(dy, x, w, mean, rstd, dsum=dsum)
    c, zero = P.f64(x) - P.f64(mean)[:, None], torch.zeros_like(mean)
    want = P.layer_norm_backward(dy, c, w, zero, rstd, dsum)
    bounds = P.layer_norm_backward_bounds(dy, c, w, zero, rstd, dsum, dtype, wdtype, min(len(x), 1300))
    for name, g, ref, bound in zip(("dx", "dweight", "dbias"), got, want, bounds):
        P.assert_within(g, ref, bound, name)
    return got


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("rows,D", [(5, 128), (40, 99), (7, 500), (4, 1023), (300, 771), (3, 4096), (3, 8191), (2, 12288),
                                    (3, 9361), (2, 20000)])
def test_backward_with_a_mean_far_from_zero(cuda_lib, rows, D, dtype, residual):
    x, w = randn(rows, D, dtype=dtype, shift=1000.0), 1 + 0.3 * randn(D, seed=1)
    dy = randn(rows, D, dtype=dtype, seed=2)
    dsum = randn(rows, D, dtype=dtype, seed=3) if residual else None
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    cuda_lib.layer_norm(x, w, mean=mean, rstd=rstd)
    centred_check(cuda_lib, dy, x, w, mean, rstd, dsum, dtype, f32)


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("D", [3, 40, 100, 259, 771, 4100, 8191, 9361, 20000])
def test_backward_of_constant_rows(cuda_lib, D, dtype):
    """x - mean is 0 exactly: no gradient of the weight, however large the constant (columns behind the row too
    must stay out of the sums: there x reads as 0, and (0 - 1e37) / sqrt(eps) is not finite)."""
    rows = 6
    for value in (1000.0, 1e37):
        x = torch.full((rows, D), value, device=DEV).to(dtype)
        mean, rstd = x[:, 0].float().contiguous(), torch.full((rows,), EPS ** -0.5, device=DEV)
        dy, w = randn(rows, D, dtype=dtype, seed=2), 1 + 0.3 * randn(D, seed=1)
        _, dw, _ = centred_check(cuda_lib, dy, x, w, mean, rstd, None, dtype, f32)
        assert not dw.any()


# ---------------------------------------------------------------- many rows per block

# Blocks stay and take row after row: enough rows that every block goes round its slots in shared memory more
# than once (two to four slots; up to sixteen small blocks per SM). Widths of one vector up to a pair of blocks.
MANY = [(230000, 40), (60000, 99), (60000, 100), (12000, 771), (9189, 1023), (12000, 1024), (4000, 2050), (3000, 4096),
        (3000, 6001), (700, 9361), (1000, 16384)]


@pytest.fixture
def plain_on_device(monkeypatch):
    """The plain 64-bit forms where the tensors are: these cases are large."""
    monkeypatch.setattr(P, "f64", lambda t: None if t is None else t.detach().double())


@pytest.mark.parametrize("dtype,wdtype", [(bf, f32), (f32, f32)], ids=["bf16", "fp32"])
@pytest.mark.parametrize("rows,D", MANY)
def test_many_rows_per_block(cuda_lib, plain_on_device, rows, D, dtype, wdtype):
    forward_check(cuda_lib, rows, D, dtype, wdtype, residual=True, seed=10)
    backward_check(cuda_lib, rows, D, dtype, wdtype)
    dy, x, w, mean, rstd, dsum, got = backward_check(cuda_lib, rows, D, dtype, wdtype, residual=True, seed=20)
    again = cuda_lib.layer_norm_backward(dy, x, w, mean, rstd, dsum=dsum)
    assert all(torch.equal(a, g) for a, g in zip(again, got))
