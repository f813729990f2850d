"""Layer norm on the GPU beyond test_layer_norm_gpu.py: the sum without a residual through the C ABI."""
import ctypes

import pytest
import torch

from tests import plain64 as P
from tests.test_layer_norm_gpu import DEV, EPS, bf, f32, randn

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
