"""Refusals of the operators around retention beyond test_operators_host.py, and the device that calls enter:
nothing is launched."""
import torch

from linear_attention_ret_b200 import ret
from tests.test_operators_host import ALIGN, BASE, UNSUPPORTED, _rot, lib, p  # noqa: F401 - lib is a fixture


def test_rotary_tables_must_be_aligned(lib):
    for bad in (dict(freqs=3 * BASE + 4), dict(freqs=3 * BASE + 1), dict(positions=4 * BASE + 4),
                dict(starts=5 * BASE + 2)):
        assert _rot(lib, **bad) == ALIGN, bad


def test_rows_longer_than_the_kernels_index(lib):
    """Above 2^29 elements of a row 32-bit column numbers would wrap (in the column sums' rows of 2 D floats from
    2^30 on, in the general kernels' loops next to 2^31)."""
    far = 1 << 44
    for n in ((1 << 29) + 1, (1 << 30), (1 << 31) - 1):
        for dt in (0, 1):
            assert lib.ret_layer_norm(p(far), None, None, None, p(2 * far), None, None, None, 1, n, 1e-5, dt, dt,
                                      None) == UNSUPPORTED
            assert lib.ret_layer_norm_backward(p(far), p(2 * far), None, p(3 * far), p(4 * far), None, p(5 * far),
                                               p(6 * far), p(7 * far), 1, n, dt, dt, None) == UNSUPPORTED
            assert lib.ret_msr_norm_gate_backward(p(far), p(2 * far), p(3 * far), p(4 * far), p(5 * far), 1, 1, 1, n,
                                                  1e-5, dt, None) == UNSUPPORTED
            rows = (n, n, n)
            for layout in (0, 1):
                assert _rot(lib, q=far, qo=2 * far, freqs=3 * far, sq=rows, sqo=rows, B=1, N=1, Hq=1, d=n, rot=0,
                            layout=layout, dt=dt) == UNSUPPORTED


def test_more_elements_than_a_byte_count_holds(lib):
    far = 1 << 44
    big = (1 << 31) - 1
    assert lib.ret_msr_norm_gate_backward(p(far), p(2 * far), p(3 * far), p(4 * far), p(5 * far), big, big, big, 64,
                                          1e-5, 1, None) == UNSUPPORTED


# ---------------------------------------------------------------- the path's calls on another device

class _Tensor:
    """Of a tensor, what a call asks before it enters the tensor's device."""

    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index


def test_every_call_on_device_tensors_enters_their_device(monkeypatch):
    entered = []

    class Entered:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            entered.append(self.index)

        def __exit__(self, *_):
            entered.append("left")

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Entered)
    call = ret._on_device_of_tensors(lambda *a, **k: list(entered))
    assert call(_Tensor(0), 64) == []             # the current device: nothing to enter
    assert call(_Tensor(-1), 64) == []            # a host tensor: refused later, by the call itself
    assert call(_Tensor(1), 64) == [1] and entered == [1, "left"]
    entered.clear()
    assert call(q=_Tensor(2), chunk=64) == [2]
    for name in ("ret_parallel", "ret_chunkwise", "ret_chunkwise_noalloc", "gated_ret_chunkwise", "ret_recurrent_step",
                 "gated_ret_recurrent_step", "chunkwise_state", "state_prefix", "chunkwise_backward", "msr_norm_gate"):
        assert hasattr(getattr(ret, name), "__wrapped__"), name
