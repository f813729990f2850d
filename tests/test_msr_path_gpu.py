"""The operators around retention together, as a RetNet block uses them: layer norm, rotary prologue,
chunkwise retention and the norm-and-gate epilogue, forward and backward against plain 64-bit torch;
prefill followed by decode steps; captured in CUDA graphs; on another stream."""
import pytest
import torch

from linear_attention_ret_b200 import autograd as A
from linear_attention_ret_b200 import inputs as I
from linear_attention_ret_b200.rotary import frequencies
from tests import plain64 as P
from tests.parity import TOL_BF16, TOL_F32, rel_l2

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
bf, f32 = torch.bfloat16, torch.float32


def randn(*shape, dtype=f32, seed=0, scale=1.0):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype).to(DEV)


def retention64(q, k, v, gamma):
    n = torch.arange(q.shape[2])
    D = torch.where(n[:, None] >= n, gamma[:, None, None] ** (n[:, None] - n).clamp(min=0), 0.0)
    return ((q @ k.transpose(-1, -2)) * D) @ v


def path64(q, k, v, gate, gamma, freqs, pos, k_scale, eps=1e-5):
    def turn(x, s):  # differentiable form of the interleaved rotation
        t = (pos.to(torch.float64)[..., None] * freqs)[:, :, None, :]
        a, b = x[..., 0::2], x[..., 1::2]
        return s * torch.stack([a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()], -1).flatten(-2)
    o = retention64(turn(q, 1.0).transpose(1, 2), turn(k, k_scale).transpose(1, 2), v.transpose(1, 2), gamma)
    o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
    return gate * torch.sigmoid(gate) * o.transpose(1, 2)


@pytest.mark.parametrize("dtype,B,N,H,dk,dv", [
    (f32, 2, 33, 2, 32, 32),
    (bf, 1, 200, 2, 64, 128),     # the tensor-core path
    (bf, 2, 130, 2, 128, 256),
    (f32, 1, 1, 2, 16, 24),       # one token
])
def test_block_matches_plain(cuda_lib, dtype, B, N, H, dk, dv):
    """A pre-norm block: y = msr(LN(x) W) + x through the framework's operators, with all gradients."""
    E = H * dv
    tol = TOL_F32 if dtype == f32 else TOL_BF16
    x = randn(B, N, E, dtype=dtype)
    lw, lb = 1 + randn(E, seed=1, scale=0.2), randn(E, seed=2, scale=0.1)
    W = randn(E, H * (2 * dk + 2 * dv), dtype=dtype, seed=3, scale=E ** -0.5)
    gamma = I.gammas(H).to(DEV)
    freqs, _ = frequencies(dk, schedule="retnet")
    dy, dres = randn(B, N, H, dv, dtype=dtype, seed=4, scale=0.1), randn(B, N, E, dtype=dtype, seed=5, scale=0.1)
    res = randn(B, N, E, dtype=dtype, seed=6)
    starts = torch.arange(B, device=DEV) * 1000
    widths = [H * dk, H * dk, H * dv, H * dv]

    def parts(h, W):
        qkvg = (h @ W).split(widths, -1)
        return [t.unflatten(-1, (H, -1)) for t in qkvg]

    leaves = [t.clone().requires_grad_() for t in (x, res, lw, lb, W)]
    h, s = A.layer_norm(leaves[0], leaves[2], leaves[3], residual=leaves[1])
    q, k, v, g = parts(h, leaves[4])
    y = A.multi_scale_retention(q, k, v, g, gamma, freqs.to(DEV), starts=starts, k_scale=dk ** -0.5)
    grads = torch.autograd.grad((y, s), leaves, (dy, dres))

    ref = [P.f64(t).requires_grad_() for t in (x, res, lw, lb, W)]
    s64 = ref[0] + ref[1]
    mu = s64.mean(-1, keepdim=True)
    h64 = (s64 - mu) / torch.sqrt(((s64 - mu) ** 2).mean(-1, keepdim=True) + 1e-5) * ref[2] + ref[3]
    pos = P.positions(B, N, None, starts)
    y64 = path64(*parts(h64, ref[4]), P.f64(gamma), freqs, pos, dk ** -0.5)
    want = torch.autograd.grad((y64, s64), ref, (P.f64(dy), P.f64(dres)))
    # The epilogue divides by the size of retention's output: where a row's output is small the relative
    # error of everything before it is magnified, so the chain is held to five times a single operator's
    # target (five roundings: norm, projection, rotation, retention, epilogue).
    assert rel_l2(y, y64.detach()) <= 5 * tol
    for name, got, w in zip(("x", "residual", "ln weight", "ln bias", "W"), grads, want):
        assert rel_l2(got, w) <= 5 * tol, name
    assert cuda_lib.last_device_error() == 0


def test_gradients_agree_with_differences(cuda_lib):
    """Directional differences of the fp32 path itself."""
    B, N, H, dk, dv = 1, 6, 2, 8, 8
    freqs = frequencies(dk, schedule="retnet")[0].to(DEV)
    leaves = [randn(B, N, H, dk), randn(B, N, H, dk, seed=1), randn(B, N, H, dv, seed=2), randn(B, N, H, dv, seed=3)]
    gamma, dy = I.gammas(H).to(DEV), randn(B, N, H, dv, seed=4)
    lw = 1 + randn(dv, seed=9, scale=0.2)

    def loss(q, k, v, g):
        return (A.layer_norm(A.multi_scale_retention(q, k, v, g, gamma, freqs, eps=0.1), lw, eps=0.1) * dy).sum()

    live = [t.clone().requires_grad_() for t in leaves]
    grads = torch.autograd.grad(loss(*live), live)
    h = 2e-2
    for i, g in enumerate(grads):
        d = randn(*leaves[i].shape, seed=20 + i)

        def at(step):
            args = list(leaves)
            args[i] = leaves[i] + step * d
            return loss(*args).double()
        # Richardson: the h^2 term cancels; fp32 noise of the loss, about 1e-6 of its terms, over 2 h
        diff = (8 * (at(h / 2) - at(-h / 2)) - (at(h) - at(-h))) / (6 * h)
        want = (g * d).double().sum()
        assert abs(diff - want) <= 2e-3 * (g * d).double().abs().sum(), i


def test_prefill_then_decode(cuda_lib):
    """Serving: a prompt through the chunkwise form, then single tokens, each at its own position."""
    B, H, dk, dv, N, steps = 2, 2, 64, 128, 70, 4
    ret = cuda_lib
    q, k = randn(B, N + steps, H, dk, dtype=bf, scale=0.125), randn(B, N + steps, H, dk, dtype=bf, seed=1, scale=0.125)
    v, g = randn(B, N + steps, H, dv, dtype=bf, seed=2), randn(B, N + steps, H, dv, dtype=bf, seed=3)
    gamma = I.gammas(H).to(DEV)
    freqs = frequencies(dk, schedule="retnet")[0]
    fd = freqs.to(DEV)
    starts = torch.tensor([0, 500], device=DEV)  # the second sequence continues an earlier document
    state = torch.zeros(B, H, dk, dv, device=DEV)
    qh, kh = ret.rotary(q[:, :N], k[:, :N], fd, starts=starts)
    vh, _ = ret.rotary(v[:, :N], None, None)
    ys = [ret.msr_norm_gate(ret.ret_chunkwise(qh, kh, vh, gamma, 64, state_in=state, state_out=state),
                            g[:, :N].contiguous())]
    starts = starts + N
    for t in range(N, N + steps):
        qh, kh = ret.rotary(q[:, t:t + 1], k[:, t:t + 1], fd, starts=starts)
        o = ret.ret_recurrent_step(qh.view(B, H, dk), kh.view(B, H, dk), v[:, t].contiguous(), gamma, state)
        ys.append(ret.msr_norm_gate(o.view(B, H, 1, dv), g[:, t:t + 1].contiguous()))
        starts += 1
    pos = P.positions(B, N + steps, None, torch.tensor([0, 500]))
    want = path64(*(P.f64(t) for t in (q, k, v, g)), P.f64(gamma), freqs, pos, 1.0)
    assert rel_l2(torch.cat(ys, 1), want) <= TOL_BF16


def _graph_of(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fn()
    return graph, out


def test_captured_decode_step_follows_its_inputs(cuda_lib):
    """One serving step in a graph: replays read the positions and tokens that are there then."""
    ret = cuda_lib
    B, H, dk, dv = 3, 2, 64, 64
    fd = frequencies(dk)[0].to(DEV)
    x, w = randn(B, 1, H * dk, dtype=bf), randn(H * dk)
    res = randn(B, 1, H * dk, dtype=bf, seed=1)
    starts = torch.tensor([0, 9, 100000], device=DEV)

    def step():
        h, s = ret.layer_norm(x, w, residual=res)
        q, k = ret.rotary(h.view(B, 1, H, dk), s.view(B, 1, H, dk), fd, starts=starts, layout="half")
        return q, k

    graph, out = _graph_of(step)
    for i in range(3):
        x.copy_(randn(B, 1, H * dk, dtype=bf, seed=10 + i))
        starts += 1
        graph.replay()
        for got, want in zip(out, step()):
            assert torch.equal(got, want)


def test_two_captured_backwards_share_nothing(cuda_lib):
    """Two graphs of the norm's backward (partial sums in scratch), replayed side by side on two streams."""
    ret = cuda_lib
    calls, want = [], []
    for i, (rows, D) in enumerate([(700, 1024), (900, 1000)]):
        x, dy, w = randn(rows, D, dtype=bf, seed=i), randn(rows, D, dtype=bf, seed=9 + i), randn(D, seed=20 + i)
        mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        ret.layer_norm(x, w, mean=mean, rstd=rstd)
        calls.append(lambda a=(dy, x, w, mean, rstd): ret.layer_norm_backward(*a))
        want.append([t.clone() for t in calls[-1]()])
    graphs = [_graph_of(c) for c in calls]
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, out), ref in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_captured_training_step(cuda_lib):
    """Forward and backward of the path in one graph (gradients by autograd.grad: nothing accumulates into leaves)."""
    B, N, H, dk, dv = 1, 128, 2, 64, 128
    freqs = frequencies(dk, schedule="retnet")[0].to(DEV)
    gamma = I.gammas(H).to(DEV)
    leaves = [randn(B, N, H, d, dtype=bf, seed=i, scale=d ** -0.5).requires_grad_()
              for i, d in enumerate((dk, dk, dv, dv))]
    lw = randn(dv, seed=7).requires_grad_()
    dy = randn(B, N, H, dv, dtype=bf, seed=8)

    def step():
        y = A.layer_norm(A.multi_scale_retention(*leaves, gamma, freqs), lw)
        return torch.autograd.grad(y, [*leaves, lw], dy)

    eager = [t.clone() for t in step()]
    graph, out = _graph_of(step)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, eager))
    del graph


def test_on_another_stream(cuda_lib):
    """stream=: the call runs there, and so are its outputs allocated."""
    ret = cuda_lib
    side = torch.cuda.Stream()
    x, w = randn(300, 1000, dtype=bf), randn(1000)
    q = randn(2, 50, 3, 64, dtype=bf)
    f = frequencies(64)[0].to(DEV)
    o, g = randn(2, 3, 50, 64, dtype=bf, seed=1), randn(2, 50, 3, 64, dtype=bf, seed=2)
    mean, rstd = torch.empty(300, device=DEV), torch.empty(300, device=DEV)
    want = [ret.layer_norm(x, w, mean=mean, rstd=rstd), *ret.layer_norm_backward(x, x, w, mean, rstd),
            *ret.rotary(q, q, f), *ret.rotary_backward(o, o, f), *ret.msr_norm_gate_backward(g, o, g)]
    torch.cuda.synchronize()
    current = torch.cuda.current_stream()
    got = [ret.layer_norm(x, w, stream=side), *ret.layer_norm_backward(x, x, w, mean, rstd, stream=side),
           *ret.rotary(q, q, f, stream=side), *ret.rotary_backward(o, o, f, stream=side),
           *ret.msr_norm_gate_backward(g, o, g, stream=side)]
    assert torch.cuda.current_stream() == current
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_back_to_back_calls_see_each_others_results(cuda_lib):
    """Kernels that are placed while the one before drains: a chain in which each call reads what the one
    before wrote, with and without a synchronise between the calls."""
    ret = cuda_lib
    B, N, H, d = 1, 300, 4, 64
    D = H * d
    freqs = frequencies(d)[0].to(DEV)

    def chain(sync):
        def settle():
            if sync:
                torch.cuda.synchronize()
        x, w, b = randn(B, N, D, dtype=bf), randn(D, seed=1), randn(D, seed=2)
        y, s = torch.empty_like(x), torch.zeros_like(x)
        mean, rstd = torch.empty(B, N, device=DEV), torch.empty(B, N, device=DEV)
        q, o = torch.empty(B, H, N, d, dtype=bf, device=DEV), torch.empty(B, N, H, d, dtype=bf, device=DEV)
        for i in range(40):
            ret.layer_norm(x, w, b, residual=s, y=y, sum_out=s, mean=mean, rstd=rstd)
            settle()
            ret.rotary(y.view(B, N, H, d), None, freqs, offset=i, q_out=q)
            settle()
            ret.msr_norm_gate_backward(y.view(B, N, H, d), q, s.view(B, N, H, d), dout=q, dgate=o)
            settle()
            _, w, b = ret.layer_norm_backward(o.view(B, N, D), s, w, mean, rstd, dsum=y, dx=x)
            settle()
            w, b = w.clamp(-2, 2), b.clamp(-2, 2)
        torch.cuda.synchronize()
        return x, s, q, o, w, b

    for got, want in zip(chain(False), chain(True)):
        assert torch.isfinite(want).all() and torch.equal(got, want)


def test_two_threads_at_once(cuda_lib):
    """Calls from several host threads, each on a stream of its own."""
    import threading
    ret = cuda_lib
    jobs = []
    for i, (rows, D) in enumerate([(513, 1024), (700, 771), (90, 12000), (4, 16384)]):
        x, dy, w = randn(rows, D, dtype=bf, seed=i), randn(rows, D, dtype=bf, seed=10 + i), randn(D, seed=20 + i)
        mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        ret.layer_norm(x, w, mean=mean, rstd=rstd)
        jobs.append((dy, x, w, mean, rstd))
    want = [ret.layer_norm_backward(*j) for j in jobs]
    torch.cuda.synchronize()
    got, errors = [None] * len(jobs), []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(30):
                    got[i] = ret.layer_norm_backward(*jobs[i])
            s.synchronize()
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


FIRST_CALL_CAPTURED = """
import torch
from linear_attention_ret_b200 import ret
from linear_attention_ret_b200.rotary import frequencies
x, w = torch.randn(300, 1024, device="cuda").bfloat16(), torch.randn(1024, device="cuda")
mean, rstd = torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
q, f = torch.randn(2, 9, 4, 64, device="cuda").bfloat16(), frequencies(64)[0].cuda()
def calls():
    y = ret.layer_norm(x, w, mean=mean, rstd=rstd)
    return [y, *ret.layer_norm_backward(y, x, w, mean, rstd), *ret.rotary(q, q, f),
            *ret.msr_norm_gate_backward(q, q.view(2, 4, 9, 64), q)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = calls()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, calls()))
print("same")
"""


def test_first_call_may_be_captured(cuda_lib):
    """A process whose first calls are made under capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "same" in p.stdout, p.stderr[-2000:]
