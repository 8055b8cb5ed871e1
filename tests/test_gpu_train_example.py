"""The training example: its gradients against torch's in 64 bits, a graph of the whole step, and steps
that lower the loss."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_moe_block as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def reference(p, x, ids, dout):
    """The block's gradients by torch's differentiation in 64 bits, with the same experts chosen."""
    q = {k: v.double().clone().requires_grad_() for k, v in p.items()}
    x = x.double().clone().requires_grad_()
    norm = lambda v, w: v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w  # noqa: E731
    h = norm(x, q["pre"])
    weights = torch.softmax((h @ q["router"].T).gather(1, ids.long()), 1)
    z = torch.zeros_like(h)
    for e in range(q["router"].shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            c = h[t] @ q["w13"][e].T
            gate, up = c.chunk(2, 1)
            z = z.index_add(0, t, (torch.nn.functional.silu(gate) * up @ q["w2"][e].T) * weights[t, j][:, None])
    out = x + ex.BLOCK_SCALE * q["gate"] * norm(z, q["post"])
    out.backward(dout.double())
    return out.detach(), {**{k: v.grad for k, v in q.items()}, "x": x.grad}


@pytest.mark.parametrize("T,H,I,E,k", [(300, 128, 64, 8, 2), (77, 200, 72, 33, 5), (1, 64, 32, 4, 4)])
def test_gradients_of_the_block(T, H, I, E, k):
    """Each stored tensor of the chain (h, rows, gate and up, act, y, z and their gradients) is rounded
    to bf16, 2^-9 of its size in the mean square at most; a gradient passes fewer than 12 of them."""
    p = ex.init_params(H, I, E, seed=T)
    g = torch.Generator().manual_seed(T + 1)
    x, dout = (torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(2))
    out, s = ex.forward(p, x, k)
    got = ex.backward(p, s, dout)
    want_out, want = reference(p, x, s["ids"], dout)
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()  # noqa: E731
    assert rel(out, want_out) < 12 * 2.0 ** -9
    for name, v in want.items():
        assert rel(got[name], v) < 12 * 2.0 ** -9, name


def test_step_in_a_graph_equals_the_step():
    H, I, E, k, T = 256, 96, 16, 4, 500
    g = torch.Generator().manual_seed(3)
    x, target = torch.randn(T, H, generator=g).bfloat16().cuda(), torch.randn(T, H, generator=g).cuda()
    a, b = ex.init_params(H, I, E), ex.init_params(H, I, E)
    want = [ex.train_step(a, x, target, k, 0.5) for _ in range(4)][-1]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ex.train_step(b, x, target, k, 0.5)      # the first step sets up outside the capture
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ex.train_step(b, x, target, k, 0.5)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_steps_lower_the_loss():
    losses = ex.main(["--tokens", "512", "--hidden", "256", "--inter", "128", "--experts", "16", "--topk", "4", "--steps", "30"])
    assert losses[-1] < 0.9 * losses[0]
