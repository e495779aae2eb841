"""The MoE layer of examples/moe_layer.py against the same layer in float64 autograd on the CPU.

Each bf16 tensor on the way (h, pre, act, o, y and their gradients, at most six in a row) adds a rounding error of
2^-9 of its norm at most (half an ulp is 2^-8 of the smallest mantissa, and errors of single elements do not
line up), a product's operands enter linearly: every result stays within 12·2^-9 of its norm (0.023)."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(layer, x, dy):
    w = {n: getattr(layer, n).cpu().double().requires_grad_() for n in ("w_router", "w_gate_up", "w_down")}
    x = x.cpu().double().requires_grad_()
    top, ids = (x @ w["w_router"].t()).topk(layer.top_k, dim=1)
    p = torch.softmax(top, 1)
    rows = []
    for t in range(x.shape[0]):
        y = x[t]
        for k in range(layer.top_k):
            e = ids[t, k]
            u, v = (w["w_gate_up"][e] @ x[t]).chunk(2)
            a = 4 * torch.tanh(u / 4) * torch.sigmoid(u) * 25 * torch.tanh(v / 25)
            y = y + p[t, k] * (w["w_down"][e] @ a)
        rows.append(y)
    y = torch.stack(rows)
    y.backward(dy.cpu().double())
    return dict(y=y.detach(), dx=x.grad, **{"d" + n: t.grad for n, t in w.items()}), ids


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,H,E,K", [(1, 64, 32, 8, 2), (37, 128, 64, 8, 3), (70, 192, 48, 16, 4)])
def test_layer_matches_autograd(T, D, H, E, K):
    layer = example().MoELayer(D, H, E, K, seed=T)
    g = torch.Generator().manual_seed(T)
    x, dy = (torch.randn(T, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    y = layer.forward(x)
    ids = layer.saved[2]
    got = dict(y=y, **layer.backward(dy))
    want, want_ids = reference(layer, x, dy)
    assert torch.equal(ids.cpu().long(), want_ids)
    for name, w in want.items():
        off = (got[name].cpu().double() - w).norm() / w.norm()
        assert off < 12 * 2.0 ** -9, (name, off.item())
    assert torch.equal(layer.forward(x, train=False), y)


@pytest.mark.gpu
def test_step_in_a_graph():
    """Nothing in a step waits for the host: forward and backward are captured and replayed on new inputs."""
    layer = example().MoELayer(128, 64, 16, 4, seed=5)
    g = torch.Generator().manual_seed(5)
    new = lambda: torch.randn(300, 128, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    x, dy = new(), new()

    def step():
        y = layer.forward(x)
        return dict(y=y, **layer.backward(dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(new())
    dy.copy_(new())
    graph.replay()
    torch.cuda.synchronize()
    for name, want in step().items():
        assert torch.equal(out[name], want), name


@pytest.mark.gpu
def test_example_runs():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "moe_layer.py"), "--tokens", "64", "--width", "256", "--hidden",
                          "128", "--experts", "8", "--top-k", "2"], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert "training step" in out.stdout and "decoding step" in out.stdout
