"""The example's bf16 layer against the same layer in 32 bits with autograd.

The reference has the bf16 weights and inputs, so what differs is the rounding of what lies between the calls: each is within
2^-8 of its value, 2^-8 / sqrt(3) = 0.23% root mean square at most.  Four of them follow one another forward (gate/up, h,
the down projection, the output), up to eight on the way to a gradient (those and dy, dh, d(gate/up), the rows of dx):
sqrt(8) x 0.23% = 0.64%, and through products of two rounded operands at most twice that.  The bound is 2% of each
result's norm; the balance loss, which passes none of them, is held to fp32."""
import importlib.util
import os

import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import nvfp4w

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    fme.ensure_built()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer_bf16.py")
    spec = importlib.util.spec_from_file_location("moe_layer_bf16", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def off(a, b):
    return float((a.float() - b).norm() / b.norm())


def reference(x, w_router, w_gate_up, w_down, ids, score, scale, top_k, alpha):
    """(output, balance loss) for the chosen experts ids."""
    experts = w_router.shape[0]
    logits = x @ w_router.t()
    p = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    chosen = p.gather(1, ids)
    w = scale * chosen / chosen.sum(1, True)
    y = torch.zeros_like(x)
    for e in range(experts):
        t, k = (ids == e).nonzero(as_tuple=True)
        gate, up = (x[t] @ w_gate_up[e].t()).chunk(2, 1)
        y = y.index_add(0, t, w[t, k][:, None] * ((gate * torch.sigmoid(gate) * up) @ w_down[e].t()))
    q = p / p.sum(1, True)
    f = torch.bincount(ids.reshape(-1), minlength=experts).float() * experts / (top_k * x.shape[0])
    return y, alpha * (f * q.mean(0)).sum()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("hidden,inter,experts,top_k,tokens", [(512, 256, 8, 2, 600), (400, 136, 5, 3, 77), (256, 192, 4, 2, 9000)])
def test_layer_against_fp32_autograd(example, score, hidden, inter, experts, top_k, tokens):
    layer = example.MoELayer(hidden, inter, experts, top_k, score=score, alpha=0.5, scale=2.0, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    d_out = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    out, loss, saved = layer.forward(x)
    grads = layer.backward(d_out, torch.full((1,), 3.0, device="cuda"), saved)
    assert fme.read_device_status(layer.status)[0] == 0

    xr = x.float().requires_grad_(True)
    wr = layer.w_router.clone().requires_grad_(True)
    wgu, wd = (w.float().requires_grad_(True) for w in (layer.gate_up, layer.down))
    y, want = reference(xr, wr, wgu, wd, saved[2].long(), score, 2.0, top_k, 0.5)
    assert abs(loss.item() - want.item()) <= 1e-5 * abs(want.item())
    ((y * d_out.float()).sum() + 3.0 * want).backward()
    got = {"out": off(out, y.detach()), "x": off(grads["x"], xr.grad), "w_router": off(grads["w_router"], wr.grad),
           "w_gate_up": off(grads["w_gate_up"], wgu.grad), "w_down": off(grads["w_down"], wd.grad)}
    assert all(v < 0.02 for v in got.values()), got


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_decode_against_the_dequantized_weights(example, tokens):
    """The same bound: the NVFP4 weights of the reference are those of the layer."""
    hidden, inter, experts, top_k = 512, 256, 8, 2
    layer = example.MoELayer(hidden, inter, experts, top_k, seed=5)
    layer.quantize()
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    out = layer.decode(x)
    ids = layer.route(x)[1].long()
    assert fme.read_device_status(layer.status)[0] == 0
    gate_up = nvfp4w.values(*layer.gate_up_4).float().view(experts, 2 * inter, hidden)
    down = nvfp4w.values(*layer.down_4).float().view(experts, hidden, inter)
    want, _ = reference(x.float(), layer.w_router, gate_up, down, ids, "sigmoid", 1.0, top_k, 0.0)
    assert off(out, want) < 0.02


def test_example_runs(example):
    losses = example.main(steps=3, tokens=200)
    assert len(losses) == 3 and all(v == v for v in losses)
