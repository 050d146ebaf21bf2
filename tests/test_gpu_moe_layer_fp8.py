"""The example's FP8 layer against the same layer in 32 bits with autograd.

An E4M3 code is within 2^-4 of its value, uniformly spread: 2^-4 / sqrt(3) = 3.6% root mean square at most.  A product
of two quantized operands is then off by sqrt(2) x 3.6% = 5.1% of its norm; two products in a row and the gradients
through both by sqrt(2) to 2 times that.  The bound is 15% of each result's norm; what does not pass through the
experts (the balance loss) is held to fp32."""
import importlib.util
import os

import pytest
import torch

import fp8_moe_expert_gb300 as fme

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    fme.ensure_built()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer_fp8.py")
    spec = importlib.util.spec_from_file_location("moe_layer_fp8", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("hidden,inter,experts,top_k,tokens", [(512, 256, 8, 2, 300), (400, 144, 5, 3, 77)])
def test_layer_against_fp32_autograd(example, score, hidden, inter, experts, top_k, tokens):
    layer = example.MoELayer(hidden, inter, experts, top_k, score=score, alpha=0.5, scale=2.0, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    d_out = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    seq = torch.tensor([0, 20, 20, tokens], dtype=torch.int32, device="cuda")
    out, loss, saved = layer.forward(x, seq_offsets=seq)
    grads = layer.backward(d_out, torch.full((1,), 3.0, device="cuda"), saved)
    assert fme.read_device_status(layer.status)[0] == 0
    ids = saved[2].long()

    xr = x.float().requires_grad_(True)
    wr, wgu, wd = (w.clone().requires_grad_(True) for w in (layer.w_router, layer.w_gate_up, layer.w_down))
    logits = xr @ wr.t()
    p = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    chosen = p.gather(1, ids)
    w = 2.0 * chosen / chosen.sum(1, True)
    y = torch.zeros((tokens, hidden), device="cuda")
    for e in range(experts):
        t, k = (ids == e).nonzero(as_tuple=True)
        gate, up = (xr[t] @ wgu[e].t()).chunk(2, 1)
        y = y.index_add(0, t, w[t, k][:, None] * ((torch.nn.functional.silu(gate) * up) @ wd[e].t()))
    q = p / p.sum(1, True)
    terms = []
    for lo, hi in ((0, 20), (20, tokens)):
        n = hi - lo
        f = torch.bincount(ids[lo:hi].reshape(-1), minlength=experts).float() * experts / (top_k * n)
        terms.append((f * q[lo:hi].mean(0)).sum())
    want = 0.5 * torch.stack(terms).mean()
    assert abs(loss.item() - want.item()) <= 1e-5 * abs(want.item())
    ((y * d_out.float()).sum() + 3.0 * want).backward()

    def off(a, b):
        return float((a.float() - b).norm() / b.norm())

    got = {"out": off(out, y.detach()), "x": off(grads["x"], xr.grad), "w_router": off(grads["w_router"], wr.grad),
           "w_gate_up": off(grads["w_gate_up"], wgu.grad), "w_down": off(grads["w_down"], wd.grad)}
    assert all(v < 0.15 for v in got.values()), got


def test_example_learns(example):
    first, last = example.main(steps=6, tokens=256)
    assert last < first
