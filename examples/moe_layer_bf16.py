"""A mixture-of-experts layer in bf16: training steps, and decode steps with its weights in NVFP4.

Runs the router and the experts' products together: gate -> route -> permute -> gate/up product -> SwiGLU -> down product
-> combine, with the load-balance loss, and the whole way back.  The experts' master weights are fp32, the products read their
bf16 form.  For decode the same weights are quantized to NVFP4 once; the few rows of a step stay bf16.

    python examples/moe_layer_bf16.py            # needs a GB300
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_moe_expert_gb300 as fme  # noqa: E402


class MoELayer:
    def __init__(self, hidden=1024, inter=512, experts=8, top_k=2, *, score="sigmoid", alpha=1e-2, scale=1.0,
                 device="cuda", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, std):
            return torch.empty(shape, device=device).normal_(0.0, std, generator=g)

        self.hidden, self.inter, self.experts, self.top_k = hidden, inter, experts, top_k
        self.score, self.alpha, self.scale = score, alpha, scale
        self.w_router = normal(experts, hidden, std=hidden ** -0.5)
        self.w_gate_up = normal(experts, 2 * inter, hidden, std=hidden ** -0.5)
        self.w_down = normal(experts, hidden, inter, std=inter ** -0.5)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.cast()

    def cast(self):
        """The experts' bf16 weights from the fp32 ones: after loading and after each update."""
        self.gate_up, self.down = self.w_gate_up.to(torch.bfloat16), self.w_down.to(torch.bfloat16)

    def quantize(self):
        """The experts' NVFP4 weights for decode steps."""
        self.gate_up_4 = fme.quantize_nvfp4_pertoken(self.gate_up.view(-1, self.hidden), status=self.status)
        self.down_4 = fme.quantize_nvfp4_pertoken(self.down.view(-1, self.inter), status=self.status)

    def route(self, x):
        logits = x.float() @ self.w_router.t()
        ids, weights = fme.moe_gate(logits, self.top_k, score=self.score, scale=self.scale)
        return logits, ids, weights, *fme.moe_route(ids, self.experts, status=self.status)

    def forward(self, x):
        """x [tokens, hidden] bf16 -> (out bf16, balance loss [1], saved for backward)."""
        st = self.status
        logits, ids, weights, offsets, row_of, src_row = self.route(x)
        loss, counts, seq_tokens = fme.moe_balance_loss(logits, ids, score=self.score, alpha=self.alpha, status=st)
        rows = fme.moe_permute(x, src_row, self.top_k, status=st)
        gu = fme.grouped_gemm_fwd_bf16(rows, self.gate_up, offsets, status=st)
        h = fme.swiglu(gu)
        y = fme.grouped_gemm_fwd_bf16(h, self.down, offsets, status=st)
        out = fme.moe_combine(y, row_of, weights, status=st)
        return out, loss, (x, logits, ids, weights, counts, seq_tokens, offsets, row_of, rows, gu, h, y)

    def backward(self, d_out, d_loss, saved):
        """Gradients of sum(out * d_out) + loss * d_loss -> dict of x, w_router, w_gate_up, w_down."""
        x, logits, ids, weights, counts, seq_tokens, offsets, row_of, rows, gu, h, y = saved
        st = self.status
        d_y, d_weights = fme.moe_combine_backward(d_out, y, row_of, weights, status=st)
        d_h = fme.grouped_gemm_dgrad_bf16(d_y, self.down, offsets, status=st)
        d_down = fme.grouped_gemm_wgrad_bf16(d_y, h, offsets, dtype=torch.float32, status=st)
        d_gu = fme.swiglu_backward(gu, d_h)
        d_rows = fme.grouped_gemm_dgrad_bf16(d_gu, self.gate_up, offsets, status=st)
        d_gate_up = fme.grouped_gemm_wgrad_bf16(d_gu, rows, offsets, dtype=torch.float32, status=st)
        d_x = fme.moe_combine(d_rows, row_of, torch.ones_like(weights), status=st).float()  # the permute's gradient
        d_logits = fme.moe_gate_backward(logits, ids, d_weights, score=self.score, scale=self.scale, status=st)
        fme.moe_balance_loss_backward(logits, counts, seq_tokens, d_loss, self.top_k, score=self.score, alpha=self.alpha,
                                      d_logits=d_logits, accumulate=True)
        return {"x": d_x + d_logits @ self.w_router, "w_router": d_logits.t() @ x.float(), "w_gate_up": d_gate_up,
                "w_down": d_down}

    def decode(self, x):
        """A decode step: x [tokens, hidden] bf16, few tokens -> out bf16, from the NVFP4 weights."""
        st = self.status
        _, _, weights, offsets, row_of, src_row = self.route(x)
        h = fme.grouped_gemv_nvfp4_swiglu(x, *self.gate_up_4, offsets, src_row=src_row, top_k=self.top_k, status=st)
        y = fme.grouped_gemv_nvfp4(h, *self.down_4, offsets, status=st)
        return fme.moe_combine(y, row_of, weights, status=st)

    def update(self, grads, rate):
        """A step of gradient descent."""
        self.w_router -= rate * grads["w_router"]
        self.w_gate_up -= rate * grads["w_gate_up"]
        self.w_down -= rate * grads["w_down"]
        self.cast()


def main(steps=12, tokens=512):
    layer = MoELayer()
    teacher = MoELayer(seed=1)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.empty((tokens, layer.hidden), device="cuda").normal_(0.0, 1.0, generator=g).to(torch.bfloat16)
    target = teacher.forward(x)[0].float()
    losses = []
    for step in range(steps):
        out, balance, saved = layer.forward(x)
        diff = out.float() - target
        losses.append(diff.square().mean().item())
        layer.update(layer.backward((2.0 * diff / diff.numel()).to(torch.bfloat16), torch.ones(1, device="cuda"), saved),
                     rate=30.0)
        print(f"step {step:2d}  error {losses[-1]:.5f}  balance {balance.item():.5f}")
    layer.quantize()
    few = x[:4].contiguous()
    exact, quantized = layer.forward(few)[0].float(), layer.decode(few).float()
    print(f"4 decoded tokens, NVFP4 weights: off by {((quantized - exact).norm() / exact.norm()).item():.3f} of their norm")
    one = layer.decode(x[:1].contiguous()).float()
    print("one token alone equals its row among the four:", torch.equal(one[0], quantized[0]))
    for l in (layer, teacher):
        code, raw = fme.read_device_status(l.status)
        assert code == 0, f"device status {raw:#x}"
    return losses


if __name__ == "__main__":
    main()
