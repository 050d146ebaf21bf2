"""A mixture-of-experts layer in FP8 with block-128 scales: training steps and a decode step.

Runs the router and the experts' products together: gate -> route -> quantize the grouped tokens -> gate/up
product -> SwiGLU -> down product -> combine, with the load-balance loss, and the whole way back to the
gradients of the input, the router and the experts.  The experts' master weights are fp32; their FP8 form is made
after each update and serves the forward and both gradients.

    python examples/moe_layer_fp8.py            # needs a GB300
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
        self.bias = torch.zeros(experts, device=device)  # steers the choice of experts alone
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.quantize()

    def quantize(self):
        """The experts' FP8 weights from the fp32 ones: after loading and after each update."""
        self.gate_up = fme.quantize_fp8_block128_weights(self.w_gate_up.to(torch.bfloat16))
        self.down = fme.quantize_fp8_block128_weights(self.w_down.to(torch.bfloat16))

    def forward(self, x, seq_offsets=None, token_mask=None):
        """x [tokens, hidden] bf16 -> (out bf16, balance loss [1], saved for backward)."""
        st = self.status
        logits = x.float() @ self.w_router.t()
        ids, weights = fme.moe_gate(logits, self.top_k, score=self.score, bias=self.bias, scale=self.scale)
        loss, counts, seq_tokens = fme.moe_balance_loss(logits, ids, score=self.score, alpha=self.alpha,
                                                        seq_offsets=seq_offsets, token_mask=token_mask, status=st)
        offsets, row_of, src_row = fme.moe_route(ids, self.experts, status=st)
        xq = fme.quantize_fp8_block128(x, src_row=src_row, top_k=self.top_k, status=st)
        gu = fme.grouped_gemm_fwd_fp8_block128(*xq, *self.gate_up, offsets, status=st)
        gate, up = gu.float().chunk(2, dim=1)
        h = (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)
        y = fme.grouped_gemm_fwd_fp8_block128(*fme.quantize_fp8_block128(h, status=st), *self.down, offsets, status=st)
        out = fme.moe_combine(y, row_of, weights, status=st)
        saved = (x, logits, ids, weights, counts, seq_tokens, offsets, row_of, src_row, gu, h, y, seq_offsets, token_mask)
        return out, loss, saved

    def backward(self, d_out, d_loss, saved):
        """Gradients of sum(out * d_out) + loss * d_loss -> dict of x, w_router, w_gate_up, w_down."""
        (x, logits, ids, weights, counts, seq_tokens, offsets, row_of, src_row, gu, h, y, seq_offsets,
         token_mask) = saved
        st = self.status
        # combine and down projection
        d_y, d_weights = fme.moe_combine_backward(d_out, y, row_of, weights, status=st)
        dy_rows, (dyc, dyc_scale, padded) = fme.quantize_fp8_block128_rowcol(d_y, offsets, status=st)
        d_h = fme.grouped_gemm_dgrad_fp8_block128(*dy_rows, *self.down, offsets, status=st)
        hc, hc_scale, _ = fme.quantize_fp8_block128(h, fme.COLWISE, offsets, status=st)
        d_down = fme.grouped_gemm_wgrad_fp8_block128(dyc, dyc_scale, hc, hc_scale, padded, dtype=torch.float32, status=st)
        # SwiGLU
        gate, up = gu.float().chunk(2, dim=1)
        sig = torch.sigmoid(gate)
        d_h = d_h.float()
        d_gu = torch.cat([d_h * up * sig * (1 + gate * (1 - sig)), d_h * gate * sig], dim=1).to(torch.bfloat16)
        # gate/up projection
        dgu_rows, (dgc, dgc_scale, padded) = fme.quantize_fp8_block128_rowcol(d_gu, offsets, status=st)
        d_rows = fme.grouped_gemm_dgrad_fp8_block128(*dgu_rows, *self.gate_up, offsets, status=st)
        grouped = x[src_row.long() // self.top_k]
        xc, xc_scale, _ = fme.quantize_fp8_block128(grouped, fme.COLWISE, offsets, status=st)
        d_gate_up = fme.grouped_gemm_wgrad_fp8_block128(dgc, dgc_scale, xc, xc_scale, padded, dtype=torch.float32,
                                                        status=st)
        d_x = fme.moe_combine(d_rows, row_of, torch.ones_like(weights), status=st).float()
        # router: the weights' gradient, and the balance loss's on top of it
        d_logits = fme.moe_gate_backward(logits, ids, d_weights, score=self.score, scale=self.scale, status=st)
        fme.moe_balance_loss_backward(logits, counts, seq_tokens, d_loss, self.top_k, score=self.score, alpha=self.alpha,
                                      seq_offsets=seq_offsets, token_mask=token_mask, d_logits=d_logits,
                                      accumulate=True)
        return {"x": d_x + d_logits @ self.w_router, "w_router": d_logits.t() @ x.float(), "w_gate_up": d_gate_up,
                "w_down": d_down}

    def update(self, grads, rate, counts=None, bias_rate=1e-2):
        """A step of gradient descent; with counts, experts chosen less than the mean are preferred more."""
        self.w_router -= rate * grads["w_router"]
        self.w_gate_up -= rate * grads["w_gate_up"]
        self.w_down -= rate * grads["w_down"]
        if counts is not None:
            load = counts.sum(dim=0).float()
            self.bias += bias_rate * torch.sign(load.mean() - load)
        self.quantize()


def main(steps=12, tokens=512):
    layer = MoELayer()
    teacher = MoELayer(seed=1)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.empty((tokens, layer.hidden), device="cuda").normal_(0.0, 1.0, generator=g).to(torch.bfloat16)
    seq = torch.tensor([0, tokens // 4, tokens], dtype=torch.int32, device="cuda")  # two packed sequences
    target = teacher.forward(x)[0].float()
    first = None
    for step in range(steps):
        out, balance, saved = layer.forward(x, seq_offsets=seq)
        diff = out.float() - target
        loss = diff.square().mean()
        d_out = (2.0 * diff / diff.numel()).to(torch.bfloat16)
        grads = layer.backward(d_out, torch.ones(1, device="cuda"), saved)
        layer.update(grads, rate=30.0, counts=saved[4])
        first = loss.item() if first is None else first
        print(f"step {step:2d}  error {loss.item():.5f}  balance {balance.item():.5f}  "
              f"busiest expert {int(saved[4].sum(dim=0).max())} of {tokens * layer.top_k} choices")
    one, _, _ = layer.forward(x[:1].contiguous())  # a decode step
    out, _, _ = layer.forward(x)
    print("one token alone equals its row in the batch:", torch.equal(one[0], out[0]))
    code, raw = fme.read_device_status(layer.status)
    assert code == 0 and teacher.status.item() == 0, f"device status {raw:#x}"
    return first, loss.item()


if __name__ == "__main__":
    main()
