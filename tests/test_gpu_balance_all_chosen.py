"""The balance loss where every token has every expert (top_k = experts): the counts are equal, the loss is constant in
the logits and its gradient exactly zero."""
import pytest
import torch

import fp8_moe_expert_gb300 as fme

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("experts", [1, 2, 5, 8, 31, 32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_is_zero(experts, score, dtype):
    fme.ensure_built()
    g = torch.Generator(device=DEV)
    g.manual_seed(experts)
    tokens = 333
    l = (3 * torch.randn((tokens, experts), generator=g, device=DEV)).to(dtype)
    ids = torch.sort(l.float(), dim=1, descending=True, stable=True).indices.int()
    seq = torch.tensor([0, 100, 100, 101, tokens], dtype=torch.int32, device=DEV)
    mask = torch.rand(tokens, generator=g, device=DEV) < 0.8
    kw = dict(score=score, alpha=0.7, seq_offsets=seq, token_mask=mask)
    loss, counts, n = fme.moe_balance_loss(l, ids, **kw)
    up = torch.full((1,), 3.0, device=DEV)
    assert not bool(fme.moe_balance_loss_backward(l, counts, n, up, experts, **kw).any())
    base = torch.randn((tokens, experts), generator=g, device=DEV).to(dtype)
    into = base.clone()
    fme.moe_balance_loss_backward(l, counts, n, up, experts, d_logits=into, accumulate=True, **kw)
    assert torch.equal(into, base)
