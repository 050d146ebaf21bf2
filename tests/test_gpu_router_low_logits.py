"""The normalized sigmoid scores of rows whose logits are all far below zero: s_i / sum of s stays a ratio of
e^(l_i - max) where the sigmoids themselves leave fp32's normal range (below -87) or vanish (below -104).

The 64-bit form is softmax(log sigmoid(l)), the same ratio.  Tolerances: u = 2^-24; an exponential of x = l - max is
within (|x| + 2) u of itself, a sum of E of them within E u, the factor 1 - sigmoid, products and divisions a few u
each, so a probability is within (E + spread + 16) u, spread the row's largest |x|, doubled for the sums' own terms."""
import pytest
import torch

import fp8_moe_expert_gb300 as fme

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")
LEVELS = [-6.0, -20.0, -60.0, -86.0, -90.0, -93.0, -95.0, -100.0, -103.0, -104.0, -120.0, -200.0, -1e4]


@pytest.fixture(scope="module", autouse=True)
def _built():
    fme.ensure_built()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def low_rows(experts, dtype, seed, spread=1.5):
    """Three rows at each level, with small differences; some with experts masked by -inf; one at the type's lowest."""
    level = torch.tensor(LEVELS, device=DEV).repeat_interleave(3)[:, None]
    l = level + spread * torch.randn((len(level), experts), generator=gen(seed), device=DEV)
    l[1::3, 1::2] = -INF
    l = torch.cat([l, torch.full((1, experts), torch.finfo(dtype).min, device=DEV)])
    return l.to(dtype)


def slack(logits):
    x = logits.double()
    top = x.amax(1, True)
    d = torch.where(torch.isfinite(x), top - x, torch.zeros_like(x))
    return 2.0 * (logits.shape[1] + d.amax(1, True) + 16.0) * 2.0 ** -24


def ratio(l):
    return torch.softmax(torch.nn.functional.logsigmoid(l), 1)


def half_ulp(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


@pytest.mark.parametrize("experts,top_k", [(2, 2), (8, 2), (32, 8), (100, 4), (256, 8), (600, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_and_gradient(experts, top_k, dtype):
    l = low_rows(experts, dtype, experts)
    ids, w = fme.moe_gate(l, top_k, score="sigmoid", scale=2.5)
    want = torch.sort(l.float(), dim=1, descending=True, stable=True).indices[:, :top_k]
    assert torch.equal(ids.long(), want)
    l64 = l.double().requires_grad_(True)
    w64 = 2.5 * ratio(l64.gather(1, want))
    tol = slack(l.gather(1, want))
    assert bool(((w.double() - w64).abs() <= tol * w64).all())

    g = torch.randn(w.shape, generator=gen(2), device=DEV)
    d = fme.moe_gate_backward(l, ids, g, score="sigmoid", scale=2.5)
    finite = torch.where(torch.isfinite(l), l, torch.full_like(l, -3e38)).double().requires_grad_(True)
    (d64,) = torch.autograd.grad(2.5 * ratio(finite.gather(1, want)), finite, g.double())
    w64 = w64.detach()
    share = (w64 * g.abs().double()).sum(1, True) / 2.5
    term = torch.zeros_like(d64).scatter_(1, want, w64 * (g.abs().double() + share))
    lim = 2 * tol * term + half_ulp(dtype) * d64.abs() + 1e-40
    assert bool(((d.double() - d64).abs() <= lim).all())


@pytest.mark.parametrize("experts,top_k", [(2, 1), (8, 2), (32, 8), (100, 4), (256, 8), (600, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_balance_loss_and_gradient(experts, top_k, dtype):
    l = low_rows(experts, dtype, experts + 1)
    tokens = l.shape[0]
    ids = torch.sort(l.float(), dim=1, descending=True, stable=True).indices[:, :top_k].int()
    loss, counts, n = fme.moe_balance_loss(l, ids, score="sigmoid", alpha=0.3)
    l64 = torch.where(torch.isfinite(l), l, torch.full_like(l, -3e38)).double().requires_grad_(True)
    p = ratio(l64)
    c = torch.bincount(ids.reshape(-1).long(), minlength=experts).double()
    part = 0.3 * experts / (top_k * tokens ** 2)
    loss64 = part * (c * p.sum(0)).sum()
    tol = slack(l)
    assert abs(loss.item() - loss64.item()) <= (float(tol.max()) + (tokens + experts) * 2.0 ** -24) * loss64.item()
    d = fme.moe_balance_loss_backward(l, counts, n, torch.full((1,), -1.7, device=DEV), top_k, score="sigmoid", alpha=0.3)
    (d64,) = torch.autograd.grad(-1.7 * loss64, l64)
    p, a = p.detach(), 1.7 * part * c
    size = p * (a + (p * a).sum(1, True))
    lim = 2 * tol * size + half_ulp(dtype) * d64.abs() + 1e-40
    assert bool(((d.double() - d64).abs() <= lim).all())


def test_a_shift_far_below_zero_changes_nothing():
    """Where 1 - sigmoid is 1 in fp32 the ratios depend on the differences alone: the same bits at -40 and at -4096
    (differences that are exact next to both)."""
    diff = torch.randint(-32, 1, (50, 16), generator=gen(3), device=DEV).float() / 8
    g = torch.randn((50, 4), generator=gen(4), device=DEV)
    at = {}
    for level in (-40.0, -96.0, -512.0, -4096.0):
        ids, w = fme.moe_gate(level + diff, 4, score="sigmoid")
        d = fme.moe_gate_backward(level + diff, ids, g, score="sigmoid")
        loss, counts, n = fme.moe_balance_loss(level + diff, ids, score="sigmoid")
        b = fme.moe_balance_loss_backward(level + diff, counts, n, torch.ones(1, device=DEV), 4, score="sigmoid")
        at[level] = (ids, w, d, loss, b)
    for level, got in at.items():
        for x, y in zip(got, at[-40.0]):
            assert torch.equal(x, y), level
