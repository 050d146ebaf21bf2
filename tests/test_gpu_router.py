"""The gate, the balance loss, the combine's gradient: against 64-bit forms of their formulas.

Tolerances.  u = 2^-24.  An fp32 exponential of x = l - max carries the rounding of x (|x| u) and at
most 2 ulp of its own; a sum of E of them at most E u; divisions and products u each.  So a
probability is within (E + |x| + 16) u of itself, doubled here for the sums' own terms (`slack`).
Gradients are differences of such terms: the bound applies to the terms' sizes, plus the rounding to the
output's type."""
import numpy as np
import pytest
import torch

import fp8_moe_expert_gb300 as fme

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    fme.ensure_built()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def logits_of(tokens, experts, dtype, seed, spread=3.0):
    return (torch.randn((tokens, experts), generator=gen(seed), device=DEV) * spread).to(dtype)


def slack(experts, logits):
    x = logits.double()
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    return 2.0 * (experts + float((x.amax() - x.amin())) + 16.0) * 2.0 ** -24


def half_ulp(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


def scores(l, score):
    return torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)


def weights_of(l, ids, score, normalize, scale):
    s = scores(l, score).gather(1, ids)
    if normalize and score == "softmax":  # the same ratio without the other experts
        s = torch.softmax(l.gather(1, ids), 1)
    elif normalize:
        s = s / s.sum(1, True)
    return scale * s


def choice(logits, bias, top_k):
    key = logits.float() if bias is None else logits.float() + bias
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :top_k]


GATE = [(1, 2, 1), (1, 32, 8), (5, 31, 4), (16, 33, 2), (100, 64, 6), (77, 100, 32), (300, 256, 8), (40, 300, 8),
        (33, 512, 16), (9, 1024, 32), (4097, 128, 1), (3, 1, 1)]


@pytest.mark.parametrize("tokens,experts,top_k", GATE)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_and_gradient(tokens, experts, top_k, score, normalize, dtype):
    l = logits_of(tokens, experts, dtype, tokens + experts)  # bf16 logits tie often
    bias = torch.randn(experts, generator=gen(1), device=DEV) if experts % 2 else None
    ids, w = fme.moe_gate(l, top_k, score=score, bias=bias, normalize=normalize, scale=2.5)
    want = choice(l, bias, top_k)
    assert torch.equal(ids.long(), want)
    l64 = l.double().requires_grad_(True)
    w64 = weights_of(l64, want, score, normalize, 2.5)
    tol = slack(experts, l)
    assert bool(((w.double() - w64).abs() <= tol * w64).all())

    g = torch.randn((tokens, top_k), generator=gen(2), device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = fme.moe_gate_backward(l, ids, g, score=score, normalize=normalize, scale=2.5, status=st)
    assert fme.read_device_status(st)[0] == 0
    assert d.dtype == dtype
    (d64,) = torch.autograd.grad(w64, l64, g.double())
    # sizes of the terms: w (|g| + sum w |g| / scale) on the choices, p times the sum elsewhere
    w64 = w64.detach()
    share = (w64 * g.abs().double()).sum(1, True) / (2.5 if normalize else 1.0)
    term = torch.zeros_like(d64).scatter_(1, want, w64 * (g.abs().double() + share))
    if not normalize and score == "softmax":
        term = term + scores(l.double(), score) * share
    lim = 2 * tol * term + half_ulp(dtype) * d64.abs() + 1e-40
    assert bool(((d.double() - d64).abs() <= lim).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gate_gradient_against_differences(score, normalize):
    """d/dh of sum(g w(l + h v)) from the forward kernel, h = 2^-6 (exact in fp32 next to these logits)."""
    tokens, experts, top_k, h = 64, 96, 6, 2.0 ** -6
    l = torch.round(logits_of(tokens, experts, torch.float32, 3, 1.0) * 4096) / 4096
    v = torch.sign(torch.randn((tokens, experts), generator=gen(4), device=DEV))
    g = torch.randn((tokens, top_k), generator=gen(5), device=DEV)
    ids, _ = fme.moe_gate(l, top_k, score=score, normalize=normalize)
    keep = torch.zeros((experts,), device=DEV)
    d = fme.moe_gate_backward(l, ids, g, score=score, normalize=normalize).double()

    def weights(at):  # of the unmoved choice, through the kernel: each token's own ids
        i, w = fme.moe_gate(at, experts if experts <= 32 else 32, score=score, bias=keep, normalize=False)
        full = torch.zeros((tokens, experts), dtype=torch.float64, device=DEV).scatter_(1, i.long(), w.double())
        s = full.gather(1, ids.long())
        return s / s.sum(1, True) if normalize else s

    up, down = weights(l + h * v), weights(l - h * v)
    diff = ((up - down) * g.double()).sum(1) / (2 * h)
    # third derivatives of these ratios are at most 6 of the weights' size in each direction; rounding 2^-20 / h
    lim = (g.abs().double().sum(1)) * (6 * h * h + 2.0 ** -20 / h)
    assert bool(((d * v.double()).sum(1) - diff).abs().le(lim).all())


def test_gate_ties_go_to_the_lower_expert():
    l = torch.zeros((4, 70), device=DEV)
    l[1, 1::2] = 1.0
    l[2, 65] = 2.0
    l[3] = -0.0
    l[3, 0::3] = 0.0
    ids, w = fme.moe_gate(l, 4)
    assert ids.tolist() == [[0, 1, 2, 3], [1, 3, 5, 7], [65, 0, 1, 2], [0, 1, 2, 3]]
    assert bool((w[0] == 0.25).all())


@pytest.mark.parametrize("experts", [24, 64, 100, 256, 1000])
@pytest.mark.parametrize("step", [0.125, 1.0, 4.0])
def test_gate_rows_with_equal_keys(experts, step):
    """Coarse logits: a few, some, or most of a row's largest keys are equal."""
    l = torch.round(logits_of(500, experts, torch.float32, experts, 3.0) / step) * step
    bias = torch.round(torch.randn((experts,), generator=gen(1), device=DEV)) * step
    for b in (None, bias):
        for k in (1, 5, 8):
            ids, _ = fme.moe_gate(l, k, bias=b)
            assert torch.equal(ids.long(), choice(l, b, k))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_masked_logits(dtype):
    low = torch.finfo(dtype).min
    l = torch.full((6, 40), -INF, dtype=dtype, device=DEV)
    l[1, 7] = 0.5                          # fewer experts left than choices
    l[2, :] = low                          # the type's lowest value everywhere
    l[3, :] = low
    l[3, 5] = low / 2
    l[4, 3] = INF
    l[5] = 0.0
    l[5, 9] = float("nan")
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            ids, w = fme.moe_gate(l, 3, score=score, normalize=normalize)
            assert ids[:5].tolist() == [[0, 1, 2], [7, 0, 1], [0, 1, 2], [5, 0, 1], [3, 0, 1]]
            assert ids[5].tolist() == [0, 1, 2]  # a NaN is chosen last
            assert w[0].tolist() == [0.0] * 3    # nothing is left of the row
            first = 0.6224593 if score == "sigmoid" and not normalize else 1.0
            assert abs(w[1, 0].item() - first) < 1e-6 and w[1, 1:].tolist() == [0.0, 0.0]
            d = fme.moe_gate_backward(l, ids, torch.ones_like(w), score=score, normalize=normalize)
            assert bool(torch.isfinite(d[:3]).all()) and not bool(d[0].any())
    ids, w = fme.moe_gate(l, 3)
    assert torch.allclose(w[2], torch.full((3,), 1 / 3, device=DEV)) and w[3].tolist() == [1.0, 0.0, 0.0]
    assert bool(torch.isnan(w[4]).any())          # +inf under softmax
    _, w = fme.moe_gate(l, 3, normalize=False)
    assert bool(torch.isnan(w[5]).all())          # the NaN is in the denominator
    l[5, 2:] = float("nan")
    _, w = fme.moe_gate(l, 3)
    assert bool(torch.isnan(w[5]).all())          # it had to be chosen


def test_gate_backward_bad_id_is_reported_and_left_out():
    l = logits_of(2, 8, torch.float32, 1)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ids = torch.tensor([[0, 8], [-1, 3]], dtype=torch.int32, device=DEV)
    d = fme.moe_gate_backward(l, ids, torch.ones((2, 2), device=DEV), score="sigmoid", normalize=False, status=st)
    assert fme.read_device_status(st)[0] == fme.ERR_DEVICE_BAD_INDEX
    assert (d != 0).nonzero().tolist() == [[0, 0], [1, 3]]


def test_gate_empty():
    l = torch.empty((0, 16), device=DEV)
    ids, w = fme.moe_gate(l, 2)
    assert ids.shape == (0, 2) and fme.moe_gate_backward(l, ids, w).shape == (0, 16)


# ------------------------------------------------------------------ balance loss --
def balance64(l, ids, score, alpha, seq, mask):
    """(loss, counts, tokens) of float64 logits l."""
    p = scores(l, score)
    p = p / p.sum(1, True)
    experts, top_k = l.shape[1], ids.shape[1]
    counts = torch.zeros((len(seq) - 1, experts), dtype=torch.int64, device=DEV)
    tokens, terms = [], []
    for q, (lo, hi) in enumerate(zip(seq, seq[1:])):
        on = mask[lo:hi]
        t = int(on.sum())
        tokens.append(t)
        counts[q] = torch.bincount(ids[lo:hi][on].reshape(-1).long(), minlength=experts)
        if t:
            terms.append((counts[q].double() * p[lo:hi][on].sum(0)).sum() * experts / (top_k * t * t))
    loss = alpha * torch.stack(terms).mean() if terms else (l * 0).sum()
    return loss, counts, tokens


BALANCE = [(1, 2, 1, 1), (1, 32, 8, 1), (15, 31, 4, 3), (100, 33, 2, 1), (513, 64, 6, 40), (1000, 100, 8, 1),
           (2050, 256, 8, 7), (300, 512, 8, 2), (70, 1024, 32, 1), (64, 16, 2, 500), (9000, 8, 2, 1)]


@pytest.mark.parametrize("tokens,experts,top_k,seqs", BALANCE)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_balance_loss_and_gradient(tokens, experts, top_k, seqs, score, masked, dtype):
    l = logits_of(tokens, experts, dtype, tokens)
    ids = choice(l, None, top_k).int()
    rng = np.random.default_rng(tokens + seqs)
    host = [0] + sorted(rng.integers(0, tokens + 1, seqs - 1).tolist()) + [tokens]
    seq = torch.tensor(host, dtype=torch.int32, device=DEV) if seqs > 1 else None
    mask = torch.rand(tokens, generator=gen(7), device=DEV) < 0.7 if masked else None
    on = mask if masked else torch.ones(tokens, dtype=torch.bool, device=DEV)
    if masked:  # what stands in masked places does not matter
        l = torch.where(on[:, None], l, torch.full_like(l, float("nan")))
        ids = torch.where(on[:, None], ids, torch.full_like(ids, -7))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(score=score, alpha=0.3, seq_offsets=seq, token_mask=mask)
    loss, counts, n = fme.moe_balance_loss(l, ids, status=st, **kw)
    assert fme.read_device_status(st)[0] == 0
    clean = torch.where(on[:, None], l, torch.zeros_like(l)).double().requires_grad_(True)
    loss64, counts64, n64 = balance64(clean, ids, score, 0.3, host, on)
    value64 = float(loss64.detach())
    assert torch.equal(counts.long(), counts64) and n.tolist() == n64
    # all terms are positive: their sums are within (tokens + experts + sequences) u of themselves at most
    tol = slack(experts, clean.detach()) + (tokens + experts + seqs) * 2.0 ** -24
    assert abs(loss.item() - value64) <= tol * abs(value64)

    again = fme.moe_balance_loss(l, ids, **kw)
    assert torch.equal(loss, again[0])

    up = torch.full((1,), -1.7, device=DEV)
    d = fme.moe_balance_loss_backward(l, counts, n, up, top_k, **kw)
    assert d.dtype == dtype
    (d64,) = torch.autograd.grad(loss64 * -1.7, clean)
    p = scores(clean.detach(), score)
    p = p / p.sum(1, True)
    live = max(1, sum(t > 0 for t in n64))
    size = torch.zeros_like(d64)
    for q, (lo, hi) in enumerate(zip(host, host[1:])):
        if n64[q]:
            a = 1.7 * 0.3 / live * experts / (top_k * n64[q] ** 2) * counts64[q].double()
            size[lo:hi] = p[lo:hi] * (a + (p[lo:hi] * a).sum(1, True))
    size[~on] = 0.0
    lim = 2 * slack(experts, clean.detach()) * size + half_ulp(dtype) * d64.abs() + 1e-40
    assert bool(((d.double() - d64).abs() <= lim).all())
    assert not bool(d[~on].any())

    base = torch.randn((tokens, experts), generator=gen(8), device=DEV).to(dtype)
    into = base.clone()
    fme.moe_balance_loss_backward(l, counts, n, up, top_k, d_logits=into, accumulate=True, **kw)
    want = base.double() + d64
    assert bool(((into.double() - want).abs() <= lim + half_ulp(dtype) * want.abs() + 2.0 ** -24 * base.abs()).all())
    assert torch.equal(into[~on], base[~on])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(score):
    """Directional difference of the forward kernel's loss with the counts held, h = 2^-5."""
    tokens, experts, top_k, h = 256, 48, 4, 2.0 ** -5
    l = torch.round(logits_of(tokens, experts, torch.float32, 11, 1.0) * 4096) / 4096
    ids = choice(l, None, top_k).int()
    loss, counts, n = fme.moe_balance_loss(l, ids, score=score)
    d = fme.moe_balance_loss_backward(l, counts, n, torch.ones(1, device=DEV), top_k, score=score)
    for e in range(0, experts, 7):  # one expert's logits of all tokens
        v = torch.zeros_like(l)
        v[:, e] = 1.0
        up = fme.moe_balance_loss(l + h * v, ids, score=score)[0].item()
        down = fme.moe_balance_loss(l - h * v, ids, score=score)[0].item()
        # the loss is about 1 to 2; its third derivative in one direction is below 6 of it
        assert abs((up - down) / (2 * h) - d[:, e].double().sum().item()) <= 2.0 * (h * h + 2.0 ** -20 / h)


def test_balance_of_uniform_routing_is_alpha():
    tokens, experts, top_k = 96, 24, 4
    l = torch.zeros((tokens, experts), device=DEV)
    ids = (torch.arange(tokens * top_k, device=DEV) % experts).reshape(tokens, top_k).int()
    for score in ("softmax", "sigmoid"):
        loss, counts, n = fme.moe_balance_loss(l, ids, score=score, alpha=0.25)
        assert abs(loss.item() - 0.25) <= 0.25 * (tokens + experts) * 2.0 ** -23
        assert bool((counts == tokens * top_k // experts).all()) and n.tolist() == [tokens]
        d = fme.moe_balance_loss_backward(l, counts, n, torch.ones(1, device=DEV), top_k, score=score, alpha=0.25)
        assert float(d.abs().max()) <= 0.25 / tokens * 2.0 ** -20


def test_balance_nothing_counted():
    for tokens, mask in ((0, None), (5, torch.zeros(5, dtype=torch.bool, device=DEV))):
        l = torch.full((tokens, 16), -INF, device=DEV)
        ids = torch.zeros((tokens, 2), dtype=torch.int32, device=DEV)
        loss, counts, n = fme.moe_balance_loss(l, ids, token_mask=mask)
        assert loss.item() == 0.0 and not bool(counts.any()) and n.tolist() == [0]
        d = fme.moe_balance_loss_backward(l, counts, n, torch.ones(1, device=DEV), 2, token_mask=mask)
        assert not bool(d.any())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_row_of_minus_infinity_has_no_probability(score):
    l = logits_of(9, 12, torch.float32, 5)
    l[4] = -INF
    l[6, 3:] = -INF
    ids = choice(l, None, 2).int()
    loss, counts, n = fme.moe_balance_loss(l, ids, score=score)
    d = fme.moe_balance_loss_backward(l, counts, n, torch.ones(1, device=DEV), 2, score=score)
    assert np.isfinite(loss.item()) and bool(torch.isfinite(d).all()) and not bool(d[4].any())
    assert int(counts.sum()) == 18


def test_balance_bad_ids_and_sequences_are_reported():
    l = logits_of(6, 8, torch.float32, 1)
    ids = torch.tensor([[0, 1]] * 5 + [[8, -1]], dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    _, counts, _ = fme.moe_balance_loss(l, ids, status=st)
    assert fme.read_device_status(st)[0] == fme.ERR_DEVICE_BAD_INDEX and int(counts.sum()) == 10
    for off in ([0, 4, 3, 6], [1, 6], [0, 7], [0, -1, 6], [0, 5]):
        st.zero_()
        fme.moe_balance_loss(l, ids[:, :1].clamp(0, 7).contiguous(), status=st,
                             seq_offsets=torch.tensor(off, dtype=torch.int32, device=DEV))
        assert fme.read_device_status(st)[0] == fme.ERR_DEVICE_BAD_OFFSETS


def test_balance_on_a_side_stream():
    l = logits_of(5000, 64, torch.float32, 2)
    ids = choice(l, None, 4).int()
    want = fme.moe_balance_loss(l, ids)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [fme.moe_balance_loss(l, ids, stream=s)[0] for _ in range(20)]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(g, want) for g in got)


# ------------------------------------------------------------- combine's gradient --
@pytest.mark.parametrize("tokens,top_k,n", [(1, 1, 8), (1, 8, 7168), (33, 2, 1000), (200, 9, 2048), (64, 20, 264)])
def test_combine_backward(tokens, top_k, n):
    rows = tokens * top_k + 3
    y = torch.randn((rows, n), generator=gen(1), device=DEV).bfloat16()
    d_out = torch.randn((tokens, n), generator=gen(2), device=DEV).bfloat16()
    w = torch.rand((tokens, top_k), generator=gen(3), device=DEV)
    row_of = torch.randperm(rows, generator=gen(4), device=DEV)[:tokens * top_k].int().reshape(tokens, top_k)
    if tokens > 1:
        row_of[1, 0] = -1  # an assignment that was not routed
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    d_y = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device=DEV)
    d_y, dw = fme.moe_combine_backward(d_out, y, row_of, w, d_y=d_y, status=st)
    assert fme.read_device_status(st)[0] == 0
    on = row_of >= 0
    want = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device=DEV)  # rows of no assignment stay
    want[row_of[on].long()] = (w[:, :, None] * d_out.float()[:, None, :]).to(torch.bfloat16)[on]
    assert torch.equal(d_y, want)
    yv = y[row_of.clamp_min(0).long()].double()
    prod = yv * d_out.double()[:, None, :]
    assert bool(((dw.double() - prod.sum(2)).abs() <= n * 2.0 ** -24 * prod.abs().sum(2))[on].all())
    assert not bool(dw[~on].any())


def test_combine_backward_is_the_gradient_of_the_combine():
    """sum(d_out * moe_combine(y, w)) moved along w and along y, against d_weights and d_y."""
    tokens, top_k, n = 40, 4, 512
    rows = tokens * top_k
    y = torch.randint(-8, 9, (rows, n), generator=gen(1), device=DEV).bfloat16()
    d_out = torch.randint(-4, 5, (tokens, n), generator=gen(2), device=DEV).bfloat16()
    w = torch.randint(1, 9, (tokens, top_k), generator=gen(3), device=DEV).float() / 8
    row_of = torch.randperm(rows, generator=gen(4), device=DEV).int().reshape(tokens, top_k)
    d_y, dw = fme.moe_combine_backward(d_out, y, row_of, w)

    def value(y_, w_):  # small integers over 8: every step is exact
        return (fme.moe_combine(y_, row_of, w_).double() * d_out.double()).sum(1)

    for k in range(top_k):
        v = torch.zeros_like(w)
        v[:, k] = 1.0
        assert torch.equal((value(y, w + v) - value(y, w - v)) / 2, dw[:, k].double())
    v = torch.randint(-1, 2, (rows, n), generator=gen(5), device=DEV).bfloat16()
    moved = (value(y + v, w) - value(y - v, w)) / 2
    assert torch.equal(moved, (d_y.double() * v.double())[row_of.long()].sum((1, 2)))


def test_combine_backward_row_out_of_range_is_reported():
    y = torch.ones((2, 16), device=DEV).bfloat16()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    row_of = torch.tensor([[0, 2], [1, -1]], dtype=torch.int32, device=DEV)
    _, dw = fme.moe_combine_backward(torch.ones((2, 16), device=DEV).bfloat16(), y, row_of,
                                     torch.ones((2, 2), device=DEV), status=st)
    assert fme.read_device_status(st)[0] == fme.ERR_DEVICE_BAD_INDEX
    assert dw.tolist() == [[16.0, 0.0], [16.0, 0.0]]
