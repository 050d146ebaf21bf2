"""The measured cases of the FP8 block-128 expert products, the router and the combine's gradient.

Each case is one pass as a serving or training program makes it.  ``run`` computes it in plain torch operations in
32 bits, or, where ``own`` is set, through the package's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
FLOOR = 2.0 ** -100  # a block's largest magnitude is taken as at least this


# ------------------------------------------------------------------------------------------------------ the cases --
def listed():
    return [
        # One token of a decode step: its 8 experts of 32, the gate/up product (n = 2 x 2048) from bf16 hidden states.
        # What counts is how fast the chosen experts' weights are read.
        {"name": "product one token", "op": "fwd", "tokens": 1, "top_k": 8, "experts": 32, "n": 4096, "k": 7168},
        # A prefill or training batch: 8192 tokens x 8, experts of very different loads, some without tokens.
        {"name": "product 65536 rows", "op": "fwd", "tokens": 8192, "top_k": 8, "experts": 32, "n": 4096, "k": 7168},
        # The two gradients of a projection, small experts of odd sizes that fill no tile (fp32 weight gradient).
        {"name": "gradients 1999 rows", "op": "bwd", "rows": 1999, "experts": 8, "n": 1040, "k": 1392, "dw": "fp32"},
        # The down projection's gradients of a long batch, bf16 weight gradient.
        {"name": "gradients 65536 rows", "op": "bwd", "rows": 65536, "experts": 32, "n": 7168, "k": 2048,
         "dw": "bf16"},
        # A few experts' weights requantized after an optimizer step.
        {"name": "quantize weights", "op": "quant", "kind": "weights", "rows": 4, "experts": 4, "n": 2048, "k": 7168},
        # The output gradient both ways: along the rows for dgrad, along each expert's tokens for wgrad.
        {"name": "quantize both ways", "op": "quant", "kind": "both", "rows": 65536, "experts": 32, "n": 1,
         "k": 7168},
        # The router of a small decode batch: latency.
        {"name": "gate 16 tokens", "op": "gate", "tokens": 16, "experts": 32, "top_k": 8, "score": "sigmoid",
         "norm": True, "bias": True, "dtype": "bf16", "grad": False},
        # The router of a training step with its gradient.
        {"name": "gate 32768 tokens", "op": "gate", "tokens": 32768, "experts": 256, "top_k": 8, "score": "softmax",
         "norm": True, "bias": False, "dtype": "fp32", "grad": True},
        # The balance loss of a short batch, one sequence.
        {"name": "balance 1023 tokens", "op": "balance", "tokens": 1023, "experts": 32, "top_k": 4, "seqs": 1,
         "score": "softmax", "mask": False, "dtype": "fp32"},
        # The balance loss of packed sequences of odd lengths with padding tokens.
        {"name": "balance 32768 tokens", "op": "balance", "tokens": 32768, "experts": 256, "top_k": 8, "seqs": 13,
         "score": "sigmoid", "mask": True, "dtype": "bf16"},
        # The combine's gradient, a short batch of a narrow model with two experts a token.
        {"name": "combine grad 300 tokens", "op": "combine", "tokens": 300, "top_k": 2, "experts": 8, "n": 1000},
        # The combine's gradient of a training batch.
        {"name": "combine grad 16384 tokens", "op": "combine", "tokens": 16384, "top_k": 8, "experts": 32, "n": 7168},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi, step):
        v = max(lo, log(lo, hi) // step * step)
        return v + step if v == 3072 else v

    op = rng.choice(["fwd", "fwd", "bwd", "quant", "gate", "balance", "combine"])
    if op == "fwd":
        top_k = rng.choice([1, 2, 4, 6, 8])
        c = {"op": op, "tokens": log(1, 8192), "top_k": top_k, "experts": max(top_k, log(1, 48)),
             "n": width(128, 4096, 16), "k": width(128, 7168, 16)}
    elif op == "bwd":
        c = {"op": op, "rows": log(1, 65536), "experts": log(1, 48), "n": width(128, 4096, 16),
             "k": width(128, 3600, 16), "dw": rng.choice(["bf16", "fp32"])}
    elif op == "quant":
        kind = rng.choice(["weights", "both", "rows"])
        weights = kind == "weights"
        c = {"op": op, "kind": kind, "rows": 1 if weights else log(1, 65536), "experts": log(1, 32),
             "n": width(16, 2048, 16) if weights else 1, "k": width(128, 7168, 16)}
    elif op in ("gate", "balance"):
        experts = log(2, 512)
        c = {"op": op, "tokens": log(1, 32768), "experts": experts, "top_k": rng.randint(1, min(8, experts)),
             "score": rng.choice(["softmax", "sigmoid"]), "dtype": rng.choice(["bf16", "fp32"])}
        if op == "gate":
            c.update(norm=rng.random() < 0.7, bias=rng.random() < 0.5, grad=rng.random() < 0.6)
        else:
            c.update(seqs=log(1, 64), mask=rng.random() < 0.5)
        if c["tokens"] * experts > 32768 * 256:
            c["tokens"] = 32768 * 256 // experts
    else:
        top_k = rng.randint(1, 8)
        c = {"op": op, "tokens": log(1, 16384), "top_k": top_k, "experts": max(top_k, log(2, 64)),
             "n": width(64, 7168, 8)}
    return c


def work(case):
    op = case["op"]
    if op == "fwd":
        t, e, n, k = case["tokens"], case["experts"], case["n"], case["k"]
        rows = t * case["top_k"]
        return {"bytes": t * k * 2 + min(e, rows) * n * k + rows * n * 2, "flops": 2 * rows * n * k}
    if op == "bwd":
        r, e, n, k = case["rows"], case["experts"], case["n"], case["k"]
        wide = 4 if case["dw"] == "fp32" else 2
        return {"bytes": 2 * r * n + r * k + min(e, r) * n * k + 2 * r * k + wide * e * n * k, "flops": 4 * r * n * k}
    if op == "quant":
        if case["kind"] == "weights":
            el = case["experts"] * case["n"] * case["k"]
            return {"bytes": 3 * el, "flops": 2 * el}
        el = case["rows"] * case["k"]
        return {"bytes": (4 if case["kind"] == "both" else 3) * el, "flops": 2 * el}
    if op == "gate":
        el, sel = case["tokens"] * case["experts"], case["tokens"] * case["top_k"]
        wide = 4 if case["dtype"] == "fp32" else 2
        grad = el * wide + sel * 4 if case["grad"] else 0
        return {"bytes": el * wide + sel * 8 + grad, "flops": 8 * el}
    if op == "balance":
        el, sel = case["tokens"] * case["experts"], case["tokens"] * case["top_k"]
        wide = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 2 * el * wide + sel * 4 + 4 * case["seqs"] * case["experts"], "flops": 12 * el}
    t, n, sel = case["tokens"], case["n"], case["tokens"] * case["top_k"]
    return {"bytes": 2 * t * n + 4 * sel * n + 12 * sel, "flops": 3 * sel * n}


# ------------------------------------------------------------------------------------------------------- inputs --
def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(shape, std, g):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g)


def activations(rows, cols, std, g):
    """N(0, std^2) with a few channels and rows far from the rest, as hidden states and their gradients have."""
    x = normal((rows, cols), std, g)
    x[:, torch.randint(cols, (max(1, cols // 1000),), generator=g, device=DEV)] *= 50.0
    x[torch.randint(rows, (max(1, rows // 100),), generator=g, device=DEV)] *= 1e-3
    return x.to(torch.bfloat16)


def grouping(rows, experts, seed):
    """Row offsets of skewed expert loads (Zipf 1.2 in a random order, about a tenth of the experts empty)."""
    rng = np.random.default_rng(seed)
    p = np.arange(1, experts + 1, dtype=np.float64) ** -1.2
    p[experts - experts // 10:] = 0.0
    counts = rng.multinomial(rows, rng.permutation(p / p.sum()))
    host = np.concatenate([[0], np.cumsum(counts)])
    return host.tolist(), torch.from_numpy(host.astype(np.int32)).to(DEV)


def routing(tokens, top_k, experts, seed):
    """Distinct experts of each token, Zipf-popular, and the grouping by expert that follows from them."""
    g = generator(seed)
    order = torch.randperm(experts, generator=g, device=DEV)
    pop = torch.empty(experts, device=DEV)
    pop[order] = -1.2 * torch.log(torch.arange(1, experts + 1, device=DEV, dtype=torch.float32))
    noise = -torch.log(-torch.log(torch.rand((tokens, experts), generator=g, device=DEV).clamp(1e-9, 1 - 1e-6)))
    ids = torch.topk(pop + noise, top_k, dim=1).indices
    src = torch.sort(ids.reshape(-1), stable=True).indices  # the assignment at each grouped row
    row_of = torch.empty_like(src)
    row_of[src] = torch.arange(tokens * top_k, device=DEV)
    counts = torch.bincount(ids.reshape(-1), minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    return (ids.int(), row_of.reshape(tokens, top_k).int(), src.int(), offsets.int(), offsets.tolist())


def to_blocks(x, rows, cols):
    """x [.., R, C] cut into blocks of rows x cols (zeros at the ragged ends) -> [.., R', rows, C', cols]."""
    r, c = x.shape[-2:]
    x = torch.nn.functional.pad(x, (0, -c % cols, 0, -r % rows))
    return x.reshape(*x.shape[:-2], x.shape[-2] // rows, rows, x.shape[-1] // cols, cols)


def plain_quantize(x, rows, cols):
    """Codes (FP8 E4M3) of x [.., R, C] with one scale for each block of rows x cols, and the scales [.., R', C']."""
    b = to_blocks(x.float(), rows, cols)
    top = b.abs().amax(dim=(-3, -1), keepdim=True).clamp_min(FLOOR)
    q = (b * (448.0 / top)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    s = (top / 448.0).reshape(*top.shape[:-4], top.shape[-4], top.shape[-2])
    r, c = x.shape[-2:]
    q = q.view(torch.uint8).reshape(*x.shape[:-2], b.shape[-4] * rows, b.shape[-2] * cols)
    return q[..., :r, :c].contiguous(), s


def plain_rows(x):
    """Codes of x [R, C] in blocks of 128 along each row, scales [C', R]."""
    q, s = plain_quantize(x, 1, 128)
    return q, s.t().contiguous()


def padded_positions(offsets, rows, experts):
    """For each padded position (every expert starts at a multiple of 128) its row, or -1; and the padded offsets."""
    counts = (offsets[1:] - offsets[:-1]).long()
    padded = torch.zeros(experts + 1, dtype=torch.int64, device=DEV)
    padded[1:] = torch.cumsum((counts + 127) // 128 * 128, 0)
    ld = (rows + 127 * experts) // 128 * 128
    at = torch.arange(ld, device=DEV)
    e = torch.searchsorted(padded, at, right=True).clamp_max(experts) - 1
    local = at - padded[e]
    row = offsets[e].long() + local
    return torch.where((local < counts[e]) & (at < padded[experts]), row, -1), padded


def plain_cols(x, offsets, experts):
    """Codes of x [R, C] in blocks of 128 along each expert's tokens, at padded positions; scales [positions/128, C]."""
    row, padded = padded_positions(offsets, x.shape[0], experts)
    grouped = torch.where((row >= 0)[:, None], x[row.clamp_min(0)], torch.zeros((), dtype=x.dtype, device=DEV))
    q, s = plain_quantize(grouped, 128, 1)
    return q, s, padded.int()


def quantized_weights(experts, n, k, g):
    """A model's stored expert weights: codes and one scale for each 128 x 128 block."""
    codes = torch.empty((experts, n, k), dtype=torch.uint8, device=DEV)
    scale = torch.empty((experts, -(-n // 128), -(-k // 128)), dtype=torch.float32, device=DEV)
    for e in range(experts):
        codes[e], scale[e] = plain_quantize(normal((n, k), 0.02, g).to(torch.bfloat16), 128, 128)
    return codes, scale


def prepare(case, seed):
    op, g = case["op"], generator(seed)
    s = dict(case)
    if op == "fwd":
        _, s["row_of"], s["src_row"], s["offsets"], s["host"] = routing(case["tokens"], case["top_k"],
                                                                        case["experts"], seed)
        s["x"] = activations(case["tokens"], case["k"], 1.0, g)
        s["w"], s["w_scale"] = quantized_weights(case["experts"], case["n"], case["k"], g)
    elif op == "bwd":
        e, rows = case["experts"], case["rows"]
        s["host"], s["offsets"] = grouping(rows, e, seed)
        s["w"], s["w_scale"] = quantized_weights(e, case["n"], case["k"], g)
        dy = activations(rows, case["n"], 0.01, g)
        s["dy"], s["dy_scale"] = plain_rows(dy)
        s["dyc"], s["dyc_scale"], s["padded"] = plain_cols(dy, s["offsets"], e)
        s["xc"], s["xc_scale"], _ = plain_cols(activations(rows, case["k"], 1.0, g), s["offsets"], e)
        s["padded_host"] = s["padded"].tolist()
    elif op == "quant":
        if case["kind"] == "weights":
            s["x"] = normal((case["experts"], case["n"], case["k"]), 0.02, g).to(torch.bfloat16)
        else:
            s["x"] = activations(case["rows"], case["k"], 0.01, g)
            s["host"], s["offsets"] = grouping(case["rows"], case["experts"], seed)
    elif op in ("gate", "balance"):
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        lean = 0.7 * normal((e,), 1.0, g)  # some experts are preferred by all tokens
        s["logits"] = (1.3 * normal((t, e), 1.0, g) + lean).to(torch.bfloat16 if case["dtype"] == "bf16"
                                                               else torch.float32)
        if op == "gate":
            s["bias_t"] = 0.2 * normal((e,), 1.0, g) if case["bias"] else None
            s["dw"] = normal((t, k), 0.1, g)
        else:
            s["ids"] = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices[:, :k].int()
            rng = np.random.default_rng(seed)
            cuts = np.sort(rng.integers(0, t + 1, case["seqs"] - 1))  # empty sequences may come up
            host = np.concatenate([[0], cuts, [t]]).astype(np.int32)
            s["seq"] = torch.from_numpy(host).to(DEV)
            s["mask_t"] = torch.rand((t,), generator=g, device=DEV) < 0.9 if case["mask"] else None
            s["d_loss"] = torch.full((1,), 1.0 + seed % 7, device=DEV)
    else:
        t, n = case["tokens"], case["n"]
        _, s["row_of"], _, _, _ = routing(t, case["top_k"], case["experts"], seed)
        w = torch.rand((t, case["top_k"]), generator=g, device=DEV) + 0.05
        s["weights"] = w / w.sum(dim=1, keepdim=True)
        s["y"] = normal((t * case["top_k"], n), 1.0, g).to(torch.bfloat16)
        s["d_out"] = normal((t, n), 0.01, g).to(torch.bfloat16)
    return s


# -------------------------------------------------------------------------------------------------- one pass --
def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import fp8_moe_expert_gb300 as fme

    op = s["op"]
    if op == "fwd":
        q, sc = fme.quantize_fp8_block128(s["x"], src_row=s["src_row"], top_k=s["top_k"])
        return fme.grouped_gemm_fwd_fp8_block128(q, sc, s["w"], s["w_scale"], s["offsets"])
    if op == "bwd":
        dx = fme.grouped_gemm_dgrad_fp8_block128(s["dy"], s["dy_scale"], s["w"], s["w_scale"], s["offsets"])
        dw = fme.grouped_gemm_wgrad_fp8_block128(s["dyc"], s["dyc_scale"], s["xc"], s["xc_scale"], s["padded"],
                                                 dtype=torch.float32 if s["dw"] == "fp32" else torch.bfloat16)
        return dx, dw
    if op == "quant":
        if s["kind"] == "weights":
            q, sc = fme.quantize_fp8_block128_weights(s["x"])
            return as_values(q), sc
        if s["kind"] == "rows":
            q, sc = fme.quantize_fp8_block128(s["x"])
            return as_values(q), sc
        (q, sc), (qc, scc, padded) = fme.quantize_fp8_block128_rowcol(s["x"], s["offsets"])
        return as_values(q), sc, as_values(qc), scc, padded
    if op == "gate":
        ids, w = fme.moe_gate(s["logits"], s["top_k"], score=s["score"], bias=s["bias_t"], normalize=s["norm"],
                              scale=2.5)
        if not s["grad"]:
            return ids, w
        d = fme.moe_gate_backward(s["logits"], ids, s["dw"], score=s["score"], normalize=s["norm"], scale=2.5)
        return ids, w, d
    if op == "balance":
        kw = dict(score=s["score"], alpha=0.01, seq_offsets=s["seq"], token_mask=s["mask_t"])
        loss, counts, tokens = fme.moe_balance_loss(s["logits"], s["ids"], **kw)
        d = fme.moe_balance_loss_backward(s["logits"], counts, tokens, s["d_loss"], s["top_k"], **kw)
        return loss, counts, tokens, d
    return fme.moe_combine_backward(s["d_out"], s["y"], s["row_of"], s["weights"])


def as_values(codes):
    return codes.view(torch.float8_e4m3fn)


def row_values(codes, scale):
    """What row-wise codes [R, C] with scales [C', R] stand for, in 32 bits."""
    return as_values(codes).float() * scale.t().repeat_interleave(128, dim=1)[:, :codes.shape[1]]


def weight_values(codes, scale):
    wide = scale.repeat_interleave(128, dim=-2).repeat_interleave(128, dim=-1)
    return as_values(codes).float() * wide[..., :codes.shape[-2], :codes.shape[-1]]


def run_plain(s):
    op = s["op"]
    if op == "fwd":
        q, sc = plain_rows(s["x"][s["src_row"].long() // s["top_k"]])
        y = torch.empty((q.shape[0], s["n"]), dtype=torch.bfloat16, device=DEV)
        for e, (lo, hi) in enumerate(zip(s["host"], s["host"][1:])):  # one library product for each expert with rows
            if hi > lo:
                y[lo:hi] = row_values(q[lo:hi], sc[:, lo:hi]) @ weight_values(s["w"][e], s["w_scale"][e]).t()
        return y
    if op == "bwd":
        e_, n, k = s["w"].shape
        dx = torch.empty((s["rows"], k), dtype=torch.bfloat16, device=DEV)
        dw = torch.zeros((e_, n, k), dtype=torch.float32 if s["dw"] == "fp32" else torch.bfloat16, device=DEV)
        for e in range(e_):
            lo, hi, a, b = *s["host"][e:e + 2], *s["padded_host"][e:e + 2]
            if hi > lo:
                w = weight_values(s["w"][e], s["w_scale"][e])
                dx[lo:hi] = row_values(s["dy"][lo:hi], s["dy_scale"][:, lo:hi]) @ w
                dy = as_values(s["dyc"][a:b]).float() * s["dyc_scale"][a // 128:b // 128].repeat_interleave(128, 0)
                x = as_values(s["xc"][a:b]).float() * s["xc_scale"][a // 128:b // 128].repeat_interleave(128, 0)
                dw[e] = dy.t() @ x
        return dx, dw
    if op == "quant":
        if s["kind"] == "weights":
            q, sc = plain_quantize(s["x"], 128, 128)
            return as_values(q), sc
        q, sc = plain_rows(s["x"])
        if s["kind"] == "rows":
            return as_values(q), sc
        qc, scc, padded = plain_cols(s["x"], s["offsets"], s["experts"])
        return as_values(q), sc, as_values(qc), scc, padded
    if op == "gate":
        l, k = s["logits"].float(), s["top_k"]
        key = l if s["bias_t"] is None else l + s["bias_t"]
        ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
        p = torch.softmax(l, dim=1) if s["score"] == "softmax" else torch.sigmoid(l)
        chosen = p.gather(1, ids)
        total = chosen.sum(dim=1, keepdim=True)
        w = 2.5 * chosen / total if s["norm"] else 2.5 * chosen
        if not s["grad"]:
            return ids.int(), w
        dw = 2.5 * s["dw"]
        dp = (dw - (chosen / total * dw).sum(dim=1, keepdim=True)) / total if s["norm"] else dw
        dense = torch.zeros_like(p).scatter_(1, ids, dp)
        if s["score"] == "softmax":
            d = p * (dense - (p * dense).sum(dim=1, keepdim=True))
        else:
            d = dense * p * (1 - p)
        return ids.int(), w, d.to(s["logits"].dtype)
    if op == "balance":
        return plain_balance(s)
    rows, w = s["row_of"].long(), s["weights"]
    d_out = s["d_out"].float()
    y = s["y"][rows].float()
    dw = (y * d_out[:, None, :]).sum(dim=2)
    dy = torch.empty_like(s["y"])
    dy[rows.reshape(-1)] = (w[:, :, None] * d_out[:, None, :]).to(torch.bfloat16).reshape(-1, s["n"])
    return dy, dw


def plain_balance(s):
    l, e, k, seqs = s["logits"].float(), s["experts"], s["top_k"], s["seqs"]
    raw = torch.softmax(l, dim=1) if s["score"] == "softmax" else torch.sigmoid(l)
    z = raw.sum(dim=1, keepdim=True)
    p = raw if s["score"] == "softmax" else raw / z
    at = torch.arange(l.shape[0], device=DEV)
    seq = torch.searchsorted(s["seq"].long(), at, right=True) - 1
    counted = torch.ones_like(at, dtype=torch.bool) if s["mask_t"] is None else s["mask_t"]
    tokens = torch.zeros(seqs, dtype=torch.int64, device=DEV).index_add_(0, seq, counted.long())
    flat = (seq[:, None] * e + s["ids"].long()).reshape(-1)
    counts = torch.zeros(seqs * e, dtype=torch.int64, device=DEV).index_add_(
        0, flat, counted.long()[:, None].expand(-1, k).reshape(-1)).reshape(seqs, e)
    sums = torch.zeros((seqs, e), device=DEV).index_add_(0, seq, p * counted[:, None])
    live = (tokens > 0).sum().clamp_min(1)
    part = 0.01 * e / (k * live * tokens.clamp_min(1).float() ** 2)  # of each sequence
    loss = (part * (counts * sums).sum(dim=1)).sum().reshape(1)
    a = (s["d_loss"] * part)[seq, None] * counts.float()[seq] * counted[:, None]
    inner = a - (p * a).sum(dim=1, keepdim=True)
    d = p * inner if s["score"] == "softmax" else raw * (1 - raw) / z * inner
    return loss, counts.int(), tokens.int(), d.to(s["logits"].dtype)


# ---------------------------------------------------------------------------------------- the definition, in 64 bits --
def e4m3_f64(v):
    """The nearest E4M3 value of each v, ties to the even one, no value past 448."""
    _, ex = torch.frexp(v)
    step = torch.pow(torch.full_like(v, 2.0), (ex - 1).clamp_min(-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def exact_rows(x):
    """Values of the codes of x [R, C] along its rows, and the scales [R, C']."""
    r, c = x.shape
    cb = -(-c // 128)
    full = torch.zeros((r, cb * 128), dtype=torch.float64, device=DEV)
    full[:, :c] = x.double()
    b = full.view(r, cb, 128)
    scale = b.abs().max(dim=2).values.clamp_min(FLOOR) / 448.0
    return e4m3_f64(b / scale[:, :, None]).view(r, cb * 128)[:, :c], scale


def exact_segments(host):
    return [(e, lo, hi) for e, (lo, hi) in enumerate(zip(host, host[1:])) if hi > lo]


def exact_row_operand(codes, scale):
    c = codes.shape[1]
    v = as_values(codes).float().double()
    at = torch.arange(c, device=DEV) // 128
    return v * scale.double()[at].t()


def exact_weight_operand(codes, scale):
    i, j = (torch.arange(m, device=DEV) // 128 for m in codes.shape)
    return as_values(codes).float().double() * scale.double()[i][:, j]


def exact_col_operand(codes, scale, a, b):
    i = torch.arange(a, b, device=DEV) // 128
    return as_values(codes[a:b]).float().double() * scale.double()[i]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "fwd":
        q, sc = exact_rows(s["x"])
        x = q * sc.repeat_interleave(128, dim=1)[:, :case["k"]]
        y = torch.empty((case["tokens"] * case["top_k"], case["n"]), dtype=torch.float64, device=DEV)
        token = torch.div(s["src_row"].long(), case["top_k"], rounding_mode="floor")
        for e, lo, hi in exact_segments(s["host"]):
            y[lo:hi] = torch.mm(x[token[lo:hi]], exact_weight_operand(s["w"][e], s["w_scale"][e]).t())
        return y
    if op == "bwd":
        dx = torch.empty((case["rows"], case["k"]), dtype=torch.float64, device=DEV)
        dw = torch.zeros((case["experts"], case["n"], case["k"]), dtype=torch.float64, device=DEV)
        for e, lo, hi in exact_segments(s["host"]):
            a, b = s["padded_host"][e], s["padded_host"][e + 1]
            w = exact_weight_operand(s["w"][e], s["w_scale"][e])
            dx[lo:hi] = torch.mm(exact_row_operand(s["dy"][lo:hi], s["dy_scale"][:, lo:hi]), w)
            dw[e] = torch.mm(exact_col_operand(s["dyc"], s["dyc_scale"], a, b).t(),
                             exact_col_operand(s["xc"], s["xc_scale"], a, b))
        return dx, dw
    if op == "quant":
        return exact_quant(case, s)
    if op == "gate":
        return exact_gate(case, s)
    if op == "balance":
        return exact_balance(case, s)
    rows = s["row_of"].long()
    dy = torch.empty(s["y"].shape, dtype=torch.float64, device=DEV)
    dw = torch.empty(rows.shape, dtype=torch.float64, device=DEV)
    g = s["d_out"].double()
    for j in range(case["top_k"]):
        dw[:, j] = torch.einsum("tn,tn->t", g, s["y"][rows[:, j]].double())
        dy[rows[:, j]] = g * s["weights"][:, j:j + 1].double()
    return dy, dw


def exact_quant(case, s):
    if case["kind"] == "weights":
        e, n, k = s["x"].shape
        nb, kb = -(-n // 128), -(-k // 128)
        vals = torch.empty((e, n, k), dtype=torch.float64, device=DEV)
        scale = torch.empty((e, nb, kb), dtype=torch.float64, device=DEV)
        for i in range(nb):
            for j in range(kb):
                b = s["x"][:, i * 128:(i + 1) * 128, j * 128:(j + 1) * 128].double()
                scale[:, i, j] = b.abs().flatten(1).max(dim=1).values.clamp_min(FLOOR) / 448.0
                vals[:, i * 128:(i + 1) * 128, j * 128:(j + 1) * 128] = e4m3_f64(b / scale[:, i, j, None, None])
        return vals, scale
    q, sc = exact_rows(s["x"])
    if case["kind"] == "rows":
        return q, sc.t().contiguous()
    experts, c = case["experts"], case["k"]
    ld = (case["rows"] + 127 * experts) // 128 * 128
    vals = torch.zeros((ld, c), dtype=torch.float64, device=DEV)
    scale = torch.full((ld // 128, c), FLOOR / 448.0, dtype=torch.float64, device=DEV)
    at = 0
    for e, (lo, hi) in enumerate(zip(s["host"], s["host"][1:])):
        if hi > lo:
            pad = torch.zeros((-(-(hi - lo) // 128) * 128, c), dtype=torch.float64, device=DEV)
            pad[:hi - lo] = s["x"][lo:hi].double()
            v, f = exact_rows(pad.t().contiguous())
            vals[at:at + pad.shape[0]] = v.t()
            scale[at // 128:(at + pad.shape[0]) // 128] = f.t()
            at += pad.shape[0]
    return q, sc.t().contiguous(), vals, scale, None


def exact_gate(case, s):
    l, k = s["logits"].double(), case["top_k"]
    key = s["logits"].float() if s["bias_t"] is None else s["logits"].float() + s["bias_t"]  # the key is a 32-bit sum
    ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :k]
    l.requires_grad_(bool(case["grad"]))
    sel = l.gather(1, ids)
    if case["score"] == "softmax":
        w = torch.exp(sel - (torch.logsumexp(sel, 1, True) if case["norm"] else torch.logsumexp(l, 1, True)))
    else:
        w = 1 / (1 + torch.exp(-sel))
        w = w / w.sum(1, True) if case["norm"] else w
    w = 2.5 * w
    if not case["grad"]:
        return None, w.detach()
    (d,) = torch.autograd.grad(w, l, s["dw"].double())
    return None, w.detach(), d


def exact_balance(case, s):
    l, e, k = s["logits"].double().requires_grad_(True), case["experts"], case["top_k"]
    host = s["seq"].tolist()
    on = torch.ones(case["tokens"], dtype=torch.bool, device=DEV) if s["mask_t"] is None else s["mask_t"]
    terms = []
    for lo, hi in zip(host, host[1:]):
        keep = on[lo:hi]
        t = int(keep.sum())
        if t == 0:
            continue
        v = l[lo:hi][keep]
        p = torch.exp(v - torch.logsumexp(v, 1, True)) if case["score"] == "softmax" else 1 / (1 + torch.exp(-v))
        p = p / p.sum(1, True)
        f = torch.bincount(s["ids"][lo:hi][keep].reshape(-1).long(), minlength=e).double() * e / (k * t)
        terms.append((f * p.mean(0)).sum())
    if not terms:
        return torch.zeros(1, dtype=torch.float64, device=DEV), None, None, torch.zeros_like(l)
    loss = 0.01 * torch.stack(terms).mean()
    (d,) = torch.autograd.grad(loss * s["d_loss"].double()[0], l)
    return loss.detach().reshape(1), None, None, d
