"""The measured cases of the bf16 expert products, the products of few rows with NVFP4 weights, the bf16 activation
and the grouping of bf16 rows.

Each case is one pass as a serving or training program makes it.  ``run`` computes it in plain torch operations in
32 bits, or, where ``own`` is set, through the package's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------------------ the cases --
def listed():
    return [
        # One token of a decode step in bf16: its 8 experts of 32, the gate/up product (n = 2 x 2048).  What counts is
        # how fast the chosen experts' weights are read.
        {"name": "bf16 product one token", "op": "fwd", "tokens": 1, "top_k": 8, "experts": 32, "n": 4096, "k": 7168},
        # A short batch of a small layer with odd sizes that fill no tile.
        {"name": "bf16 product 333 tokens", "op": "fwd", "tokens": 333, "top_k": 3, "experts": 8, "n": 1048,
         "k": 1400},
        # A prefill or training batch: 8192 tokens x 8, experts of very different loads, some without tokens.
        {"name": "bf16 product 65536 rows", "op": "fwd", "tokens": 8192, "top_k": 8, "experts": 32, "n": 4096,
         "k": 7168},
        # The two gradients of a projection, small experts of odd sizes (fp32 weight gradient).
        {"name": "bf16 gradients 1999 rows", "op": "bwd", "rows": 1999, "experts": 8, "n": 1048, "k": 1400,
         "dw": "fp32"},
        # The down projection's gradients of a long batch, bf16 weight gradient.
        {"name": "bf16 gradients 65536 rows", "op": "bwd", "rows": 65536, "experts": 32, "n": 7168, "k": 2048,
         "dw": "bf16"},
        # One token of a decode step with NVFP4 weights: gate/up product and activation of its 8 experts.
        {"name": "4-bit gate/up one token", "op": "gemv", "tokens": 1, "top_k": 8, "experts": 32, "n": 4096, "k": 7168,
         "swiglu": True},
        # A small decode batch's down projection: rows are grouped already, several to most experts.
        {"name": "4-bit down 16 tokens", "op": "gemv", "tokens": 16, "top_k": 8, "experts": 32, "n": 7168, "k": 2048,
         "swiglu": False},
        # Rows of odd number and width, a few experts.
        {"name": "4-bit product 37 tokens", "op": "gemv", "tokens": 37, "top_k": 2, "experts": 8, "n": 1000, "k": 1344,
         "swiglu": False},
        # The activation of a small decode batch: latency.
        {"name": "swiglu 64 rows", "op": "act", "rows": 64, "inter": 2048, "grad": False},
        # The activation of a training step with its gradient.
        {"name": "swiglu 65536 rows", "op": "act", "rows": 65536, "inter": 2048, "grad": True},
        # Grouping a short batch by expert: latency.
        {"name": "group 32 tokens", "op": "group", "tokens": 32, "top_k": 8, "experts": 32, "n": 7168},
        # Grouping a training batch.
        {"name": "group 8192 tokens", "op": "group", "tokens": 8192, "top_k": 8, "experts": 32, "n": 7168},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi, step):
        return max(lo, log(lo, hi) // step * step)

    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "gemv", "gemv", "act", "group"])
    top_k = rng.choice([1, 2, 3, 4, 6, 8])
    experts = max(top_k, log(1, 48))
    if op == "fwd":
        return {"op": op, "tokens": log(1, 8192), "top_k": top_k, "experts": min(experts, 32),
                "n": width(64, 4096, 8), "k": width(64, 7168, 8)}
    if op == "bwd":
        return {"op": op, "rows": log(1, 65536), "experts": experts, "n": width(64, 4096, 8), "k": width(64, 3584, 8),
                "dw": rng.choice(["bf16", "fp32"])}
    if op == "gemv":
        swiglu = rng.random() < 0.5
        return {"op": op, "tokens": log(1, 64), "top_k": top_k, "experts": min(experts, 32),
                "n": width(256, 4096, 256) if swiglu else width(64, 7168, 8),
                "k": width(64, 7168 if swiglu else 4096, 64), "swiglu": swiglu}
    if op == "act":
        return {"op": op, "rows": log(1, 65536), "inter": width(64, 2048, 8), "grad": rng.random() < 0.6}
    return {"op": op, "tokens": log(1, 8192), "top_k": top_k, "experts": experts, "n": width(64, 7168, 8)}


def work(case):
    op = case["op"]
    if op == "fwd":
        t, e, n, k = case["tokens"], case["experts"], case["n"], case["k"]
        rows = t * case["top_k"]
        return {"bytes": 2 * (t * k + min(e, rows) * n * k + rows * n), "flops": 2 * rows * n * k}
    if op == "bwd":
        r, e, n, k = case["rows"], case["experts"], case["n"], case["k"]
        wide = 4 if case["dw"] == "fp32" else 2
        return {"bytes": 2 * (r * n + 2 * r * k + min(e, r) * n * k) + wide * e * n * k, "flops": 4 * r * n * k}
    if op == "gemv":
        t, n, k = case["tokens"], case["n"], case["k"]
        rows = t * case["top_k"]
        hit = min(case["experts"], rows)
        x_rows = t if case["swiglu"] else rows
        out = n // 2 if case["swiglu"] else n
        return {"bytes": hit * (n * k * 9 // 16 + 4 * n) + 2 * x_rows * k + 2 * rows * out, "flops": 2 * rows * n * k}
    if op == "act":
        el = case["rows"] * case["inter"]
        return {"bytes": 2 * el * (3 + (3 if case["grad"] else 0)), "flops": el * (20 if case["grad"] else 6)}
    t, n, sel = case["tokens"], case["n"], case["tokens"] * case["top_k"]
    return {"bytes": 2 * t * n + 2 * sel * n + 4 * sel, "flops": 0}


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
    counts = torch.bincount(ids.reshape(-1), minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    return src.int(), offsets.int(), offsets.tolist()


def tile_index(row0, rows, groups, device=DEV):
    """Where the tiled layout keeps the scales of rows row0 .. row0 + rows, `groups` (a multiple of 4) to a row."""
    r = torch.arange(row0, row0 + rows, device=device)[:, None]
    c = torch.arange(groups, device=device)[None, :]
    return (r // 128 * (groups // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4


def nvfp4_weights(experts, n, k, g):
    """A model's stored expert weights: E2M1 codes two to a byte, an E4M3 scale per 16 values in tiles of 128 rows x 4,
    and one fp32 scale to a row."""
    rows = experts * n
    codes = torch.empty((rows, k // 2), dtype=torch.uint8, device=DEV)
    sf = torch.zeros((rows + 127) // 128 * 128 * (k // 16), dtype=torch.uint8, device=DEV)
    scale = torch.empty((rows,), dtype=torch.float32, device=DEV)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    for e in range(experts):
        b = normal((n, k), 0.02, g).to(torch.bfloat16).float().reshape(n, k // 16, 16)
        top = b.abs().amax(dim=2)
        s = top.amax(dim=1) / 2688.0
        sb = (top / (6.0 * s)[:, None]).clamp(max=448.0).to(torch.float8_e4m3fn)
        unit = sb.float() * s[:, None]
        q = torch.where(unit > 0, 1.0 / unit, torch.zeros_like(unit))[:, :, None] * b
        c = (torch.bucketize(q.abs(), borders) + 8 * (q < 0)).to(torch.uint8).reshape(n, k // 2, 2)
        codes[e * n:(e + 1) * n] = c[:, :, 0] + 16 * c[:, :, 1]
        sf[tile_index(e * n, n, k // 16)] = sb.view(torch.uint8)
        scale[e * n:(e + 1) * n] = s
    return codes, sf, scale


def prepare(case, seed):
    op, g = case["op"], generator(seed)
    s = dict(case)
    if op == "fwd":
        s["src_row"], s["offsets"], s["host"] = routing(case["tokens"], case["top_k"], case["experts"], seed)
        s["x"] = activations(case["tokens"], case["k"], 1.0, g)
        s["w"] = torch.empty((case["experts"], case["n"], case["k"]), dtype=torch.bfloat16, device=DEV)
        for e in range(case["experts"]):
            s["w"][e] = normal((case["n"], case["k"]), 0.02, g)
    elif op == "bwd":
        s["host"], s["offsets"] = grouping(case["rows"], case["experts"], seed)
        s["w"] = torch.empty((case["experts"], case["n"], case["k"]), dtype=torch.bfloat16, device=DEV)
        for e in range(case["experts"]):
            s["w"][e] = normal((case["n"], case["k"]), 0.02, g)
        s["dy"] = activations(case["rows"], case["n"], 0.01, g)
        s["x"] = activations(case["rows"], case["k"], 1.0, g)
    elif op == "gemv":
        s["src_row"], s["offsets"], s["host"] = routing(case["tokens"], case["top_k"], case["experts"], seed)
        rows = case["tokens"] if case["swiglu"] else case["tokens"] * case["top_k"]
        s["x"] = activations(rows, case["k"], 1.0, g)
        s["codes"], s["sf"], s["scale"] = nvfp4_weights(case["experts"], case["n"], case["k"], g)
    elif op == "act":
        s["gate_up"] = activations(case["rows"], 2 * case["inter"], 1.5, g)
        s["dh"] = activations(case["rows"], case["inter"], 0.01, g)
    else:
        s["src_row"], _, _ = routing(case["tokens"], case["top_k"], case["experts"], seed)
        s["x"] = activations(case["tokens"], case["n"], 1.0, g)
    return s


# -------------------------------------------------------------------------------------------------- one pass --
def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import fp8_moe_expert_gb300 as fme

    op = s["op"]
    if op == "fwd":
        rows = fme.moe_permute(s["x"], s["src_row"], s["top_k"])
        return fme.grouped_gemm_fwd_bf16(rows, s["w"], s["offsets"])
    if op == "bwd":
        dx = fme.grouped_gemm_dgrad_bf16(s["dy"], s["w"], s["offsets"])
        dw = fme.grouped_gemm_wgrad_bf16(s["dy"], s["x"], s["offsets"],
                                         dtype=torch.float32 if s["dw"] == "fp32" else torch.bfloat16)
        return dx, dw
    if op == "gemv":
        if s["swiglu"]:
            return fme.grouped_gemv_nvfp4_swiglu(s["x"], s["codes"], s["sf"], s["scale"], s["offsets"],
                                                 src_row=s["src_row"], top_k=s["top_k"])
        return fme.grouped_gemv_nvfp4(s["x"], s["codes"], s["sf"], s["scale"], s["offsets"])
    if op == "act":
        h = fme.swiglu(s["gate_up"])
        return (h, fme.swiglu_backward(s["gate_up"], s["dh"])) if s["grad"] else h
    return fme.moe_permute(s["x"], s["src_row"], s["top_k"])


def weight_values(s, e):
    """What expert e's codes and scales stand for, [n, k] in 32 bits."""
    n, k = s["n"], s["k"]
    c = s["codes"][e * n:(e + 1) * n]
    c = torch.stack([c & 15, c >> 4], dim=2).reshape(n, k).int()
    v = torch.tensor(E2M1 + tuple(-a for a in E2M1), device=DEV)[c]
    sb = s["sf"][tile_index(e * n, n, k // 16)].view(torch.float8_e4m3fn).float()
    return v * sb.repeat_interleave(16, dim=1) * s["scale"][e * n:(e + 1) * n, None]


def run_plain(s):
    op = s["op"]
    if op == "fwd":
        x = s["x"][s["src_row"].long() // s["top_k"]].float()
        y = torch.empty((x.shape[0], s["n"]), dtype=torch.bfloat16, device=DEV)
        for e, (lo, hi) in enumerate(zip(s["host"], s["host"][1:])):  # one library product for each expert with rows
            if hi > lo:
                y[lo:hi] = x[lo:hi] @ s["w"][e].float().t()
        return y
    if op == "bwd":
        dx = torch.empty((s["rows"], s["k"]), dtype=torch.bfloat16, device=DEV)
        dw = torch.zeros(s["w"].shape, dtype=torch.float32 if s["dw"] == "fp32" else torch.bfloat16, device=DEV)
        for e, (lo, hi) in enumerate(zip(s["host"], s["host"][1:])):
            if hi > lo:
                dy = s["dy"][lo:hi].float()
                dx[lo:hi] = dy @ s["w"][e].float()
                dw[e] = dy.t() @ s["x"][lo:hi].float()
        return dx, dw
    if op == "gemv":
        x = s["x"].float()
        if s["swiglu"]:
            x = x[s["src_row"].long() // s["top_k"]]
        y = torch.empty((x.shape[0], s["n"] // 2 if s["swiglu"] else s["n"]), dtype=torch.bfloat16, device=DEV)
        for e, (lo, hi) in enumerate(zip(s["host"], s["host"][1:])):
            if hi > lo:
                v = x[lo:hi] @ weight_values(s, e).t()
                if s["swiglu"]:
                    gate, up = v.chunk(2, dim=1)
                    v = gate / (1.0 + torch.exp(-gate)) * up
                y[lo:hi] = v
        return y
    if op == "act":
        gate, up = s["gate_up"].float().chunk(2, dim=1)
        sig = 1.0 / (1.0 + torch.exp(-gate))
        h = (gate * sig * up).to(torch.bfloat16)
        if not s["grad"]:
            return h
        dh = s["dh"].float()
        d_gate = dh * up * sig * (1.0 + gate * (1.0 - sig))
        return h, torch.cat([d_gate, dh * gate * sig], dim=1).to(torch.bfloat16)
    return s["x"][s["src_row"].long() // s["top_k"]]


# ---------------------------------------------------------------------------------------- the definition, in 64 bits --
def segments(host):
    return [(e, lo, hi) for e, (lo, hi) in enumerate(zip(host, host[1:])) if hi > lo]


def exact_weight(s, e):
    """Expert e's weights from the bits of their codes: the magnitude's exponent and mantissa, times both scales."""
    n, k = s["n"], s["k"]
    packed = s["codes"][e * n:(e + 1) * n].short()
    v = torch.empty((n, k), dtype=torch.float64, device=DEV)
    for half in (0, 1):
        c = (packed >> (4 * half)) & 15
        ex, man = ((c >> 1) & 3).double(), (c & 1).double()
        mag = torch.where(ex > 0, torch.exp2(ex - 1) * (1 + 0.5 * man), 0.5 * man)
        v[:, half::2] = torch.where(c > 7, -mag, mag)
    tiles = s["sf"].reshape(-1, k // 64, 32, 4, 4)  # block of 128 rows, 4 groups, row % 32, row / 32, group
    sb = tiles.permute(0, 3, 2, 1, 4).reshape(-1, k // 16)[e * n:(e + 1) * n]
    v.view(n, k // 16, 16).mul_(sb.contiguous().view(torch.float8_e4m3fn).double()[:, :, None])
    return v.mul_(s["scale"][e * n:(e + 1) * n].double()[:, None])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("fwd", "gemv"):
        rows = case["tokens"] * case["top_k"]
        gathered = op == "fwd" or case["swiglu"]
        token = torch.div(s["src_row"].long(), case["top_k"], rounding_mode="floor") if gathered else None
        y = torch.empty((rows, case["n"]), dtype=torch.float64, device=DEV)
        for e, lo, hi in segments(s["host"]):
            x = (s["x"].index_select(0, token[lo:hi]) if gathered else s["x"][lo:hi]).double()
            w = s["w"][e].double() if op == "fwd" else exact_weight(s, e)
            y[lo:hi] = torch.mm(w, x.t()).t()
        if op == "gemv" and case["swiglu"]:
            inter = case["n"] // 2
            y = torch.sigmoid(y[:, :inter]) * y[:, :inter] * y[:, inter:]
        return y
    if op == "bwd":
        dx = torch.empty((case["rows"], case["k"]), dtype=torch.float64, device=DEV)
        dw = torch.zeros((case["experts"], case["n"], case["k"]), dtype=torch.float64, device=DEV)
        for e, lo, hi in segments(s["host"]):
            d = s["dy"][lo:hi].double()
            torch.mm(d, s["w"][e].double(), out=dx[lo:hi])
            torch.mm(d.t(), s["x"][lo:hi].double(), out=dw[e])
        return dx, dw
    if op == "act":
        inter = case["inter"]
        gu = s["gate_up"].double().requires_grad_(bool(case["grad"]))
        h = torch.sigmoid(gu[:, :inter]) * gu[:, :inter] * gu[:, inter:]
        if not case["grad"]:
            return h
        (d,) = torch.autograd.grad(h, gu, s["dh"].double())
        return h.detach(), d
    token = torch.div(s["src_row"].long(), case["top_k"], rounding_mode="floor")
    return s["x"].index_select(0, token).double()
