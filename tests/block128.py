"""Plain 64-bit forms of the FP8 block-128 format and products, for the tests."""
import numpy as np
import torch

FLOOR = 2.0 ** -100


def e4m3_round(v):
    """Nearest E4M3 value of float64 v (ties to the even code), saturating at 448."""
    _, ex = torch.frexp(v)
    step = (((ex - 1).clamp_min(-6).long() - 3 + 1023) << 52).view(torch.float64)  # exact powers of two
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def values(codes):
    """E4M3 codes (u8) -> float64."""
    return codes.view(torch.float8_e4m3fn).float().double()


def scales(amax):
    """(scale, r) of the blocks' largest magnitudes: fp32 IEEE divisions, by numpy."""
    a = np.maximum(amax.float().cpu().numpy(), np.float32(FLOOR))
    s, r = a / np.float32(448.0), np.float32(448.0) / a
    return torch.from_numpy(s).to(amax.device), torch.from_numpy(r).to(amax.device)


def _code_values(x, r):
    """Values of E4M3(fl32(x r)): the fp32 product of bf16 x and fp32 r, then exact rounding."""
    return e4m3_round((x.float() * r).double())


def quantize_rows(x):
    rows, cols = x.shape
    cb = -(-cols // 128)
    full = torch.zeros((rows, cb * 128), dtype=torch.bfloat16, device=x.device)
    full[:, :cols] = x
    b = full.view(rows, cb, 128)
    s, r = scales(b.float().abs().amax(dim=2))
    return _code_values(b, r[:, :, None]).view(rows, -1)[:, :cols], s.t()


def padded(offsets):
    """Padded start of every group (and the end) for host row offsets."""
    p = [0]
    for lo, hi in zip(offsets, offsets[1:]):
        p.append(p[-1] + -(-(hi - lo) // 128) * 128)
    return p


def quantize_cols(x, offsets):
    """Values [ld, cols] and scales [ld/128, cols] over padded positions."""
    rows, cols = x.shape
    g = len(offsets) - 1
    ld = (rows + 127 * g) // 128 * 128
    v = torch.zeros((ld, cols), dtype=torch.bfloat16, device=x.device)
    for p, lo, hi in zip(padded(offsets), offsets, offsets[1:]):
        v[p:p + hi - lo] = x[lo:hi]
    b = v.view(ld // 128, 128, cols)
    s, r = scales(b.float().abs().amax(dim=1)) if ld else (torch.zeros((0, cols), device=x.device),) * 2
    return _code_values(b, r[:, None, :]).view(ld, cols), s


def quantize_weights(w):
    e, n, k = w.shape
    nb, kb = -(-n // 128), -(-k // 128)
    full = torch.zeros((e, nb * 128, kb * 128), dtype=torch.bfloat16, device=w.device)
    full[:, :n, :k] = w
    b = full.view(e, nb, 128, kb, 128)
    s, r = scales(b.float().abs().amax(dim=(2, 4)))
    return _code_values(b, r[:, :, None, :, None]).reshape(e, nb * 128, kb * 128)[:, :n, :k], s


def row_operand(codes, scale):
    return values(codes) * scale.double().t().repeat_interleave(128, dim=1)[:, :codes.shape[1]]


def weight_operand(codes, scale):
    s = scale.double().repeat_interleave(128, dim=-2).repeat_interleave(128, dim=-1)
    return values(codes) * s[..., :codes.shape[-2], :codes.shape[-1]]


def col_operand(codes, scale):
    return values(codes) * scale.double().repeat_interleave(128, dim=0)


def bound(ref, size, contraction, half_ulp):
    """Largest |y - ref| allowed: one rounding of the output, and fp32 sums.  Within a block of
    128 at most 128 additions each lose 2^-23 of the terms' total size `size` (sum of |a||b|,
    whether they round or truncate); each of the outer sums and the two scale products lose
    2^-23 of it at most once a block."""
    blocks = -(-contraction // 128)
    return half_ulp * ref.abs() + (128 + blocks + 3) * 2.0 ** -23 * size


def split(rows, groups, seed, empty=True):
    """Host offsets of `rows` rows in `groups` groups of uneven sizes, some empty."""
    rng = np.random.default_rng(seed)
    p = rng.dirichlet(np.full(groups, 0.5))
    if empty and groups > 2:
        p[rng.integers(groups)] = 0.0
        p /= p.sum()
    return np.concatenate([[0], np.cumsum(rng.multinomial(rows, p))]).tolist()


def normal(shape, std, seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return torch.empty(shape, dtype=torch.float32, device=device).normal_(0.0, std, generator=g).to(torch.bfloat16)
