"""NVFP4 expert weights in 64 bits, for the tests of the products that read them."""
import torch

from tests import block128 as ref

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def scale_index(rows, k, device):
    """Byte of the tiled layout for every (row, group of 16)."""
    r = torch.arange(rows, device=device)[:, None]
    c = torch.arange(k // 16, device=device)[None, :]
    return (r // 128 * (k // 64) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4


def values(codes, sf, scale):
    """The weights [rows, k] in float64."""
    rows, k = codes.shape[0], 2 * codes.shape[1]
    c = torch.stack([codes & 15, codes >> 4], dim=2).reshape(rows, k).long()
    v = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=torch.float64, device=codes.device)[c]
    s = ref.values(sf[scale_index(rows, k, codes.device)])
    return v * s.repeat_interleave(16, dim=1) * scale.double()[:, None]


def tiled(scales):
    """Scale bytes [rows, k / 16] -> the tiled buffer; bytes of rows behind the last are those of a NaN, as a buffer
    that was never written may hold them."""
    rows, groups = scales.shape
    out = torch.full(((rows + 127) // 128 * 128 * groups,), 0x7F, dtype=torch.uint8, device=scales.device)
    out[scale_index(rows, 16 * groups, scales.device)] = scales
    return out


def random_weights(rows, k, seed, scales=(0x30, 0x38, 0x40), row_scale=1.0):
    """Codes and scales drawn from all codes and the given scale bytes (0.5, 1 and 2), one row scale."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    codes = torch.randint(0, 256, (rows, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    pick = torch.tensor(scales, dtype=torch.uint8, device="cuda")
    s = pick[torch.randint(0, len(scales), (rows, k // 16), generator=g, device="cuda")]
    return codes, tiled(s), torch.full((rows,), row_scale, device="cuda")
