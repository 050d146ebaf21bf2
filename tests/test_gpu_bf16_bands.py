"""The order of the weight gradient's tiles where an expert's operands exceed L2, against 64 bits."""
import pytest
import torch

import fp8_moe_expert_gb300 as fme

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    fme.ensure_built()


@pytest.fixture
def status():
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    yield st
    assert fme.read_device_status(st)[0] == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def integers(shape, seed, low=-2, high=3):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(low, high, shape, generator=g, device=DEV).to(torch.bfloat16)


def wgrad64(dy, x, off):
    dw = torch.zeros((len(off) - 1, dy.shape[1], x.shape[1]), dtype=torch.float64, device=DEV)
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        for at in range(lo, hi, 1 << 22):
            to = min(hi, at + (1 << 22))
            dw[e] += dy[at:to].double().t() @ x[at:to].double()
    return dw


# tile rows: a band of 8 and one of 2; two bands of 8; one band, which is lower, of 10 columns
@pytest.mark.parametrize("n,k", [(2312, 520), (4096, 264), (264, 2312)])
@pytest.mark.parametrize("mode", ["bf16", "fp32", "added"])
def test_experts_whose_tiles_go_band_by_band(n, k, mode, status):
    """14000 rows of n + k columns are more than 64 MB; the experts beside them go row by row.  Every sum is exact."""
    off = [0, 500, 14500, 14500, 14600]
    dy, x = integers((off[-1], n), 5), integers((off[-1], k), 6)
    assert 14000 * (n + k) > 1 << 25
    want = wgrad64(dy, x, off)
    dtype = torch.bfloat16 if mode == "bf16" else torch.float32
    dw = torch.full((4, n, k), float("nan"), dtype=dtype, device=DEV)
    if mode == "added":
        dw = integers((4, n, k), 7).float()
        want += dw
    fme.grouped_gemm_wgrad_bf16(dy, x, i32(off), dw=dw, accumulate=mode == "added", status=status)
    assert torch.equal(dw, want.to(dtype))
