"""The weight gradient of many rows of an expert: sums that are cut every 65536 rows (bf16) or 1024 (fp32), against
64 bits."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sums_of_one_sign_over_millions_of_rows(dtype, status):
    """Each step of the tensor cores cuts a sum towards zero, by a step of the running sum at most for each of its 16 products
    and the sum: over 65536 rows by 17 / 16 x 65536 x 2^-23 = 0.83% of it at most, over 1024 by 0.013%.  The sums are then added
    rounded to nearest, 2^-24 of the running sum each: 512 of them 0.003%, 32768 of them 0.2%.  In a single sum the cuts
    of 2^25 rows, of half a step each on the average, are 4%."""
    rows, n, k = 1 << 25, 8, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    dy, x = ((1.0 + torch.rand((rows, c), generator=g, device=DEV)).to(torch.bfloat16) for c in (n, k))
    dw = fme.grouped_gemm_wgrad_bf16(dy, x, i32([0, rows]), dtype=dtype, status=status)
    want = wgrad64(dy, x, [0, rows])
    of_a_sum = 65536 if dtype == torch.bfloat16 else 1024
    allowed = 17 / 16 * of_a_sum * 2.0 ** -23 + rows // of_a_sum * 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24)
    assert float(((dw.double() - want) / want).abs().max()) <= allowed


@pytest.mark.parametrize("last", [1, 63, 65536, 70001])
def test_bf16_sums_cut_at_65536_rows(last, status):
    """Experts just below, at and past a sum's rows, and of several, beside short ones; every sum is exact."""
    off = [0, 40, 65576, 131113, 131113, 262500]
    off.append(off[-1] + last)
    n, k = 264, 136
    dy, x = integers((off[-1], n), 1), integers((off[-1], k), 2)
    dw = torch.full((len(off) - 1, n, k), float("nan"), dtype=torch.bfloat16, device=DEV)
    assert fme.grouped_gemm_wgrad_bf16(dy, x, i32(off), dw=dw, status=status) is dw
    assert torch.equal(dw, wgrad64(dy, x, off).to(torch.bfloat16))


def test_bf16_sums_of_65536_rows_are_added_in_order_in_fp32(status):
    """Sums of 65536 products up to 225 are exact in fp32; those of several are not, and are rounded as they are added."""
    off, n, k = [0, 1000000, 1000300], 40, 72
    dy, x = integers((off[-1], n), 3, 0, 16), integers((off[-1], k), 4, 0, 16)
    want = torch.zeros((2, n, k), device=DEV)
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        for at in range(lo, hi, 65536):
            to = min(at + 65536, hi)
            want[e] += (dy[at:to].double().t() @ x[at:to].double()).float()
    got = fme.grouped_gemm_wgrad_bf16(dy, x, i32(off), status=status)
    assert torch.equal(got, want.to(torch.bfloat16))
