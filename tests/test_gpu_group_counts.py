"""The tables that the kernels make of the experts' offsets, at the counts of experts where their reading changes (32 at a
time, 128 in flight): padded offsets, products and malformed offsets."""
import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import block128 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
COUNTS = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 160, 161, 256, 257, 1023, 1024]


@pytest.fixture(scope="module", autouse=True)
def _built():
    fme.ensure_built()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def integers(shape, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device=DEV).to(torch.bfloat16)


def status_of(call):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = call(st)
    return fme.read_device_status(st)[0], out


@pytest.mark.parametrize("experts", COUNTS)
def test_offsets_of_any_number_of_experts(experts):
    rows, n, k = 40 + 5 * experts, 72, 64
    off = ref.split(rows, experts, experts)
    x, w = integers((rows, k), 1), integers((experts, n, k), 2)
    expert = torch.repeat_interleave(torch.arange(experts), torch.tensor(off).diff()).to(DEV)
    want = torch.einsum("rk,rnk->rn", x.double(), w[expert].double()).to(torch.bfloat16)
    code, y = status_of(lambda st: fme.grouped_gemm_fwd_bf16(x, w, i32(off), status=st))
    assert code == 0 and torch.equal(y, want)
    code, (_, _, padded) = status_of(lambda st: fme.quantize_fp8_block128(x, fme.COLWISE, i32(off), experts, status=st))
    sizes = (torch.tensor(off).diff() + 127) // 128 * 128
    assert code == 0 and padded.tolist() == [0] + sizes.cumsum(0).tolist()


@pytest.mark.parametrize("experts", [c for c in COUNTS if c > 1])
def test_a_malformed_offset_anywhere_is_reported(experts):
    rows, n, k = 40 + 5 * experts, 72, 64
    off = ref.split(rows, experts, experts)
    x, w = integers((rows, k), 1), integers((experts, n, k), 2)
    for at in {0, 1, experts // 2, experts - 1, experts, min(32, experts), min(33, experts), min(128, experts), min(129, experts)}:
        for bad in (-1, rows + 1):
            o = list(off)
            o[at] = bad
            code, _ = status_of(lambda st: fme.grouped_gemm_fwd_bf16(x, w, i32(o), status=st))
            assert code == fme.ERR_DEVICE_BAD_OFFSETS, at
            code, _ = status_of(lambda st: fme.quantize_fp8_block128(x, fme.COLWISE, i32(o), experts, status=st))
            assert code == fme.ERR_DEVICE_BAD_OFFSETS, at
