"""Products with NVFP4 weights in each number of warps that share a unit: the same bits, and near their 64-bit form.

The bound is that of tests/test_gpu_gemv_nvfp4.py: sums in fp32, (k + 10) 2^-23 of the terms' total size, one rounding to bf16
(2^-8), and the fast exponential and reciprocal of the activation (2^-14)."""
import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import block128 as ref
from tests import launch_rules, nvfp4w

pytestmark = pytest.mark.gpu
DEV = "cuda"
EXPERTS, N = 24, 2048
ROWS = [1, 2, 6, 2 * EXPERTS]  # of the first experts, two to each


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


def shares(k, swiglu, sms):
    """The numbers of warps that the calls of ROWS take."""
    return {launch_rules.gemv_share(swiglu, m, N, k, EXPERTS, sms) for m in ROWS}


def product64(x, w, offsets):
    """(result, size of its terms) of grouped rows and weights in 64 bits."""
    n = w.shape[0] // (len(offsets) - 1)
    want = torch.empty((x.shape[0], n), dtype=torch.float64, device=DEV)
    size = torch.empty_like(want)
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if hi > lo:
            a, b = x[lo:hi].double(), w[e * n:(e + 1) * n].t()
            want[lo:hi], size[lo:hi] = a @ b, a.abs() @ b.abs()
    return want, size


def near(y, x, w, offsets, swiglu):
    want, size = product64(x, w, offsets)
    d = (x.shape[1] + 10) * 2.0 ** -23 * size
    if not swiglu:
        return bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + d).all())
    gate, up = want.chunk(2, dim=1)
    d_gate, d_up = d.chunk(2, dim=1)
    silu = torch.sigmoid(gate) * gate
    # |silu'| <= 1.1
    allowed = 1.1 * d_gate * (up.abs() + d_up) + silu.abs() * d_up + (2.0 ** -8 + 2.0 ** -14) * (silu * up).abs()
    return bool(((y.double() - silu * up).abs() <= 1.01 * allowed + 1e-30).all())


@pytest.mark.parametrize("k", [512, 1536, 1856, 2368, 7168])
@pytest.mark.parametrize("swiglu", [False, True])
def test_every_number_of_warps(k, swiglu, status):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert len(shares(k, swiglu, sms)) >= 2
    call = fme.grouped_gemv_nvfp4_swiglu if swiglu else fme.grouped_gemv_nvfp4
    weights = fme.quantize_nvfp4_pertoken(ref.normal((EXPERTS * N, k), 0.05, 1), status=status)
    x = ref.normal((2 * EXPERTS, k), 1.0, 2)
    results = []
    for m in ROWS:
        off = [min(2 * e, m) for e in range(EXPERTS + 1)]
        results.append(call(x[:m].contiguous(), *weights, i32(off), status=status))
    whole = results[-1]
    for m, part in zip(ROWS, results):
        assert torch.equal(part, whole[:m])
    assert near(whole, x, nvfp4w.values(*weights), off, swiglu)


@pytest.mark.parametrize("tokens,top_k,experts,n,k,form", [(1, 8, 32, 4096, 7168, 4), (64, 4, 32, 1024, 1344, 2),
                                                           (3, 2, 8, 512, 2048, 8)])
def test_gathered_rows(tokens, top_k, experts, n, k, form, status):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert launch_rules.gemv_share(True, tokens * top_k, n, k, experts, sms) == form
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    ids = torch.rand((tokens, experts), generator=g, device=DEV).argsort(dim=1)[:, :top_k].int().contiguous()
    offsets, _, src = fme.moe_route(ids, experts, status=status)
    weights = fme.quantize_nvfp4_pertoken(ref.normal((experts * n, k), 0.05, 4), status=status)
    x = ref.normal((tokens, k), 1.0, 5)
    h = fme.grouped_gemv_nvfp4_swiglu(x, *weights, offsets, src_row=src, top_k=top_k, status=status)
    assert near(h, x[src.long() // top_k], nvfp4w.values(*weights), offsets.tolist(), True)


@pytest.mark.parametrize("experts,n,k", [(6, 1024, 1536), (40, 1024, 1536), (40, 1024, 2048), (12, 2048, 7168), (256, 512, 320),
                                         (1024, 256, 64)])
def test_experts_taken_together_with_activation(experts, n, k, status):
    """Units of several experts side by side, experts without rows and with more rows than fit between them."""
    g = torch.Generator(device=DEV)
    g.manual_seed(experts + k)
    few = torch.randint(0, 3, (experts,), generator=g, device=DEV)
    few[torch.randint(0, experts, (experts // 6 + 1,), generator=g, device=DEV)] = 9
    off = [0] + few.cumsum(0).tolist()
    weights = nvfp4w.random_weights(experts * n, k, 6, row_scale=2.0 ** -5)
    x = ref.normal((off[-1], k), 1.0, 7)
    h = fme.grouped_gemv_nvfp4_swiglu(x, *weights, i32(off), status=status)
    assert near(h, x, nvfp4w.values(*weights), off, True)


@pytest.mark.parametrize("small", [1.0, 2.0 ** -60])
def test_rows_with_infinities(small, status):
    """An infinity alone leaves a row exact in fp16; beside values that fp16 does not hold it takes the other decoding.  Either way
    its outputs are the infinities and NaN of the 64-bit product, and its neighbours' bits are as they were."""
    n, k = 512, 320
    weights = nvfp4w.random_weights(n, k, 8)
    x = ref.normal((8, k), 1.0, 9)
    clean = fme.grouped_gemv_nvfp4(x, *weights, i32([0, 8]), status=status)
    x[3] = small
    x[3, ::100] = float("inf")
    y = fme.grouped_gemv_nvfp4(x, *weights, i32([0, 8]), status=status)
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(y[keep], clean[keep])
    want = product64(x[3:4], nvfp4w.values(*weights), [0, 1])[0][0]
    assert torch.equal(y[3].isnan(), want.isnan()) and torch.equal(y[3].isposinf(), want.isposinf())
    assert torch.equal(y[3].isneginf(), want.isneginf()) and not bool(y[3].isfinite().any())
