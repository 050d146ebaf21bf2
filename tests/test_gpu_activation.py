"""SwiGLU in bf16 with its gradient, and the grouping of bf16 rows."""
import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import block128 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    fme.ensure_built()


@pytest.fixture(autouse=True)
def _nothing_cached():
    torch.cuda.empty_cache()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def forward64(gu):
    g, u = gu.double().chunk(2, dim=1)
    return g * torch.sigmoid(g) * u


# Half a bf16 step, and a few 2^-17 of the fast exponential and reciprocal (2^-14); results below the smallest normal
# fp32 may be flushed.
HALF, FAST, TINY = 2.0 ** -8, 2.0 ** -14, 2.0 ** -125


@pytest.mark.parametrize("rows,inter", [(1, 8), (3, 40), (64, 2048), (129, 1000), (1000, 264), (5, 65536)])
def test_swiglu_and_its_gradient(rows, inter):
    gu = (4.0 * ref.normal((rows, 2 * inter), 1.0, 1).float()).to(torch.bfloat16)
    gu[:, ::5] *= 8.0
    dh = ref.normal((rows, inter), 0.1, 2)
    want = forward64(gu)
    h = fme.swiglu(gu)
    assert bool(((h.double() - want).abs() <= (HALF + FAST) * want.abs() + TINY).all())

    d = fme.swiglu_backward(gu, dh).double()
    g, u = gu.double().chunk(2, dim=1)
    sig, neg = torch.sigmoid(g), torch.sigmoid(-g)
    d_gate, d_up = dh.double() * u * sig * (1 + g * neg), dh.double() * g * sig
    size = torch.cat([(dh.double() * u * sig).abs() * (1 + g.abs() * neg), d_up.abs()], dim=1)
    formula = torch.cat([d_gate, d_up], dim=1)
    assert bool(((d - formula).abs() <= HALF * formula.abs() + FAST * size + TINY).all())

    # against differences of the forward in 64 bits: the step's own error is far below the bound's
    eps = 1e-4
    for col in range(0, 2 * inter, max(1, inter // 7)):
        plus, minus = gu.double(), gu.double()
        plus[:, col] += eps
        minus[:, col] -= eps
        at = col % inter
        diff = ((forward64(plus) - forward64(minus))[:, at] / (2 * eps)) * dh[:, at].double()
        near = HALF * diff.abs() + FAST * size[:, col] + 1e-6 * (1 + u[:, at].abs()) * dh[:, at].double().abs()
        assert bool(((d[:, col] - diff).abs() <= near).all())


def test_the_bits_of_the_fused_forms():
    rows, inter = 300, 256
    gu, dh = ref.normal((rows, 2 * inter), 3.0, 3), ref.normal((rows, inter), 0.1, 4)
    assert torch.equal(fme.swiglu(gu), fme.swiglu_quantize_nvfp4(gu)[3])
    assert torch.equal(fme.swiglu_backward(gu, dh), fme.swiglu_backward_quantize_mxfp8(gu, dh, want_d=True)[-1])


def test_far_gates():
    """Gates so far from zero that the exponential under- or overflows: h is u g or 0, never NaN."""
    far = torch.tensor([-3e38, -1e4, -200.0, -100.0, -0.0, 0.0, 100.0, 200.0, 1e4, 3e38], device=DEV).to(torch.bfloat16)
    gu = torch.cat([far.repeat(4)[None, :], torch.full((1, 40), 0.5, device=DEV).to(torch.bfloat16)], dim=1)
    h = fme.swiglu(gu).double()
    want = forward64(gu)
    assert bool(h.isfinite().all()) and bool(((h - want).abs() <= (HALF + FAST) * want.abs() + TINY).all())
    d = fme.swiglu_backward(gu, torch.ones((1, 40), dtype=torch.bfloat16, device=DEV)).double()
    assert bool(d.isfinite().all())
    assert torch.equal(d[0, 6:10], torch.full((4,), 0.5, dtype=torch.float64, device=DEV))
    assert bool((d[0, :4].abs() <= 1e-36).all())


def test_no_rows():
    gu = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    assert fme.swiglu(gu).shape == (0, 32)
    assert fme.swiglu_backward(gu, torch.empty((0, 32), dtype=torch.bfloat16, device=DEV)).shape == (0, 64)
    assert fme.moe_permute(gu, i32([]), 2).shape == (0, 64)


@pytest.mark.parametrize("tokens,top_k,n", [(1, 1, 8), (1, 8, 7168), (33, 3, 1000), (500, 2, 2056), (777, 1, 64),
                                            (40, 64, 24), (3, 2, 65536)])
def test_permute(tokens, top_k, n):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    x = ref.normal((tokens, n), 1.0, 1)
    x[0, 0] = float("nan")
    src = torch.randperm(tokens * top_k, device=DEV).int()
    whole = torch.full((tokens * top_k * n + 2048,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = whole[1024:-1024].view(tokens * top_k, n)
    assert fme.moe_permute(x, src, top_k, out=out, status=st) is out
    assert torch.equal(out.view(torch.int16), x[src.long() // top_k].view(torch.int16))
    assert bool((whole[:1024] == 7.0).all()) and bool((whole[-1024:] == 7.0).all())
    assert fme.read_device_status(st)[0] == 0


def test_permute_out_of_range_reads_row_0_and_is_reported():
    x = ref.normal((4, 136), 1.0, 1)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = fme.moe_permute(x, i32([0, -1, 8, 3, 7, 1, 2, 1 << 30]), 2, status=st)
    assert fme.read_device_status(st)[0] == fme.ERR_DEVICE_BAD_INDEX
    assert torch.equal(out, x[[0, 0, 0, 1, 3, 0, 1, 0]])


def test_permutes_gradient_is_the_combine_with_ones():
    tokens, top_k, n, experts = 50, 3, 72, 6
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    ids = torch.rand((tokens, experts), generator=g, device=DEV).argsort(dim=1)[:, :top_k].int().contiguous()
    _, row_of, src = fme.moe_route(ids, experts)
    d = ref.normal((tokens * top_k, n), 1.0, 2)
    got = fme.moe_combine(d, row_of, torch.ones((tokens, top_k), device=DEV)).double()
    want = torch.zeros((tokens, n), dtype=torch.float64, device=DEV).index_add_(0, src.long() // top_k, d.double())
    size = torch.zeros_like(want).index_add_(0, src.long() // top_k, d.double().abs())
    assert bool(((got - want).abs() <= HALF * want.abs() + 3 * 2.0 ** -23 * size).all())
