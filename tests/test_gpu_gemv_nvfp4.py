"""Products of few bf16 rows with NVFP4 weights against their 64-bit form.

c sf is exact, the sums are in fp32: with s = sum |x| |w| each of at most k additions and the 8 of the partial sums loses
2^-23 of s, the row scale's product 2^-24, and the output is rounded once (bf16, half a step 2^-8).  On small
integers and scales that are powers of two every sum is exact."""
import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import block128 as ref
from tests import nvfp4w

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    fme.ensure_built()


@pytest.fixture(autouse=True)
def _nothing_cached():
    torch.cuda.empty_cache()


@pytest.fixture
def status():
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    yield st
    assert fme.read_device_status(st)[0] == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def integers(shape, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device=DEV).to(torch.bfloat16)


def product64(x, w, off, n):
    """(y, size) for grouped rows x and weights w [E n, k] in 64 bits."""
    y = torch.zeros((x.shape[0], n), dtype=torch.float64, device=DEV)
    size = torch.zeros_like(y)
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        a, b = x[lo:hi].double(), w[e * n:(e + 1) * n].t()
        y[lo:hi], size[lo:hi] = a @ b, a.abs() @ b.abs()
    return y, size


def sum_error(size, k):
    return (k + 8 + 2) * 2.0 ** -23 * size


# rows, experts, n, k: rows of the weights that fill no group of 128, experts that start inside one, a last chunk of 64
SHAPES = [(1, 1, 1, 64), (1, 1, 128, 64), (1, 4, 256, 128), (3, 2, 130, 192), (8, 1, 100, 320), (9, 1, 7, 1024), (17, 3, 200, 1344),
          (8, 8, 384, 7168), (40, 3, 1000, 512), (70, 2, 128, 8192), (130, 5, 264, 2048), (33, 200, 40, 192),
          (2000, 1024, 8, 64)]


@pytest.mark.parametrize("rows,experts,n,k", SHAPES)
def test_product(rows, experts, n, k, status):
    off = ref.split(rows, experts, rows + n)
    w = ref.normal((experts * n, k), 0.05, 1)
    w[::7] *= 1e-3
    w[:, : k // 4] *= 30.0
    codes, sf, scale = fme.quantize_nvfp4_pertoken(w, status=status)
    x = ref.normal((rows, k), 1.0, 2)
    y = fme.grouped_gemv_nvfp4(x, codes, sf, scale, i32(off), status=status)
    want, size = product64(x, nvfp4w.values(codes, sf, scale), off, n)
    assert bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + sum_error(size, k)).all())


@pytest.mark.parametrize("rows,experts,n,k", SHAPES)
def test_exact_sums(rows, experts, n, k, status):
    off = ref.split(rows, experts, rows + n)
    codes, sf, scale = nvfp4w.random_weights(experts * n, k, 3)
    x = integers((rows, k), 4)
    y = fme.grouped_gemv_nvfp4(x, codes, sf, scale, i32(off), status=status)
    want, _ = product64(x, nvfp4w.values(codes, sf, scale), off, n)
    assert torch.equal(y, want.to(torch.bfloat16))


def test_every_code_and_scale(status):
    """One-hot rows pick single weights: every code under every finite scale, subnormal ones among them."""
    k = 64
    scales = torch.arange(0, 0x7F, dtype=torch.uint8, device=DEV)[:, None].expand(-1, k // 16).contiguous()
    n = scales.shape[0]
    one = torch.arange(16, dtype=torch.uint8, device=DEV)
    codes = (one[0::2] + 16 * one[1::2]).repeat(4)[None, :].expand(n, -1).contiguous()  # k -> code k % 16
    sf, scale = nvfp4w.tiled(scales), torch.full((n,), 0.5, device=DEV)
    x = torch.eye(k, device=DEV).to(torch.bfloat16)
    y = fme.grouped_gemv_nvfp4(x, codes, sf, scale, i32([0, k]), status=status)
    assert torch.equal(y.double(), nvfp4w.values(codes, sf, scale).t())


@pytest.mark.parametrize("big", [2.0 ** 100, 2.0 ** -100])
def test_large_and_small_rows(big, status):
    n, k = 200, 256
    codes, sf, scale = nvfp4w.random_weights(n, k, 5)
    x = (integers((3, k), 6).float() * big).to(torch.bfloat16)
    y = fme.grouped_gemv_nvfp4(x, codes, sf, scale, i32([0, 3]), status=status)
    want, _ = product64(x, nvfp4w.values(codes, sf, scale), [0, 3], n)
    assert torch.equal(y.double(), want.to(torch.bfloat16).double())


@pytest.mark.parametrize("tokens,top_k,experts,n,k", [(1, 8, 32, 256, 7168), (5, 2, 4, 512, 192), (16, 4, 4, 256, 1024),
                                                      (40, 3, 5, 256, 320), (1, 1, 1, 256, 64)])
def test_gathered_with_activation(tokens, top_k, experts, n, k, status):
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    ids = torch.rand((tokens, experts), generator=g, device=DEV).argsort(dim=1)[:, :top_k].int().contiguous()
    offsets, _, src = fme.moe_route(ids, experts, status=status)
    w = ref.normal((experts * n, k), 0.05, 8)
    codes, sf, scale = fme.quantize_nvfp4_pertoken(w, status=status)
    x = ref.normal((tokens, k), 1.0, 9)
    h = fme.grouped_gemv_nvfp4_swiglu(x, codes, sf, scale, offsets, src_row=src, top_k=top_k, status=status)
    y = fme.grouped_gemv_nvfp4(x, codes, sf, scale, offsets, src_row=src, top_k=top_k, status=status)
    rows = x[src.long() // top_k]
    assert torch.equal(y, fme.grouped_gemv_nvfp4(rows, codes, sf, scale, offsets, status=status))
    want, size = product64(rows, nvfp4w.values(codes, sf, scale), offsets.tolist(), n)
    gate, up = want.chunk(2, dim=1)
    d_gate, d_up = sum_error(size, k).chunk(2, dim=1)
    silu = torch.sigmoid(gate) * gate
    # |silu'| <= 1.1; the fast exponential and reciprocal a few 2^-17
    allowed = 1.1 * d_gate * (up.abs() + d_up) + silu.abs() * d_up + (2.0 ** -8 + 2.0 ** -14) * (silu * up).abs()
    err = (h.double() - silu * up).abs()
    assert bool((err <= 1.01 * allowed + 1e-30).all()), float((err - allowed).max())


@pytest.mark.parametrize("experts,n,k", [(6, 1000, 1536), (40, 1000, 1536), (40, 1000, 2048), (12, 2048, 7168), (256, 512, 320),
                                         (1024, 256, 64)])
def test_experts_taken_together(experts, n, k, status):
    """Units of several experts side by side, experts without rows and with more rows than fit between them, and every other
    expert's rows NaN, infinite or of a range that only the other decoding takes."""
    g = torch.Generator(device=DEV)
    g.manual_seed(experts + k)
    few = torch.randint(0, 3, (experts,), generator=g, device=DEV)
    few[torch.randint(0, experts, (experts // 6 + 1,), generator=g, device=DEV)] = 9
    off = [0] + few.cumsum(0).tolist()
    codes, sf, scale = nvfp4w.random_weights(experts * n, k, 11)
    x = integers((off[-1], k), 12)
    y = fme.grouped_gemv_nvfp4(x, codes, sf, scale, i32(off), status=status)
    want, _ = product64(x, nvfp4w.values(codes, sf, scale), off, n)
    assert torch.equal(y, want.to(torch.bfloat16))
    rows = torch.repeat_interleave(torch.arange(experts, device=DEV), few) % 2 == 1
    for bad in (float("nan"), float("inf"), 2.0 ** -60):
        other = x.clone()
        other[rows, ::5] = bad
        got = fme.grouped_gemv_nvfp4(other, codes, sf, scale, i32(off), status=status)
        assert torch.equal(got[~rows], y[~rows])
        if n % 256 == 0:
            clean = fme.grouped_gemv_nvfp4_swiglu(x, codes, sf, scale, i32(off), status=status)
            got = fme.grouped_gemv_nvfp4_swiglu(other, codes, sf, scale, i32(off), status=status)
            assert torch.equal(got[~rows], clean[~rows])


def test_a_rows_bits_do_not_depend_on_the_batch(status):
    """Alone, and among more rows of an expert than are taken at a time."""
    n, k = 512, 1344
    codes, sf, scale = fme.quantize_nvfp4_pertoken(ref.normal((2 * n, k), 0.05, 1))
    x = ref.normal((100, k), 1.0, 2)
    for call in (fme.grouped_gemv_nvfp4, fme.grouped_gemv_nvfp4_swiglu):
        whole = call(x, codes, sf, scale, i32([0, 37, 100]), status=status)
        for lo, hi in ((0, 1), (3, 9), (5, 20), (0, 30)):
            part = call(x[lo:hi].contiguous(), codes, sf, scale, i32([0, hi - lo, hi - lo]), status=status)
            assert torch.equal(part, whole[lo:hi])


def within(y, want, size, k):
    """Where no partial sum can leave fp32's range: one of terms of total size 2^127 and more (2^127 x 2 is an infinity
    already) may overflow on the way to a sum that would not."""
    fits = size < 2.0 ** 127
    return bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + sum_error(size, k))[fits].all())


def test_rows_of_any_range(status):
    """A row with values far apart is not exact in fp16: it takes its neighbours the other way, with their bits as they
    were; and nothing of it is lost, weights of 0 at its large values among them."""
    n, k = 256, 320
    codes, sf, scale = nvfp4w.random_weights(n, k, 5)
    x = integers((8, k), 6)
    near = fme.grouped_gemv_nvfp4(x, codes, sf, scale, i32([0, 8]), status=status)
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    for far in (2.0 ** 15, 2.0 ** 28, 2.0 ** 30, 2.0 ** 40, 2.0 ** 100, 2.0 ** 127):
        y = x.clone()
        y[3] = torch.where(torch.rand(k, generator=g, device=DEV) < 0.1, far, 2.0 ** -20).to(torch.bfloat16) * y[3]
        got = fme.grouped_gemv_nvfp4(y, codes, sf, scale, i32([0, 8]), status=status)
        keep = [0, 1, 2, 4, 5, 6, 7]
        assert torch.equal(got[keep], near[keep])
        want, size = product64(y, nvfp4w.values(codes, sf, scale), [0, 8], n)
        assert within(got, want, size, k)
        # one large value at a weight of 0 for every output, the rest small
        c0 = codes.clone()
        c0[:, 0] &= 0xF0
        y[3] = 2.0 ** -20
        y[3, 0] = far
        got = fme.grouped_gemv_nvfp4(y, c0, sf, scale, i32([0, 8]), status=status)
        want, size = product64(y, nvfp4w.values(c0, sf, scale), [0, 8], n)
        assert within(got, want, size, k)


def test_the_bits_with_two_four_and_eight_warps(status):
    """One row alone and the same row among the rows of more and more experts, so that fewer warps share its sums."""
    n, k = 2048, 1856
    experts = 24
    codes, sf, scale = fme.quantize_nvfp4_pertoken(ref.normal((experts * n, k), 0.05, 1))
    x = ref.normal((2 * experts, k), 1.0, 2)
    whole = fme.grouped_gemv_nvfp4(x, codes, sf, scale, i32([2 * e for e in range(experts + 1)]), status=status)
    for e in (1, 2, 6, 13):
        part = fme.grouped_gemv_nvfp4(x[:2 * e].contiguous(), codes, sf, scale,
                                      i32([2 * min(i, e) for i in range(experts + 1)]), status=status)
        assert torch.equal(part, whole[:2 * e])
    one = fme.grouped_gemv_nvfp4(x[:1].contiguous(), codes, sf, scale, i32([0] + [1] * experts), status=status)
    assert torch.equal(one, whole[:1])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_rows_values_stay_its_own(bad, status):
    n, k = 256, 192
    codes, sf, scale = fme.quantize_nvfp4_pertoken(ref.normal((3 * n, k), 0.05, 1))
    x = ref.normal((11, k), 1.0, 2)
    off = i32([0, 4, 4, 11])
    clean = fme.grouped_gemv_nvfp4(x, codes, sf, scale, off, status=status)
    x[6, k - 1] = bad
    y = fme.grouped_gemv_nvfp4(x, codes, sf, scale, off, status=status)
    keep = [i for i in range(11) if i != 6]
    assert torch.equal(y[keep], clean[keep]) and not bool(y[6].isfinite().all())


def test_no_rows_and_malformed_offsets():
    n, k = 128, 64
    codes, sf, scale = nvfp4w.random_weights(2 * n, k, 1)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    empty = torch.empty((0, k), dtype=torch.bfloat16, device=DEV)
    assert fme.grouped_gemv_nvfp4(empty, codes, sf, scale, i32([0, 0, 0]), status=st).shape == (0, n)
    assert fme.read_device_status(st)[0] == 0
    x = integers((5, k), 2)
    for off in ([0, 6, 5], [1, 2, 5], [0, 2, 4], [0, -1, 5]):
        st.zero_()
        y = torch.full((5, n), 7.0, dtype=torch.bfloat16, device=DEV)
        fme.grouped_gemv_nvfp4(x, codes, sf, scale, i32(off), y=y, status=st)
        assert fme.read_device_status(st)[0] == fme.ERR_DEVICE_BAD_OFFSETS and bool((y == 7.0).all())


def test_gather_out_of_range_reads_row_0_and_is_reported():
    n, k = 128, 64
    codes, sf, scale = nvfp4w.random_weights(n, k, 1)
    x = integers((3, k), 2)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = fme.grouped_gemv_nvfp4(x, codes, sf, scale, i32([0, 6]), src_row=i32([0, -1, 6, 5, 2, 1 << 30]), top_k=2, status=st)
    assert fme.read_device_status(st)[0] == fme.ERR_DEVICE_BAD_INDEX
    assert torch.equal(y, fme.grouped_gemv_nvfp4(x[[0, 0, 0, 2, 1, 0]], codes, sf, scale, i32([0, 6])))


def test_nothing_outside_the_output_is_written(status):
    rows, n, k = 13, 200, 128
    codes, sf, scale = nvfp4w.random_weights(2 * n, k, 1)
    whole = torch.full((rows * n + 2048,), 7.0, dtype=torch.bfloat16, device=DEV)
    fme.grouped_gemv_nvfp4(integers((rows, k), 2), codes, sf, scale, i32([0, 5, rows]),
                           y=whole[1024:1024 + rows * n].view(rows, n), status=status)
    assert bool((whole[:1024] == 7.0).all()) and bool((whole[-1024:] == 7.0).all())
