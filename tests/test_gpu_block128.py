"""FP8 block-128 quantizers and grouped GEMMs against their 64-bit forms (tests/block128.py).

Codes and scales are compared bit for bit; the products within block128.bound."""
import numpy as np
import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import block128 as ref

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


def outliers(shape, seed):
    x = ref.normal(shape, 1.0, seed).float()
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 1)
    x *= torch.pow(2.0, torch.randint(-20, 21, (shape[0], 1), generator=g, device=DEV).float())
    x[torch.rand(shape, generator=g, device=DEV) < 0.01] *= 100.0
    x[torch.rand(shape, generator=g, device=DEV) < 0.05] = 0.0
    return x.to(torch.bfloat16)


def special(rows, cols):
    """Zero blocks, signed zeros, the smallest and largest bf16, amax at and below the floor."""
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    vals = [0.0, -0.0, 9.2e-41, -9.2e-41, 3.38e38, -3.38e38, 2.0 ** -100, 2.0 ** -101, -1.0, 448.0]
    for i in range(rows):
        x[i, i % cols] = vals[i % len(vals)]
        x[i, (7 * i + 3) % cols] = -0.5 * vals[i % len(vals)]
    return x


def same(codes, want):
    assert torch.equal(ref.values(codes), want)


ROW_SHAPES = [(1, 16), (1, 128), (3, 144), (8, 512), (9, 528), (130, 1040), (37, 7168), (1000, 2048)]


@pytest.mark.parametrize("rows,cols", ROW_SHAPES)
@pytest.mark.parametrize("make", ["outliers", "special"])
def test_rows(rows, cols, make, status):
    x = outliers((rows, cols), rows + cols) if make == "outliers" else special(rows, cols)
    codes, scale = fme.quantize_fp8_block128(x, status=status)
    v, s = ref.quantize_rows(x)
    assert torch.equal(scale, s)
    same(codes, v)


def test_every_magnitude(status):
    """A row for each positive finite bf16 value as its block's magnitude, the rest random fractions of it."""
    bits = torch.arange(1, 255 << 7, device=DEV, dtype=torch.int32)
    top = (bits << 16).view(torch.float32)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = (top[:, None] * (2 * torch.rand((len(top), 128), generator=g, device=DEV) - 1)).to(torch.bfloat16)
    x[:, 77] = top.to(torch.bfloat16)
    codes, scale = fme.quantize_fp8_block128(x, status=status)
    v, s = ref.quantize_rows(x)
    assert torch.equal(scale, s)
    same(codes, v)


@pytest.mark.parametrize("tokens,top_k,cols", [(1, 8, 7168), (33, 3, 272), (500, 1, 128)])
def test_gathered_rows_equal_the_quantized_copy(tokens, top_k, cols, status):
    x = outliers((tokens, cols), 5)
    src = torch.randperm(tokens * top_k, device=DEV).int()
    codes, scale = fme.quantize_fp8_block128(x, src_row=src, top_k=top_k, status=status)
    c2, s2 = fme.quantize_fp8_block128(x[src.long() // top_k].contiguous(), status=status)
    assert torch.equal(codes, c2) and torch.equal(scale, s2)


def test_gather_out_of_range_reads_row_0_and_is_reported():
    x = outliers((4, 256), 6)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    codes, scale = fme.quantize_fp8_block128(x, src_row=i32([0, -1, 8, 3, 7, 1, 2, 5]), top_k=2, status=st)
    assert fme.read_device_status(st)[0] == fme.ERR_DEVICE_BAD_INDEX
    c2, s2 = fme.quantize_fp8_block128(x[[0, 0, 0, 1, 3, 0, 1, 2]].contiguous())
    assert torch.equal(codes, c2) and torch.equal(scale, s2)


COL_CASES = [(0, 128, 1), (0, 48, 5), (1, 16, 1), (127, 144, 1), (128, 256, 2), (129, 272, 3), (1000, 528, 8),
             (777, 1040, 40), (3000, 2048, 5)]


@pytest.mark.parametrize("rows,cols,groups", COL_CASES)
def test_cols_and_rowcol(rows, cols, groups, status):
    x = outliers((rows, cols), rows + groups) if rows else torch.empty((0, cols), dtype=torch.bfloat16, device=DEV)
    off = ref.split(rows, groups, rows + groups)
    codes, scale, po = fme.quantize_fp8_block128(x, fme.COLWISE, i32(off), status=status)
    v, s = ref.quantize_cols(x, off)
    assert po.tolist() == ref.padded(off)
    assert torch.equal(scale, s)
    same(codes, v)
    (rc, rs), (cc, cs, po2) = fme.quantize_fp8_block128_rowcol(x, i32(off), status=status)
    assert torch.equal(cc, codes) and torch.equal(cs, scale) and torch.equal(po2, po)
    if rows:
        r1, s1 = fme.quantize_fp8_block128(x, status=status)
        assert torch.equal(rc, r1) and torch.equal(rs, s1)


def test_cols_without_offsets_is_one_group(status):
    x = special(200, 144)
    codes, scale, po = fme.quantize_fp8_block128(x, fme.COLWISE, status=status)
    v, s = ref.quantize_cols(x, [0, 200])
    assert torch.equal(scale, s) and po.tolist() == [0, 256]
    same(codes, v)


@pytest.mark.parametrize("off", [[1, 5, 10], [0, 6, 5, 10], [0, 5, 9], [0, 5, 11], [0, -3, 10]])
def test_cols_malformed_offsets(off):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    fme.quantize_fp8_block128(outliers((10, 128), 1), fme.COLWISE, i32(off), status=st)
    assert fme.read_device_status(st)[0] == fme.ERR_DEVICE_BAD_OFFSETS


@pytest.mark.parametrize("e,n,k", [(1, 16, 16), (1, 128, 128), (3, 144, 272), (2, 1040, 400), (5, 256, 1024)])
def test_weights(e, n, k, status):
    w = torch.stack([outliers((n, k), i) if i % 2 == 0 else special(n, k) for i in range(e)])
    codes, scale = fme.quantize_fp8_block128_weights(w)
    v, s = ref.quantize_weights(w)
    assert torch.equal(scale, s)
    same(codes, v)


# (rows, experts, n, k): one row, one tile, tiles cut in every direction, contractions below and past a block
GEMM_CASES = [(1, 1, 16, 16), (1, 4, 128, 128), (5, 3, 48, 144), (128, 1, 256, 128), (256, 1, 256, 256),
              (300, 2, 272, 528), (999, 7, 400, 656), (64, 8, 1040, 272), (2000, 4, 512, 1040), (37, 40, 144, 384),
              (3000, 3, 2048, 768)]


def check(y, r, size, contraction, half_ulp=2.0 ** -8):
    err = (y.double() - r).abs()
    lim = ref.bound(r, size, contraction, half_ulp)
    bad = err > lim
    assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} off, worst {float((err / lim.clamp_min(1e-300)).max()):.3g}"
                                 f" of the bound at {bad.nonzero()[0].tolist()}")


@pytest.mark.parametrize("rows,e,n,k", GEMM_CASES)
def test_forward(rows, e, n, k, status):
    off = ref.split(rows, e, rows + n)
    w = fme.quantize_fp8_block128_weights(torch.stack([ref.normal((n, k), 0.02 * 4 ** i, i) for i in range(e)]))
    a = fme.quantize_fp8_block128(outliers((rows, k), 3), status=status)
    y = fme.grouped_gemm_fwd_fp8_block128(*a, *w, i32(off), status=status)
    x, wv = ref.row_operand(*a), ref.weight_operand(*w)
    for i, (lo, hi) in enumerate(zip(off, off[1:])):
        check(y[lo:hi], x[lo:hi] @ wv[i].t(), x[lo:hi].abs() @ wv[i].abs().t(), k) if hi > lo else None


@pytest.mark.parametrize("rows,e,n,k", GEMM_CASES)
def test_dgrad(rows, e, n, k, status):
    off = ref.split(rows, e, rows + k)
    w = fme.quantize_fp8_block128_weights(torch.stack([ref.normal((n, k), 0.02 * 4 ** i, i) for i in range(e)]))
    a = fme.quantize_fp8_block128(outliers((rows, n), 4), status=status)
    dx = fme.grouped_gemm_dgrad_fp8_block128(*a, *w, i32(off), status=status)
    dy, wv = ref.row_operand(*a), ref.weight_operand(*w)
    for i, (lo, hi) in enumerate(zip(off, off[1:])):
        check(dx[lo:hi], dy[lo:hi] @ wv[i], dy[lo:hi].abs() @ wv[i].abs(), n) if hi > lo else None


@pytest.mark.parametrize("rows,e,n,k", GEMM_CASES + [(0, 3, 144, 272)])
def test_wgrad(rows, e, n, k, status):
    off = ref.split(rows, e, rows + 3)
    empty = lambda c: torch.empty((0, c), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    dyc, dys, po = fme.quantize_fp8_block128(outliers((rows, n), 5) if rows else empty(n), fme.COLWISE, i32(off))
    xc, xs, _ = fme.quantize_fp8_block128(outliers((rows, k), 6) if rows else empty(k), fme.COLWISE, i32(off))
    dw = fme.grouped_gemm_wgrad_fp8_block128(dyc, dys, xc, xs, po, status=status)
    dw32 = fme.grouped_gemm_wgrad_fp8_block128(dyc, dys, xc, xs, po, dtype=torch.float32, status=status)
    base = torch.randn((e, n, k), device=DEV)
    acc = base.clone()
    fme.grouped_gemm_wgrad_fp8_block128(dyc, dys, xc, xs, po, dw=acc, accumulate=True, status=status)
    assert torch.equal(dw, dw32.to(torch.bfloat16))
    assert torch.equal(acc, base + dw32)
    dy, x, p = ref.col_operand(dyc, dys), ref.col_operand(xc, xs), ref.padded(off)
    for i in range(e):
        a, b = dy[p[i]:p[i + 1]], x[p[i]:p[i + 1]]
        check(dw32[i], a.t() @ b, a.abs().t() @ b.abs(), p[i + 1] - p[i], 0.0)
    assert not any(bool(dw32[i].any()) for i in range(e) if off[i] == off[i + 1])


@pytest.mark.parametrize("n,k", [(4096, 7168), (400, 656)])
def test_forward_rows_do_not_depend_on_the_batch(n, k, status):
    """The rows of a small batch, alone and inside a large one of the same experts: the same bits."""
    e = 3
    w = fme.quantize_fp8_block128_weights(torch.stack([ref.normal((n, k), 0.02, i) for i in range(e)]))
    x = outliers((3000, k), 9)
    big = [0, 1500, 1600, 3000]
    y = fme.grouped_gemm_fwd_fp8_block128(*fme.quantize_fp8_block128(x), *w, i32(big), status=status)
    for take in ([1, 0, 1], [70, 100, 3], [0, 17, 0], [128, 64, 150]):
        off = np.concatenate([[0], np.cumsum(take)]).tolist()
        rows = torch.cat([torch.arange(big[i], big[i] + take[i], device=DEV) for i in range(e)])
        small = fme.grouped_gemm_fwd_fp8_block128(*fme.quantize_fp8_block128(x[rows].contiguous()), *w, i32(off),
                                                  status=status)
        assert torch.equal(small, y[rows])


@pytest.mark.parametrize("rows", [10, 2000])
@pytest.mark.parametrize("bad", [[1, 0, 0], [0, 1, 0], [0, 0, 1], [0, 5000, 0], [0, -3000, 0]])
def test_products_malformed_offsets_write_nothing(rows, bad):
    n = k = 256
    w = fme.quantize_fp8_block128_weights(torch.stack([ref.normal((n, k), 0.02, i) for i in range(2)]))
    a = fme.quantize_fp8_block128(outliers((rows, k), 1))
    off = i32([bad[0], rows // 2 + bad[1] if bad[1] != 1 else rows + 1, rows + bad[2]])
    for call in (fme.grouped_gemm_fwd_fp8_block128, fme.grouped_gemm_dgrad_fp8_block128):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = torch.full((rows, 256), 3.0, dtype=torch.bfloat16, device=DEV)
        call(*a, *w, off, status=st, **{"y" if call is fme.grouped_gemm_fwd_fp8_block128 else "dx": out})
        assert fme.read_device_status(st)[0] == fme.ERR_DEVICE_BAD_OFFSETS
        assert bool((out == 3.0).all())


@pytest.mark.parametrize("po", [[128, 256, 384], [0, 100, 384], [0, 256, 128], [0, 256, 512]])
def test_wgrad_malformed_offsets_write_nothing(po):
    c = torch.zeros((384, 128), dtype=torch.uint8, device=DEV)
    s = torch.ones((3, 128), device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dw = torch.full((2, 128, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    fme.grouped_gemm_wgrad_fp8_block128(c, s, c, s, i32(po), dw=dw, status=st)
    assert fme.read_device_status(st)[0] == fme.ERR_DEVICE_BAD_OFFSETS and bool((dw == 3.0).all())


def test_nan_codes_of_one_expert_and_row_stay_there(status):
    """0x7F codes (NaN) in one expert's weights and in one row reach no other expert or row, also where
    n and k end inside a tile."""
    n, k = 144, 272
    w, ws = fme.quantize_fp8_block128_weights(torch.stack([ref.normal((n, k), 0.02, i) for i in range(3)]))
    w[1] = 0x7F
    for rows in (30, 900):
        off = [0, rows // 3, 2 * rows // 3, rows]
        a, s = fme.quantize_fp8_block128(ref.normal((rows, k), 1.0, 4))
        a[0] = 0x7F
        y = fme.grouped_gemm_fwd_fp8_block128(a, s, w, ws, i32(off), status=status)
        bad = torch.isnan(y).all(dim=1)
        want = torch.zeros(rows, dtype=torch.bool, device=DEV)
        want[off[1]:off[2]] = True
        want[0] = True
        assert torch.equal(bad, want) and torch.equal(torch.isnan(y).any(dim=1), want)
        d, ds = fme.quantize_fp8_block128(ref.normal((rows, n), 1.0, 4))
        dx = fme.grouped_gemm_dgrad_fp8_block128(d, ds, w, ws, i32(off), status=status)
        want[0] = False
        assert torch.equal(torch.isnan(dx).any(dim=1), want)
