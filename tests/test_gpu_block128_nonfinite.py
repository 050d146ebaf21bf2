"""Blocks that hold infinities and NaN, in every layout of the FP8 block-128 quantizers: the largest magnitude is taken
over the values that are not NaN, scale = A / 448 and r = 448 / A are IEEE quotients also for A = inf (inf and 0), so
finite values of such a block get codes 0 and its infinities NaN; a NaN gets a NaN code and leaves the others alone."""
import numpy as np
import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import block128 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    fme.ensure_built()


def with_inf(rows, cols):
    x = ref.normal((rows, cols), 1.0, 1)
    x[3, 5], x[3, 200], x[77, 130], x[rows - 1, cols - 1] = INF, -INF, -INF, INF
    x[9, 64:70] = INF
    return x


def blocks(x, rows, cols):
    """x [R, C] zero-padded and cut: [R', C', rows, cols]."""
    r, c = x.shape
    full = torch.zeros((-(-r // rows) * rows, -(-c // cols) * cols), dtype=torch.float32, device=DEV)
    full[:r, :c] = x.float()
    return full.view(full.shape[0] // rows, rows, full.shape[1] // cols, cols).transpose(1, 2)


def expected(x, rows, cols):
    """(values the codes stand for, scales) of x in blocks of rows x cols."""
    b = blocks(x, rows, cols)
    mag = torch.where(torch.isnan(b), torch.zeros_like(b), b.abs()).amax(dim=(2, 3)).clamp_min(2.0 ** -100)
    a = mag.cpu().numpy()
    scale = torch.from_numpy(a / np.float32(448.0)).to(DEV)
    r = torch.from_numpy(np.float32(448.0) / a).to(DEV)
    v = (b * r[:, :, None, None]).double()
    v = torch.where(torch.isnan(v), v, ref.e4m3_round(torch.where(torch.isnan(v), torch.zeros_like(v), v)))
    full = v.transpose(1, 2).reshape(b.shape[0] * rows, b.shape[1] * cols)
    return full, scale


def same(codes, want):
    got = ref.values(codes)
    want = want[:got.shape[0], :got.shape[1]]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


def check_every_layout(x):
    rows, cols = x.shape
    v, s = expected(x, 1, 128)
    codes, scale = fme.quantize_fp8_block128(x)
    assert torch.equal(scale, s.t())
    same(codes, v)
    src = torch.arange(2 * rows, dtype=torch.int32, device=DEV)
    gathered = fme.quantize_fp8_block128(x, src_row=src, top_k=2)
    assert torch.equal(gathered[0][0::2], codes) and torch.equal(gathered[1][:, 1::2], scale)
    vc, sc = expected(x, 128, 1)
    cols_out = fme.quantize_fp8_block128(x, fme.COLWISE)
    ld = cols_out[0].shape[0]
    assert torch.equal(cols_out[1], sc[:, :cols][:ld // 128])
    same(cols_out[0], vc)
    both = fme.quantize_fp8_block128_rowcol(x)
    for got, want in zip(both[0] + both[1], (codes, scale) + cols_out):
        assert torch.equal(got, want)
    vw, sw = expected(x[:288] if rows > 288 else x, 128, 128)
    w = (x[:288] if rows > 288 else x)[None].contiguous()
    wq = fme.quantize_fp8_block128_weights(w)
    assert torch.equal(wq[1][0], sw)
    same(wq[0][0], vw)


@pytest.mark.parametrize("rows,cols", [(160, 272), (300, 512)])
def test_infinities(rows, cols):
    check_every_layout(with_inf(rows, cols))


def with_nan(rows, cols):
    """NaN at every even, every odd, all, or single positions of rows, and down the columns."""
    x = ref.normal((rows, cols), 1.0, 2)
    x[2, 0::2], x[4, 1::2], x[6], x[8, 17], x[10, 130:140] = NAN, NAN, NAN, NAN, NAN
    x[:, 40], x[0::2, 41], x[1::2, 42], x[20:30, 150:160] = NAN, NAN, NAN, NAN
    x[128:136, 144:152] = NAN  # a thread's whole share of a tile
    return x


@pytest.mark.parametrize("rows,cols", [(160, 272), (300, 512)])
def test_nan(rows, cols):
    check_every_layout(with_nan(rows, cols))
