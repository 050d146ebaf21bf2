"""Guard bands around every output of the FP8 block-128, router and combine-gradient calls: sizes that end inside
tiles, vectors and warps leave the bytes before and after each output untouched."""
import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import block128 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BAND = 4096  # bytes on each side


@pytest.fixture(scope="module", autouse=True)
def _built():
    fme.ensure_built()


class Guarded:
    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype):
        n = int(torch.tensor(shape).prod()) * torch.empty(0, dtype=dtype).element_size()
        raw = torch.full((2 * BAND + -(-n // 16) * 16,), 0xA5, dtype=torch.uint8, device=DEV)
        self.all.append((raw, n))
        return raw[BAND:BAND + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for i, (raw, n) in enumerate(self.all):
            assert bool((raw[:BAND] == 0xA5).all()), f"output {i}: written before its start"
            assert bool((raw[BAND + n:] == 0xA5).all()), f"output {i}: written past its end"


@pytest.mark.parametrize("rows,cols,groups", [(1, 16, 1), (131, 144, 3), (77, 1040, 9), (300, 528, 2)])
def test_quantizers(rows, cols, groups):
    g = Guarded()
    x = ref.normal((rows, cols), 1.0, 1)
    off = torch.tensor(ref.split(rows, groups, 1), dtype=torch.int32, device=DEV)
    cb, ld = -(-cols // 128), fme.colwise_ld(rows, groups)
    fme.quantize_fp8_block128(x, codes=g((rows, cols), torch.uint8), scale=g((cb, rows), torch.float32))
    fme.quantize_fp8_block128(x, src_row=torch.randperm(3 * rows, device=DEV).int(), top_k=3,
                              codes=g((3 * rows, cols), torch.uint8), scale=g((cb, 3 * rows), torch.float32))
    fme.quantize_fp8_block128(x, fme.COLWISE, off, codes=g((ld, cols), torch.uint8),
                              scale=g((ld // 128, cols), torch.float32), padded_offsets=g((groups + 1,), torch.int32))
    fme.quantize_fp8_block128_rowcol(x, off, row_codes=g((rows, cols), torch.uint8), row_scale=g((cb, rows), torch.float32),
                                     col_codes=g((ld, cols), torch.uint8), col_scale=g((ld // 128, cols), torch.float32),
                                     padded_offsets=g((groups + 1,), torch.int32))
    fme.quantize_fp8_block128_weights(ref.normal((3, 48, cols), 1.0, 2),
                                      codes=g((3, 48, cols), torch.uint8), scale=g((3, 1, cb), torch.float32))
    g.check()


@pytest.mark.parametrize("rows,e,n,k", [(1, 1, 16, 16), (70, 3, 144, 272), (1500, 3, 400, 656), (999, 5, 1040, 144)])
def test_products(rows, e, n, k):
    g = Guarded()
    host = ref.split(rows, e, 2)
    off = torch.tensor(host, dtype=torch.int32, device=DEV)
    w = fme.quantize_fp8_block128_weights(ref.normal((e, n, k), 0.02, 3))
    x, dy = ref.normal((rows, k), 1.0, 4), ref.normal((rows, n), 1.0, 5)
    fme.grouped_gemm_fwd_fp8_block128(*fme.quantize_fp8_block128(x), *w, off, y=g((rows, n), torch.bfloat16))
    fme.grouped_gemm_dgrad_fp8_block128(*fme.quantize_fp8_block128(dy), *w, off, dx=g((rows, k), torch.bfloat16))
    dc, ds, po = fme.quantize_fp8_block128(dy, fme.COLWISE, off)
    xc, xs, _ = fme.quantize_fp8_block128(x, fme.COLWISE, off)
    for dtype, add in ((torch.bfloat16, False), (torch.float32, False), (torch.float32, True)):
        fme.grouped_gemm_wgrad_fp8_block128(dc, ds, xc, xs, po, dw=g((e, n, k), dtype), accumulate=add)
    g.check()


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (5, 31, 3), (33, 100, 8), (9, 256, 8), (3, 1000, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_router(tokens, experts, top_k, dtype):
    g = Guarded()
    l = torch.randn((tokens, experts), device=DEV).to(dtype)
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            ids, w = fme.moe_gate(l, top_k, score=score, normalize=normalize, ids=g((tokens, top_k), torch.int32),
                                  weights=g((tokens, top_k), torch.float32))
            fme.moe_gate_backward(l, ids, w, score=score, normalize=normalize, d_logits=g((tokens, experts), dtype))
        ws = g((fme.balance_workspace_bytes(tokens, 1, experts),), torch.uint8)
        loss, counts, n = fme.moe_balance_loss(l, ids, score=score, loss=g((1,), torch.float32),
                                               counts=g((1, experts), torch.int32), seq_tokens=g((1,), torch.int32),
                                               workspace=ws)
        fme.moe_balance_loss_backward(l, counts, n, loss, top_k, score=score, d_logits=g((tokens, experts), dtype))
    g.check()


@pytest.mark.parametrize("tokens,top_k,n", [(1, 1, 8), (7, 3, 1000), (20, 9, 2056)])
def test_combine_backward(tokens, top_k, n):
    g = Guarded()
    rows = tokens * top_k
    y, d = ref.normal((rows, n), 1.0, 1), ref.normal((tokens, n), 1.0, 2)
    row_of = torch.randperm(rows, device=DEV).int().view(tokens, top_k)
    fme.moe_combine_backward(d, y, row_of, torch.rand((tokens, top_k), device=DEV), d_y=g((rows, n), torch.bfloat16),
                             d_weights=g((tokens, top_k), torch.float32))
    g.check()
