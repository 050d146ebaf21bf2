"""The combine and its gradient at the widest rows they accept, 2^31 - 8 columns, and past them."""
import pytest

import fp8_moe_expert_gb300 as fme

P = 0x1000
WIDEST = (1 << 31) - 8


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 64])
def test_wider_rows_are_refused(n):
    fme.ensure_built()
    lib = fme.lib()
    assert lib.moe_combine(P, 1, P, P, 1, 1, n, P, None, None) == fme.ERR_UNSUPPORTED_SHAPE
    assert lib.moe_combine_backward(P, P, 1, P, P, 1, 1, n, P, P, None, None) == fme.ERR_UNSUPPORTED_SHAPE


@pytest.mark.gpu
def test_gradient_of_the_widest_row():
    import torch

    fme.ensure_built()
    bf16, dev = torch.bfloat16, "cuda"
    y = torch.zeros((1, WIDEST), dtype=bf16, device=dev)
    at = [0, 5, (1 << 30) + 3, WIDEST - 2049, WIDEST - 2048, WIDEST - 9, WIDEST - 1]
    y[0, at] = torch.arange(1, len(at) + 1, dtype=bf16, device=dev)
    d_out = torch.full((1, WIDEST), 2.0, dtype=bf16, device=dev)
    d_out[0, at] = 4.0
    row_of, w = torch.zeros((1, 1), dtype=torch.int32, device=dev), torch.full((1, 1), 0.5, device=dev)
    d_y, dw = fme.moe_combine_backward(d_out, y, row_of, w)
    assert dw.item() == 4.0 * sum(range(1, len(at) + 1))
    assert bool((d_y[0, at] == 2.0).all())
    d_y[0, at] = 1.0
    assert bool((d_y == 1.0).all())
