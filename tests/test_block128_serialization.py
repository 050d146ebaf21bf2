"""The FP8 block-128 products start while the quantizer before them still writes their operands' scales: they may read
those, and the offsets, with ordinary loads only (__ldg is for data that no one writes while the kernel runs)."""
import os
import re

import pytest

import fp8_moe_expert_gb300 as fme

CSRC = os.path.join(os.path.dirname(os.path.abspath(fme.__file__)), "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", ["gemm_block128.cu", "block128.cuh"])
def test_no_non_coherent_loads(name):
    assert not re.findall(r"__ldg|ld\.global\.nc|__restrict__", source(name))


@pytest.mark.gpu
def test_scales_written_by_the_kernel_right_before():
    """Quantizer and product back to back into the same buffers, many times, with scales that change each time: the
    bits of a run that waits between the two.  The forward in both its forms, dgrad, and two products in a row."""
    import torch

    from tests import block128 as ref

    fme.ensure_built()
    dev = "cuda"
    for rows in (64, 1024):
        n, k, rounds = 384, 2048, 40
        off = torch.tensor([0, rows // 4, rows], dtype=torch.int32, device=dev)
        w = fme.quantize_fp8_block128_weights(ref.normal((2, n, k), 0.05, 1))
        wt = fme.quantize_fp8_block128_weights(ref.normal((2, k, n), 0.05, 2))
        x = [ref.normal((rows, k), 2.0 ** (i % 9 - 4), i) for i in range(rounds)]
        codes, scale = fme.quantize_fp8_block128(x[0])
        y = torch.empty((rounds, rows, n), dtype=torch.bfloat16, device=dev)
        dx = torch.empty((rounds, rows, n), dtype=torch.bfloat16, device=dev)

        def run(wait):
            for i in range(rounds):
                fme.quantize_fp8_block128(x[i], codes=codes, scale=scale)
                wait()
                fme.grouped_gemm_fwd_fp8_block128(codes, scale, *w, off, y=y[i])
                wait()
                fme.grouped_gemm_dgrad_fp8_block128(codes, scale, *wt, off, dx=dx[i])
                wait()

        run(torch.cuda.synchronize)
        want = y.clone(), dx.clone()
        y.zero_()
        dx.zero_()
        run(lambda: None)
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
