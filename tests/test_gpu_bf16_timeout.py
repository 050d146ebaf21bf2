"""The bounded waits of the bf16 products and of those with NVFP4 weights in a build whose waits give up after 1 ns (as tests/test_gpu_block128_timeout.py).
Every run must report FME_DEV_TIMEOUT or give the normal build's bits, each pair kernel must time out at least once (the others'
waits may end within a poll), and the
normal build's result afterwards must be unchanged.  No wait is made to hang: copies and MMAs in flight are awaited
with a limit of their own."""
import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import block128 as ref
from tests.test_gpu_block128_timeout import check, short_lib  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
DEEP, N = 32768, 1024


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("counts, pairs", [((2000, 4560), True), ((3, 40), False)])
def test_forward(short_lib, counts, pairs):  # noqa: F811
    m = sum(counts)
    off = i32(0, counts[0], m)
    x, w = ref.normal((m, DEEP), 1.0, 1), ref.normal((2, N, DEEP), 0.02, 2)
    check(lambda st: fme.grouped_gemm_fwd_bf16(x, w, off, status=st),
          lambda y, st, s: short_lib.grouped_gemm_fwd_bf16(x.data_ptr(), w.data_ptr(), off.data_ptr(), 2, m, N, DEEP,
                                                           y.data_ptr(), st, s), gives_up=pairs)


def test_dgrad(short_lib):  # noqa: F811
    m = 456
    off = i32(0, 200, m)
    dy, w = ref.normal((m, DEEP), 1.0, 1), ref.normal((2, DEEP, N), 0.02, 2)
    check(lambda st: fme.grouped_gemm_dgrad_bf16(dy, w, off, status=st),
          lambda y, st, s: short_lib.grouped_gemm_dgrad_bf16(dy.data_ptr(), w.data_ptr(), off.data_ptr(), 2, m, DEEP, N,
                                                             y.data_ptr(), st, s))


@pytest.mark.parametrize("first", [128, 99, 20])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wgrad(short_lib, first, dtype):  # noqa: F811
    """With whole blocks, with blocks that end inside, and with an end in the first 64 rows, which has a producer of its own.  (In fp32 a
    sum is handed over every 16 stages, within a poll.)"""
    off = i32(0, first, DEEP - 1)
    m = DEEP - 1
    dy, x = ref.normal((m, N), 1.0, 1), ref.normal((m, N), 0.02, 2)
    check(lambda st: fme.grouped_gemm_wgrad_bf16(dy, x, off, dtype=dtype, status=st),
          lambda y, st, s: short_lib.grouped_gemm_wgrad_bf16(dy.data_ptr(), x.data_ptr(), m, off.data_ptr(), 2, N, N,
                                                             y.data_ptr(), fme.DW_FP32 if dtype == torch.float32 else fme.DW_BF16, st, s),
          gives_up=dtype == torch.bfloat16)


@pytest.mark.parametrize("rows, k", [(5, 8192), (40, 2048)])
def test_products_with_nvfp4_weights(short_lib, rows, k):  # noqa: F811
    experts, n = 3, 2048
    off = i32(0, rows // 2, rows // 2, rows)
    codes, sf, scale = fme.quantize_nvfp4_pertoken(ref.normal((experts * n, k), 0.05, 1))
    x = ref.normal((rows, k), 1.0, 2)
    for name in ("grouped_gemv_nvfp4", "grouped_gemv_nvfp4_swiglu"):
        check(lambda st: getattr(fme, name)(x, codes, sf, scale, off, status=st),
              lambda y, st, s: getattr(short_lib, name)(x.data_ptr(), rows, None, 1, codes.data_ptr(), sf.data_ptr(),
                                                        scale.data_ptr(), off.data_ptr(), experts, rows, n, k,
                                                        y.data_ptr(), st, s), gives_up=False)
