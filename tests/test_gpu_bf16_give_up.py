"""The bf16 products and those with NVFP4 weights in a build whose waits give up at their first look at a barrier that is not
there yet.  Every kernel must give up in each of its forms, report FME_DEV_TIMEOUT and leave an output that is the normal build's
where it was written and untouched elsewhere; the normal build's result afterwards must be unchanged.  No wait is made to
hang: copies and MMAs in flight are awaited with a limit of their own."""
import ctypes
import os

import pytest
import torch

import fp8_moe_expert_gb300 as fme
from fp8_moe_expert_gb300 import build as fme_build
from tests import block128 as ref
from tests import launch_rules

pytestmark = pytest.mark.gpu
ONE_LOOK_LIB = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libfme_one_look.so")
RUNS = 4


@pytest.fixture(scope="module")
def one_look():
    fme.ensure_built()
    os.makedirs(os.path.dirname(ONE_LOOK_LIB), exist_ok=True)
    fme_build.build(output=ONE_LOOK_LIB, extra_flags=["-DFME_WAIT_LIMIT_NS=1ull", "-DFME_WAIT_ONE_LOOK"])
    return fme._declare(ctypes.CDLL(ONE_LOOK_LIB))


def check(fill, normal, short):
    """fill: what the output holds before; normal(out, status) -> the output; short(out pointer, status pointer, stream) ->
    the launch's result."""
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = normal(fill.clone(), st)
    assert fme.read_device_status(st)[0] == 0
    given_up = 0
    for _ in range(RUNS):
        st.zero_()
        out = fill.clone()
        torch.zeros(1 << 26, device="cuda")  # the operands are no longer in L2
        assert short(out.data_ptr(), st.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0, "the launch must succeed"
        code = fme.read_device_status(st)[0]  # synchronises: the kernel has returned
        given_up += code == fme.ERR_DEVICE_TIMEOUT
        assert code in (0, fme.ERR_DEVICE_TIMEOUT)
        assert bool(((out == before) | (out == fill) & (code != 0)).all())
    assert given_up > 0
    st.zero_()
    assert torch.equal(normal(fill.clone(), st), before) and fme.read_device_status(st)[0] == 0


def unlike(*shape, dtype=torch.bfloat16):
    """Values that no result is."""
    return torch.full(shape, 3e38, dtype=dtype, device="cuda")


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# the forward's tiles, and items of 128, 64 and 32 rows of W
@pytest.mark.parametrize("m, n, k, form", [(6000, 1000, 1400, 0), (40, 1000, 1400, 2), (20, 1000, 4096, 4), (3, 1000, 4096, 8)])
def test_forward(one_look, m, n, k, form):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert launch_rules.few_halves(m, n, k, 2, sms) == form
    off = i32(0, m // 3, m)
    x, w = ref.normal((m, k), 1.0, 1), ref.normal((2, n, k), 0.02, 2)
    check(unlike(m, n), lambda y, st: fme.grouped_gemm_fwd_bf16(x, w, off, y=y, status=st),
          lambda y, st, s: one_look.grouped_gemm_fwd_bf16(x.data_ptr(), w.data_ptr(), off.data_ptr(), 2, m, n, k, y, st, s))


def test_dgrad(one_look):
    m, n, k = 3000, 1400, 1000
    off = i32(0, 1000, m)
    dy, w = ref.normal((m, n), 1.0, 1), ref.normal((2, n, k), 0.02, 2)
    check(unlike(m, k), lambda y, st: fme.grouped_gemm_dgrad_bf16(dy, w, off, dx=y, status=st),
          lambda y, st, s: one_look.grouped_gemm_dgrad_bf16(dy.data_ptr(), w.data_ptr(), off.data_ptr(), 2, m, n, k, y, st, s))


# one sum a tile and several, in bf16 and fp32, and an expert that ends within the first 64 rows
@pytest.mark.parametrize("m", [1000, 9000, 70000])
@pytest.mark.parametrize("first", [20, 500])
@pytest.mark.parametrize("mode", [fme.DW_BF16, fme.DW_FP32, fme.DW_FP32_ADD])
def test_wgrad(one_look, m, first, mode):
    n, k = 520, 776
    off = i32(0, first, m)
    dy, x = ref.normal((m, n), 1.0, 1), ref.normal((m, k), 0.02, 2)
    old = unlike(2, n, k, dtype=torch.bfloat16 if mode == fme.DW_BF16 else torch.float32)
    if mode == fme.DW_FP32_ADD:
        old = ref.normal((2, n, k), 1.0, 3).float()
    check(old, lambda dw, st: fme.grouped_gemm_wgrad_bf16(dy, x, off, dw=dw, accumulate=mode == fme.DW_FP32_ADD, status=st),
          lambda dw, st, s: one_look.grouped_gemm_wgrad_bf16(dy.data_ptr(), x.data_ptr(), m, off.data_ptr(), 2, n, k, dw,
                                                             mode, st, s))


# eight, four and two warps to a unit
@pytest.mark.parametrize("experts, n, k, form", [(9, 1024, 8192, 8), (24, 2048, 4096, 4), (24, 2048, 2304, 2)])
@pytest.mark.parametrize("name", ["grouped_gemv_nvfp4", "grouped_gemv_nvfp4_swiglu"])
def test_products_with_nvfp4_weights(one_look, experts, n, k, form, name):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    m = experts
    assert launch_rules.gemv_share(name.endswith("swiglu"), m, n, k, experts, sms) == form
    off = i32(*range(m + 1))
    codes, sf, scale = fme.quantize_nvfp4_pertoken(ref.normal((experts * n, k), 0.05, 1))
    x = ref.normal((m, k), 1.0, 2)
    out, cols = ("h", n // 2) if name.endswith("swiglu") else ("y", n)
    check(unlike(m, cols), lambda y, st: getattr(fme, name)(x, codes, sf, scale, off, status=st, **{out: y}),
          lambda y, st, s: getattr(one_look, name)(x.data_ptr(), m, None, 1, codes.data_ptr(), sf.data_ptr(),
                                                   scale.data_ptr(), off.data_ptr(), experts, m, n, k, y, st, s))
