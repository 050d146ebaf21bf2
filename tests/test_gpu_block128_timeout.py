"""The FP8 block-128 products' bounded waits in a build whose waits give up after 1 ns (as tests/test_gpu_timeout.py
does with 1 us: these kernels wait for one block of 128 at a time, a third of a microsecond).  Every run must report
FME_DEV_TIMEOUT or give the normal build's bits, each pair kernel must time out at least once (the few-rows kernel's
waits end within a poll), and the normal build's result afterwards must be unchanged.  No wait is made to hang: copies
and MMAs in flight are awaited with a limit of their own."""
import ctypes
import os

import pytest
import torch

import fp8_moe_expert_gb300 as fme
from fp8_moe_expert_gb300 import build as fme_build

pytestmark = pytest.mark.gpu
SHORT_LIB = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libfme_shortest_wait.so")
DEEP, N, RUNS = 65536, 1024, 4


@pytest.fixture(scope="module")
def short_lib():
    fme.ensure_built()
    os.makedirs(os.path.dirname(SHORT_LIB), exist_ok=True)
    fme_build.build(output=SHORT_LIB, extra_flags=["-DFME_WAIT_LIMIT_NS=1ull", "-DFME_WAIT_SPINS=1"])
    return fme._declare(ctypes.CDLL(SHORT_LIB))


def codes(*shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(len(shape))
    return torch.randint(0, 120, shape, generator=g, dtype=torch.uint8, device="cuda")


def check(normal, short, gives_up=True):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    before = normal(st)
    assert fme.read_device_status(st)[0] == 0
    timeouts = 0
    for _ in range(RUNS):
        st.zero_()
        out = torch.zeros_like(before)
        assert short(out, st.data_ptr(), stream) == 0, "the launch itself must succeed"
        code, raw = fme.read_device_status(st)  # synchronises: the kernel has returned
        if code == fme.ERR_DEVICE_TIMEOUT:
            timeouts += 1
        else:
            assert code == 0 and torch.equal(out, before), hex(raw)
    assert timeouts > 0 or not gives_up, "no short-wait run timed out"
    st.zero_()
    assert torch.equal(normal(st), before) and fme.read_device_status(st)[0] == 0


@pytest.mark.parametrize("counts, pairs", [((200, 456), True), ((3, 40), False)])
def test_forward(short_lib, counts, pairs):
    m = sum(counts)
    off = torch.tensor([0, counts[0], m], dtype=torch.int32, device="cuda")
    a, sa = codes(m, DEEP), torch.ones((DEEP // 128, m), device="cuda")
    w, sw = codes(2, N, DEEP), torch.ones((2, N // 128, DEEP // 128), device="cuda")
    check(lambda st: fme.grouped_gemm_fwd_fp8_block128(a, sa, w, sw, off, status=st),
          lambda y, st, s: short_lib.grouped_gemm_fwd_fp8_block128(a.data_ptr(), sa.data_ptr(), w.data_ptr(), sw.data_ptr(),
                                                                   off.data_ptr(), 2, m, N, DEEP, y.data_ptr(), st, s),
          gives_up=pairs)


def test_dgrad(short_lib):
    m = 456
    off = torch.tensor([0, 200, m], dtype=torch.int32, device="cuda")
    a, sa = codes(m, DEEP), torch.ones((DEEP // 128, m), device="cuda")
    w, sw = codes(2, DEEP, N), torch.ones((2, DEEP // 128, N // 128), device="cuda")
    check(lambda st: fme.grouped_gemm_dgrad_fp8_block128(a, sa, w, sw, off, status=st),
          lambda y, st, s: short_lib.grouped_gemm_dgrad_fp8_block128(a.data_ptr(), sa.data_ptr(), w.data_ptr(), sw.data_ptr(),
                                                                     off.data_ptr(), 2, m, DEEP, N, y.data_ptr(), st, s))


def test_wgrad(short_lib):
    po = torch.tensor([0, 128, DEEP], dtype=torch.int32, device="cuda")
    d, sd = codes(DEEP, N), torch.ones((DEEP // 128, N), device="cuda")
    x, sx = codes(DEEP, N), torch.ones((DEEP // 128, N), device="cuda")
    check(lambda st: fme.grouped_gemm_wgrad_fp8_block128(d, sd, x, sx, po, dtype=torch.float32, status=st),
          lambda y, st, s: short_lib.grouped_gemm_wgrad_fp8_block128(d.data_ptr(), sd.data_ptr(), x.data_ptr(), sx.data_ptr(),
                                                                     DEEP, po.data_ptr(), 2, N, N, y.data_ptr(),
                                                                     fme.DW_FP32, st, s))
