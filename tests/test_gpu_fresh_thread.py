"""The first call of a host thread that has made no CUDA call yet: every kind of tensor map is encoded there, too."""
import threading

import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import block128 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def in_a_new_thread(call):
    got = []

    def run():
        try:
            got.append(call())
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make(kind):
    """(library function, arguments up to the status) with an output of its own; the output."""
    lib = fme.lib()
    x, off = ref.normal((300, 256), 1.0, 1), i32(0, 300)
    out = torch.zeros((300, 256), dtype=torch.bfloat16, device=DEV)
    if kind.startswith("block128"):
        rows = 40 if kind == "block128 few" else 300
        w = fme.quantize_fp8_block128_weights(ref.normal((1, 256, 256), 0.1, 2))
        a = fme.quantize_fp8_block128(x[:rows].contiguous())
        if kind == "block128 wgrad":
            d, ds, po = fme.quantize_fp8_block128(x, fme.COLWISE, off)
            out = torch.zeros((1, 256, 256), device=DEV)
            return lib.grouped_gemm_wgrad_fp8_block128, (d, ds, d, ds, d.shape[0], po, 1, 256, 256, out, fme.DW_FP32), out
        f = lib.grouped_gemm_dgrad_fp8_block128 if kind == "block128 dgrad" else lib.grouped_gemm_fwd_fp8_block128
        return f, (*a, *w, i32(0, rows), 1, rows, 256, 256, out), out
    if kind == "mxfp8":
        a, b = fme.quantize_mxfp8(x, fme.ROWWISE, off), fme.quantize_mxfp8(x[:256].contiguous())
        return lib.grouped_gemm_fwd_mxfp8, (*a, *b, off, 1, 300, 256, 256, out), out
    a, b = fme.quantize_nvfp4_pertoken(x, off), fme.quantize_nvfp4_pertoken(x[:256].contiguous())
    return lib.grouped_gemm_fwd_nvfp4, (*a, *b, off, 1, 300, 256, 256, out), out


@pytest.mark.parametrize("kind", ["block128 few", "block128 pairs", "block128 dgrad", "block128 wgrad", "mxfp8", "nvfp4"])
def test_first_call_of_a_thread(kind):
    fme.ensure_built()
    f, args, out = make(kind)
    raw = [a.data_ptr() if torch.is_tensor(a) else a for a in args]
    stream = torch.cuda.current_stream().cuda_stream
    assert f(*raw, None, stream) == fme.OK
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    assert in_a_new_thread(lambda: f(*raw, None, stream)) == fme.OK
    torch.cuda.synchronize()
    assert torch.equal(out, want) and bool(want.any())
