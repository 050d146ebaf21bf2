"""The NVFP4, MXFP8 and routing calls on a stream of their own, as tests/test_gpu_side_stream.py: what they allocate is not
memory that the current stream still uses, and their hidden workspace is not given out while they run."""
import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import block128 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
SLEEP = 200_000_000


@pytest.fixture(scope="module", autouse=True)
def _built():
    fme.ensure_built()


def flat(out):
    return [out] if torch.is_tensor(out) else [t for o in out if not isinstance(o, int) for t in flat(o)]


def calls(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x, y = ref.normal((512, 1024), 1.0, seed), ref.normal((512, 256), 1.0, seed + 1)
    off = torch.tensor([0, 256, 512], dtype=torch.int32, device=DEV)
    ids = torch.randint(0, 8, (300, 2), generator=g, device=DEV).int()
    row_of = torch.randperm(512, generator=g, device=DEV).int().reshape(256, 2)
    w = torch.rand((256, 2), generator=g, device=DEV)
    a4, b4 = fme.quantize_nvfp4_pertoken(x, off), fme.quantize_nvfp4_pertoken(x)
    a8, b8 = fme.quantize_mxfp8(x, fme.ROWWISE, off), fme.quantize_mxfp8(x)
    c8 = fme.quantize_mxfp8(y, fme.COLWISE, off)
    src = torch.arange(1024, dtype=torch.int32, device=DEV)
    off2 = 2 * off
    return {
        "nvfp4": lambda s: fme.quantize_nvfp4_pertoken(x, off, stream=s)[::2],
        "swiglu nvfp4": lambda s: fme.swiglu_quantize_nvfp4(x, off, stream=s)[::2],
        "mxfp8": lambda s: fme.quantize_mxfp8(x, fme.ROWWISE, off, stream=s)[0],
        # (positions past the 512 rows' are not written)
        "mxfp8 columns": lambda s: fme.quantize_mxfp8(x, fme.COLWISE, off, stream=s)[0][:, :512],
        "forward nvfp4": lambda s: fme.grouped_gemm_fwd_nvfp4(*a4, b4[0], b4[1], b4[2], off, 256, 1024, stream=s),
        "forward mxfp8": lambda s: fme.grouped_gemm_fwd_mxfp8(*a8, *b8, off, 256, 1024, stream=s),
        "wgrad mxfp8": lambda s: fme.grouped_gemm_wgrad_mxfp8(c8[0], c8[1], c8[3], c8[0], c8[1], c8[3], c8[2], 256, 256,
                                                              stream=s),
        "route": lambda s: fme.moe_route(ids, 8, stream=s),
        "gathered nvfp4": lambda s: fme.permute_quantize_nvfp4(x, src, 2, off2, stream=s)[::2],
        "combine": lambda s: fme.moe_combine(y, row_of, w, stream=s),
    }


NAMES = ["nvfp4", "swiglu nvfp4", "mxfp8", "mxfp8 columns", "forward nvfp4", "forward mxfp8", "wgrad mxfp8", "route",
         "gathered nvfp4", "combine"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_uses(name):
    call = calls(1)[name]
    want = [t.clone() for t in flat(call(None))]
    side = torch.cuda.Stream()
    sizes = [t.numel() * t.element_size() for t in want]
    if name == "route":
        sizes.append(fme.route_workspace_bytes(300, 2, 8))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(SLEEP)
    kept = []
    for n in sizes:
        t = torch.empty(n, dtype=torch.uint8, device=DEV)
        t.fill_(0x5B)
        kept.append(t.clone())
        del t
    got = flat(call(side))
    assert not torch.cuda.current_stream().query(), "the current stream's work is over: nothing was tested"
    side.synchronize()
    torch.cuda.synchronize()
    assert all(bool((k == 0x5B).all()) for k in kept)
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_route_workspace_stays_its_own_until_the_call_is_done():
    ids = torch.randint(0, 8, (20000, 2), device=DEV).int()
    want = [t.clone() for t in fme.moe_route(ids, 8)]
    n = fme.route_workspace_bytes(20000, 2, 8)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    got = fme.moe_route(ids, 8, stream=side)  # its workspace is freed when it returns, its kernels still wait
    taken = [torch.full((n,), 0x5B, dtype=torch.uint8, device=DEV) for _ in range(8)]
    torch.cuda.current_stream().synchronize()
    assert not side.query(), "the side stream's work is over: nothing was tested"
    torch.cuda.synchronize()
    assert all(bool((t == 0x5B).all()) for t in taken)
    for g, w in zip(got, want):
        assert torch.equal(g, w)
