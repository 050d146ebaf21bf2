"""Calls on a stream of their own while the current stream still has work queued on memory that was just freed: what
the calls allocate is not that memory, and an output that the current stream still reads is not given out again."""
import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import block128 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
SLEEP = 200_000_000  # clock cycles: a tenth of a second, far longer than a call


@pytest.fixture(scope="module", autouse=True)
def _built():
    fme.ensure_built()


def flat(out):
    return [out] if torch.is_tensor(out) else [t for o in out for t in flat(o)]


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def calls(seed):
    """Calls of different inputs for each seed, as functions of the stream."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    l = torch.randn((4096, 64), generator=g, device=DEV)
    ids, w = fme.moe_gate(l, 4)
    seq = i32(0, 1000, 4096)
    _, counts, n = fme.moe_balance_loss(l, ids, seq_offsets=seq)
    x = ref.normal((512, 1024), 1.0, seed)
    off = i32(0, 200, 512)
    a = fme.quantize_fp8_block128(x)
    b = fme.quantize_fp8_block128_weights(ref.normal((2, 512, 1024), 0.1, seed))
    c = fme.quantize_fp8_block128(x, fme.COLWISE, off)
    y, d_out = ref.normal((1024, 256), 1.0, seed), ref.normal((256, 256), 1.0, seed + 9)
    row_of = torch.randperm(1024, generator=g, device=DEV).int().reshape(256, 4)
    one = torch.ones(1, device=DEV)
    out = {
        "gate": lambda s: fme.moe_gate(l, 4, stream=s),
        "gate gradient": lambda s: fme.moe_gate_backward(l, ids, w, stream=s),
        "balance": lambda s: fme.moe_balance_loss(l, ids, seq_offsets=seq, stream=s),
        "balance gradient": lambda s: fme.moe_balance_loss_backward(l, counts, n, one, 4, seq_offsets=seq, stream=s),
        "rows": lambda s: fme.quantize_fp8_block128(x, stream=s),
        "columns": lambda s: fme.quantize_fp8_block128(x, fme.COLWISE, off, stream=s),
        "both ways": lambda s: fme.quantize_fp8_block128_rowcol(x, off, stream=s),
        "weights": lambda s: fme.quantize_fp8_block128_weights(y[None], stream=s),
        "forward": lambda s: fme.grouped_gemm_fwd_fp8_block128(*a, *b, off, stream=s),
        "wgrad": lambda s: fme.grouped_gemm_wgrad_fp8_block128(*c[:2], *c, stream=s),
        "combine gradient": lambda s: fme.moe_combine_backward(d_out, y, row_of, w[:256], stream=s),
    }
    return out


NAMES = ["gate", "gate gradient", "balance", "balance gradient", "rows", "columns", "both ways", "weights", "forward",
         "wgrad", "combine gradient"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_uses(name):
    call = calls(1)[name]
    want = [t.clone() for t in flat(call(None))]
    side = torch.cuda.Stream()
    sizes = [t.numel() * t.element_size() for t in want]
    if name == "balance":
        sizes.append(fme.balance_workspace_bytes(4096, 2, 64))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(SLEEP)
    kept = []
    for n in sizes:  # written and read after the sleep, freed now
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


@pytest.mark.parametrize("name", NAMES)
def test_outputs_that_the_current_stream_still_reads(name):
    first, second = calls(2)[name], calls(3)[name]
    want = [t.clone() for t in flat(first(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    out = flat(first(side))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SLEEP)
    kept = [t.clone() for t in out]  # after the sleep
    del out
    again = second(side)
    assert not torch.cuda.current_stream().query(), "the current stream's work is over: nothing was tested"
    torch.cuda.synchronize()
    for k, w in zip(kept, want):
        assert torch.equal(k, w)
    for g, w in zip(flat(again), flat(second(None))):
        assert torch.equal(g, w)
