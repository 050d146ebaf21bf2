"""The bf16 products, the products with NVFP4 weights, SwiGLU and the grouping as a program calls them: one after the other
without a wait, on streams of their own, from several host threads, captured and replayed."""
import os
import re
import threading

import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import block128 as ref

DEV = "cuda"
SLEEP = 200_000_000  # clock cycles: a tenth of a second, far longer than a call
CSRC = os.path.join(os.path.dirname(os.path.abspath(fme.__file__)), "csrc")


@pytest.mark.parametrize("name", ["gemm_bf16.cu", "gemm_tiles.cuh", "gemv_nvfp4.cu", "activation.cu", "swiglu.cuh"])
def test_no_non_coherent_loads(name):
    """These kernels start while the one before them still writes their operands: ordinary loads only."""
    source = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert not re.findall(r"__ldg|ld\.global\.nc|__restrict__", source)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module", autouse=True)
def _built():
    fme.ensure_built()


def calls(seed):
    """Calls of different inputs for each seed, as functions of the stream."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    tokens, top_k, experts, n, k = 3000, 4, 6, 256, 384
    ids = torch.rand((tokens, experts), generator=g, device=DEV).argsort(dim=1)[:, :top_k].int().contiguous()
    off, _, src = fme.moe_route(ids, experts)
    x, w = ref.normal((tokens, k), 1.0, seed), ref.normal((experts, n, k), 0.05, seed + 1)
    rows = fme.moe_permute(x, src, top_k)
    dy = ref.normal((tokens * top_k, n), 0.1, seed + 2)
    w4 = fme.quantize_nvfp4_pertoken(w.view(-1, k))
    few_off, few = i32(0, 3, 3, 4, 8, 9, 11), x[:11].contiguous()
    dh = ref.normal((tokens * top_k, n // 2), 0.1, seed + 3)
    return {
        "forward": lambda s: fme.grouped_gemm_fwd_bf16(rows, w, off, stream=s),
        "forward, few rows": lambda s: fme.grouped_gemm_fwd_bf16(few, w, few_off, stream=s),
        "dgrad": lambda s: fme.grouped_gemm_dgrad_bf16(dy, w, off, stream=s),
        "wgrad": lambda s: fme.grouped_gemm_wgrad_bf16(dy, rows, off, stream=s),
        "gemv": lambda s: fme.grouped_gemv_nvfp4(few, *w4, few_off, stream=s),
        "gathered gemv with activation": lambda s: fme.grouped_gemv_nvfp4_swiglu(x, *w4, off, src_row=src, top_k=top_k,
                                                                                 stream=s),
        "swiglu": lambda s: fme.swiglu(dy, stream=s),
        "swiglu gradient": lambda s: fme.swiglu_backward(dy, dh, stream=s),
        "permute": lambda s: fme.moe_permute(x, src, top_k, stream=s),
    }


NAMES = ["forward", "forward, few rows", "dgrad", "wgrad", "gemv", "gathered gemv with activation", "swiglu",
         "swiglu gradient", "permute"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_uses(name):
    call = calls(1)[name]
    want = call(None).clone()
    side = torch.cuda.Stream()
    size = want.numel() * want.element_size()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(SLEEP)
    t = torch.empty(size, dtype=torch.uint8, device=DEV)  # written and read after the sleep, freed now
    t.fill_(0x5B)
    kept = t.clone()
    del t
    got = call(side)
    assert not torch.cuda.current_stream().query(), "the current stream's work is over: nothing was tested"
    side.synchronize()
    torch.cuda.synchronize()
    assert bool((kept == 0x5B).all()) and torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_outputs_that_the_current_stream_still_reads(name):
    first, second = calls(2)[name], calls(30)[name]
    want, later = first(None).clone(), second(None).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    out = first(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SLEEP)
    kept = out.clone()  # after the sleep
    del out
    again = second(side)
    assert not torch.cuda.current_stream().query(), "the current stream's work is over: nothing was tested"
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and torch.equal(again, later)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [40, 4000])
def test_each_call_reads_what_the_call_before_wrote(rows):
    """A chain through the same buffers, many times, with other rows each time: the bits of a chain that waits after
    every call.  40 rows: the forward's form for few."""
    experts, k, rounds = 3, 512, 30
    inter = 256
    off = i32(0, rows // 4, rows // 4, rows)
    gate_up, down = ref.normal((experts, 2 * inter, k), 0.05, 1), ref.normal((experts, k, inter), 0.05, 2)
    gu4, down4 = fme.quantize_nvfp4_pertoken(gate_up.view(-1, k)), fme.quantize_nvfp4_pertoken(down.view(-1, inter))
    xs = [ref.normal((rows, k), 2.0 ** (i % 5 - 2), i) for i in range(rounds)]
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    src = torch.randperm(rows, generator=g, device=DEV).int()
    perm = torch.empty((rows, k), dtype=torch.bfloat16, device=DEV)
    gu = torch.empty((rows, 2 * inter), dtype=torch.bfloat16, device=DEV)
    h = torch.empty((rows, inter), dtype=torch.bfloat16, device=DEV)
    dgu, dh = torch.empty_like(gu), torch.empty_like(h)
    y = torch.empty((rounds, rows, k), dtype=torch.bfloat16, device=DEV)
    dx, y4 = torch.empty_like(y), torch.empty_like(y)
    dw = torch.empty((rounds, experts, 2 * inter, k), dtype=torch.bfloat16, device=DEV)

    def run(wait):
        for i in range(rounds):
            fme.moe_permute(xs[i], src, 1, out=perm)
            wait()
            fme.grouped_gemm_fwd_bf16(perm, gate_up, off, y=gu)
            wait()
            fme.swiglu(gu, h=h)
            wait()
            fme.grouped_gemm_fwd_bf16(h, down, off, y=y[i])
            wait()
            fme.grouped_gemm_dgrad_bf16(y[i], down, off, dx=dh)
            wait()
            fme.swiglu_backward(gu, dh, d_gate_up=dgu)
            wait()
            fme.grouped_gemm_wgrad_bf16(dgu, perm, off, dw=dw[i])
            wait()
            fme.grouped_gemm_dgrad_bf16(dgu, gate_up, off, dx=dx[i])
            wait()
            fme.grouped_gemv_nvfp4_swiglu(perm, *gu4, off, h=h)
            wait()
            fme.grouped_gemv_nvfp4(h, *down4, off, y=y4[i])
            wait()

    run(torch.cuda.synchronize)
    want = [t.clone() for t in (y, dx, dw, y4)]
    for t in (y, dx, dw, y4):
        t.zero_()
    run(lambda: None)
    torch.cuda.synchronize()
    for got, w in zip((y, dx, dw, y4), want):
        assert torch.equal(got, w)


@pytest.mark.gpu
def test_two_host_threads_on_two_streams():
    """The same calls at once from two threads, each on its own stream and with its own expert count."""
    made = [calls(5), calls(60)]
    want = [{n: c(None).clone() for n, c in m.items()} for m in made]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    for name, call in made[i].items():
                        if not torch.equal(call(None), want[i][name]):
                            wrong.append((i, name))
        except Exception as e:  # noqa: BLE001
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name):
    call = calls(7)[name]
    want = call(None).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(None)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


@pytest.mark.gpu
def test_tensors_of_more_than_32_bits_of_elements():
    """Outputs of 2.6e9 elements and weights of 4.3e9 bytes: rows at both ends and in the middle against 64 bits (small
    integers: every sum is exact)."""
    def ints(*shape):
        return torch.randint(-2, 3, shape, device=DEV).to(torch.bfloat16)

    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    torch.manual_seed(1)
    m, n, k = 40000, 65536, 8
    x, w, off = ints(m, k), ints(2, n, k), i32(0, 30000, m)
    y = fme.grouped_gemm_fwd_bf16(x, w, off, status=st)
    for r in (0, 29999, 30000, m - 1):
        assert torch.equal(y[r], (x[r].double() @ w[int(r >= 30000)].double().t()).to(torch.bfloat16))
    dx = fme.grouped_gemm_dgrad_bf16(y, w, off, status=st)  # rows of y past 2^31 elements
    for r in (0, m - 1):
        want = y[r].double() @ w[int(r >= 30000)].double()
        size = y[r].double().abs() @ w[int(r >= 30000)].double().abs()
        assert bool(((dx[r].double() - want).abs() <= 2.0 ** -8 * want.abs() + (n + 1) * 2.0 ** -23 * size).all())
    g = fme.swiglu(y, h=torch.empty((m, n // 2), dtype=torch.bfloat16, device=DEV))
    assert torch.equal(g[m - 1:], fme.swiglu(y[m - 1:].clone()))
    d = fme.swiglu_backward(y, g)
    assert torch.equal(d[m - 1:], fme.swiglu_backward(y[m - 1:].clone(), g[m - 1:].clone()))
    del d, g
    src = torch.arange(m - 1, -1, -1, dtype=torch.int32, device=DEV)
    p = fme.moe_permute(y, src, 1, out=torch.empty_like(y), status=st)
    assert torch.equal(p[0], y[m - 1]) and torch.equal(p[m - 1], y[0]) and torch.equal(p[30001], y[m - 30002])
    del p, y
    experts, n, k = 40, 8192, 8192
    dy, x = ints(300, n), ints(300, k)
    off = torch.tensor([0] * experts + [300], dtype=torch.int32, device=DEV)
    off[1:experts] = 100
    dw = fme.grouped_gemm_wgrad_bf16(dy, x, off, status=st)
    assert torch.equal(dw[-1, -5:], (dy[100:, -5:].double().t() @ x[100:].double()).to(torch.bfloat16))
    assert torch.equal(dw[0, :5], (dy[:100, :5].double().t() @ x[:100].double()).to(torch.bfloat16))
    assert not bool(dw[1].any())
    del dw
    experts, n, k = 64, 16384, 8192
    codes = torch.randint(0, 256, (experts * n, k // 2), dtype=torch.uint8, device=DEV)
    sf = torch.full((experts * n * k // 16,), 0x38, dtype=torch.uint8, device=DEV)
    scale = torch.ones(experts * n, device=DEV)
    x = ints(3, k)
    off = torch.tensor([0] * (experts - 1) + [1, 3], dtype=torch.int32, device=DEV)
    y = fme.grouped_gemv_nvfp4(x, codes, sf, scale, off, status=st)
    from tests import nvfp4w

    last = slice((experts - 1) * n, experts * n)
    w = nvfp4w.values(codes[last][-512:], sf[:512 * k // 16], scale[:512])
    assert torch.equal(y[1:, -512:], (x[1:].double() @ w.t()).to(torch.bfloat16))
    assert fme.read_device_status(st)[0] == 0
