"""Calls of different expert counts from two host threads at once: a launch's shared memory grows with the number of
experts, and no thread's call may take that room from another's."""
import threading

import pytest
import torch

import fp8_moe_expert_gb300 as fme

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROUNDS = 3000


@pytest.fixture(scope="module", autouse=True)
def _built():
    fme.ensure_built()


def offsets(experts, rows):
    off = torch.full((experts + 1,), rows, dtype=torch.int32, device=DEV)
    off[0] = 0
    return off


def block128(kind, experts, n=16, k=16):
    """One call of a product with `experts` experts, all rows in the first."""
    rows = 40 if kind == "few" else 40000
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    codes = lambda *s: torch.randint(0, 120, s, generator=g, dtype=torch.uint8, device=DEV)  # noqa: E731
    off = offsets(experts, rows)
    a, sa = codes(rows, k), torch.ones((1, rows), device=DEV)
    w, sw = codes(1, n, k).repeat(experts, 1, 1), torch.ones((experts, 1, 1), device=DEV)
    if kind == "wgrad":
        po = offsets(experts, 256)
        d, sd = codes(256, n), torch.ones((2, n), device=DEV)
        out = torch.empty((experts, n, k), dtype=torch.bfloat16, device=DEV)
        return lambda: fme.grouped_gemm_wgrad_fp8_block128(d, sd, d, sd, po, dw=out)[0]
    out = torch.empty((rows, n), dtype=torch.bfloat16, device=DEV)
    if kind == "dgrad":
        return lambda: fme.grouped_gemm_dgrad_fp8_block128(a, sa, w, sw, off, dx=out)
    return lambda: fme.grouped_gemm_fwd_fp8_block128(a, sa, w, sw, off, y=out)


def nvfp4_quantizer(experts):
    x = torch.ones((64, 256), device=DEV).bfloat16()
    off = offsets(experts, 64)
    out = fme.quantize_nvfp4_pertoken(x, off)
    kw = dict(codes=out[0], sf=out[1], row_scale=out[2])
    return lambda: fme.quantize_nvfp4_pertoken(x, off, **kw)[0]


def mxfp8_product(experts):
    x = torch.ones((64, 256), device=DEV).bfloat16()
    off = offsets(experts, 64)
    a = fme.quantize_mxfp8(x, fme.ROWWISE, off)
    b = fme.quantize_mxfp8(torch.ones((experts * 256, 256), device=DEV).bfloat16())
    y = torch.empty((64, 256), dtype=torch.bfloat16, device=DEV)
    return lambda: fme.grouped_gemm_fwd_mxfp8(*a, *b, off, 256, 256, y=y)


MAKERS = {"few": lambda e: block128("few", e), "pairs": lambda e: block128("pairs", e),
          "dgrad": lambda e: block128("dgrad", e), "wgrad": lambda e: block128("wgrad", e),
          "nvfp4 quantizer": nvfp4_quantizer, "mxfp8 product": mxfp8_product}


@pytest.mark.parametrize("what", list(MAKERS))
def test_two_threads(what):
    calls = [MAKERS[what](e) for e in (1, fme.MAX_GROUPS)]
    want = [c().clone() for c in calls]
    torch.cuda.synchronize()
    start, failed = threading.Barrier(2), []

    def run(i):
        stream = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(stream):
            for r in range(ROUNDS):
                try:
                    calls[i]()
                except Exception as e:  # noqa: BLE001
                    failed.append((i, r, str(e)))
                    return
                if r % 256 == 255:
                    stream.synchronize()
        stream.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert torch.equal(c(), w)


def test_no_symbol_of_the_library_is_shared_between_two_builds_of_it():
    """State that a launcher keeps must be its own library's: a process may load a second build, whose functions need
    their limits raised as well.  (`u` in nm: one object for the whole process.)"""
    import subprocess

    out = subprocess.run(["nm", fme.LIBRARY], capture_output=True, text=True, check=True).stdout
    assert not [line for line in out.splitlines() if line.split()[-2:-1] == ["u"] and "fme" in line]
