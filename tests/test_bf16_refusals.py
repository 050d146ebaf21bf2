"""What the bf16 products, the products with NVFP4 weights, SwiGLU and the grouping refuse, on the host and before any
launch (no GPU needed)."""
import pytest

import fp8_moe_expert_gb300 as fme

INVALID, MISALIGNED, SHAPE = fme.ERR_INVALID_ARGUMENT, fme.ERR_MISALIGNED, fme.ERR_UNSUPPORTED_SHAPE
P = 0x1000  # an aligned address that is never used: the checks come first
ODD = 0x1008
LAST = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    fme.ensure_built()
    return fme.lib()


@pytest.mark.parametrize("name", ["grouped_gemm_fwd_bf16", "grouped_gemm_dgrad_bf16"])
def test_row_products(lib, name):
    f = getattr(lib, name)

    def call(**kw):
        a = dict(x=P, w=P, off=P, e=4, m=8, n=128, k=256, y=P)
        a.update(kw)
        return f(a["x"], a["w"], a["off"], a["e"], a["m"], a["n"], a["k"], a["y"], None, None)

    assert call(m=-1) == INVALID and call(n=-8) == INVALID and call(k=-8) == INVALID
    assert call(e=0) == INVALID and call(e=1025) == INVALID and call(off=None) == INVALID
    for bad in (0, 4, 12, 100, 65544):
        assert call(n=bad) == SHAPE and call(k=bad) == SHAPE
    assert call(m=LAST - 200) == SHAPE and call(m=LAST - 256, n=65536, k=65536) == SHAPE
    assert call(m=0, x=None, y=None) == fme.OK
    for arg in ("x", "w", "y"):
        assert call(**{arg: None}) == INVALID and call(**{arg: ODD}) == MISALIGNED
    assert call(off=ODD) == MISALIGNED


def test_weight_gradient(lib):
    def call(**kw):
        a = dict(dy=P, x=P, m=100, off=P, e=2, n=128, k=256, dw=P, mode=0)
        a.update(kw)
        return lib.grouped_gemm_wgrad_bf16(a["dy"], a["x"], a["m"], a["off"], a["e"], a["n"], a["k"], a["dw"], a["mode"],
                                           None, None)

    assert call(mode=3) == INVALID and call(mode=-1) == INVALID and call(m=-1) == INVALID and call(e=0) == INVALID
    assert call(off=None) == INVALID and call(dw=None) == INVALID and call(dy=None) == INVALID and call(x=None) == INVALID
    assert call(n=4) == SHAPE and call(k=12) == SHAPE and call(m=LAST) == SHAPE and call(m=-8) == INVALID
    for arg in ("dy", "x", "off", "dw"):
        assert call(**{arg: ODD}) == MISALIGNED


@pytest.mark.parametrize("name", ["grouped_gemv_nvfp4", "grouped_gemv_nvfp4_swiglu"])
def test_products_with_nvfp4_weights(lib, name):
    f = getattr(lib, name)

    def call(**kw):
        a = dict(x=P, rows=8, src=None, top_k=1, c=P, sf=P, s=P, off=P, e=4, m=8, n=256, k=128, y=P)
        a.update(kw)
        return f(a["x"], a["rows"], a["src"], a["top_k"], a["c"], a["sf"], a["s"], a["off"], a["e"], a["m"], a["n"],
                 a["k"], a["y"], None, None)

    assert call(m=-1) == INVALID and call(rows=-1) == INVALID and call(e=0) == INVALID and call(e=1025) == INVALID
    assert call(m=9) == INVALID and call(top_k=2, m=16) == INVALID            # grouped rows: m rows, top_k 1
    assert call(src=P, top_k=2) == INVALID and call(src=P, top_k=0) == INVALID and call(src=P, top_k=65, m=520) == INVALID
    for bad in (0, 32, 100, 8256):
        assert call(k=bad) == SHAPE
    assert call(n=0) == SHAPE and call(n=65792) == SHAPE
    assert name == "grouped_gemv_nvfp4" or call(n=128) == SHAPE
    assert call(rows=LAST + 1, m=LAST + 1) == SHAPE and call(rows=LAST - 300, m=LAST - 300) == SHAPE
    assert call(off=None) == INVALID
    assert call(rows=0, m=0, x=None, y=None) == fme.OK
    for arg in ("x", "c", "sf", "s", "y"):
        assert call(**{arg: None}) == INVALID and call(**{arg: ODD}) == MISALIGNED
    assert call(off=ODD) == MISALIGNED and call(src=ODD, top_k=2, m=16) == MISALIGNED


def test_swiglu(lib):
    assert lib.swiglu(P, -1, 64, P, None) == INVALID and lib.swiglu(P, 4, -8, P, None) == INVALID
    for bad in (0, 4, 12, 65544):
        assert lib.swiglu(P, 4, bad, P, None) == SHAPE and lib.swiglu_backward(P, P, 4, bad, P, None) == SHAPE
    assert lib.swiglu(P, LAST + 1, 64, P, None) == SHAPE and lib.swiglu(P, LAST, 65536, P, None) == SHAPE
    assert lib.swiglu(None, 0, 64, None, None) == fme.OK and lib.swiglu_backward(None, None, 0, 64, None, None) == fme.OK
    assert lib.swiglu(None, 4, 64, P, None) == INVALID and lib.swiglu(P, 4, 64, None, None) == INVALID
    assert lib.swiglu_backward(P, None, 4, 64, P, None) == INVALID
    assert lib.swiglu(ODD, 4, 64, P, None) == MISALIGNED and lib.swiglu(P, 4, 64, ODD, None) == MISALIGNED
    assert lib.swiglu_backward(P, ODD, 4, 64, P, None) == MISALIGNED


def test_permute(lib):
    f = lib.moe_permute
    assert f(P, -1, 64, P, 2, P, None, None) == INVALID and f(P, 4, -8, P, 2, P, None, None) == INVALID
    assert f(P, 4, 64, P, 0, P, None, None) == INVALID and f(P, 4, 64, P, 65, P, None, None) == INVALID
    for bad in (0, 4, 12, 65544):
        assert f(P, 4, bad, P, 2, P, None, None) == SHAPE
    assert f(P, 1 << 31, 64, P, 1, P, None, None) == SHAPE and f(P, (1 << 63) - 1, 64, P, 64, P, None, None) == SHAPE
    assert f(P, LAST, 65536, P, 1, P, None, None) == SHAPE
    assert f(None, 0, 64, None, 2, None, None, None) == fme.OK
    assert f(None, 4, 64, P, 2, P, None, None) == INVALID and f(P, 4, 64, None, 2, P, None, None) == INVALID
    assert f(ODD, 4, 64, P, 2, P, None, None) == MISALIGNED and f(P, 4, 64, ODD, 2, P, None, None) == MISALIGNED


def test_binding_refuses_other_tensors():
    """Wrong type, place, shape or order: a ValueError that names the argument."""
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    w = torch.zeros((2, 64, 128), dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: fme.grouped_gemm_fwd_bf16(x, w, off), lambda: fme.swiglu(x), lambda: fme.moe_permute(x, off, 1),
                 lambda: fme.grouped_gemm_wgrad_bf16(x, x, off)):
        with pytest.raises(ValueError, match="must be a contiguous CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="w must have 3 dimensions"):
        fme.grouped_gemm_fwd_bf16(x, x, off)
    with pytest.raises(ValueError, match="accumulate into"):
        fme.grouped_gemm_wgrad_bf16(x, x, off, accumulate=True)
    with pytest.raises(ValueError, match="dw is bfloat16 or float32"):
        fme.grouped_gemm_wgrad_bf16(x, x, off, dtype=torch.float16)
    codes, sf, scale = torch.zeros((5, 64), dtype=torch.uint8), torch.zeros(64, dtype=torch.uint8), torch.zeros(5)
    with pytest.raises(ValueError, match="the same number of rows for each of the 2 experts"):
        fme.grouped_gemv_nvfp4(x, codes, sf, scale, off)
    with pytest.raises(ValueError, match="offsets must have at least 2 elements"):
        fme.grouped_gemv_nvfp4(x, codes, sf, scale, off[:1])
    with pytest.raises(ValueError, match="top_k goes with src_row"):
        fme.grouped_gemv_nvfp4(x, codes, sf, scale, off[:2], top_k=2)


def test_mixed_devices_are_refused():
    torch = pytest.importorskip("torch")
    from tests.test_binding_devices import BF16, F32, I32, U8, arguments

    calls = {
        "forward": (fme.grouped_gemm_fwd_bf16, [("x", (4, 128), BF16), ("w", (2, 64, 128), BF16), ("offsets", (3,), I32),
                                                ("=y", (4, 64), BF16), ("=status", (1,), I32)]),
        "dgrad": (fme.grouped_gemm_dgrad_bf16, [("dy", (4, 64), BF16), ("w", (2, 64, 128), BF16), ("offsets", (3,), I32),
                                                ("=status", (1,), I32)]),
        "wgrad": (fme.grouped_gemm_wgrad_bf16, [("dy", (4, 64), BF16), ("x", (4, 128), BF16), ("offsets", (3,), I32),
                                                ("=status", (1,), I32)]),
        "gemv": (lambda *a, **k: fme.grouped_gemv_nvfp4(*a, top_k=2, **k),
                 [("x", (4, 128), BF16), ("w_codes", (256, 64), U8), ("w_sf", (2048,), U8), ("w_scale", (256,), F32),
                  ("offsets", (3,), I32), ("=src_row", (8,), I32), ("=status", (1,), I32)]),
        "gemv with activation": (fme.grouped_gemv_nvfp4_swiglu,
                                 [("x", (4, 128), BF16), ("w_codes", (512, 64), U8), ("w_sf", (4096,), U8),
                                  ("w_scale", (512,), F32), ("offsets", (3,), I32), ("=status", (1,), I32)]),
        "swiglu gradient": (fme.swiglu_backward, [("gate_up", (4, 128), BF16), ("dh", (4, 64), BF16)]),
        "permute": (lambda *a, **k: fme.moe_permute(*a, 2, **k),
                    [("x", (4, 128), BF16), ("src_row", (8,), I32), ("=status", (1,), I32)]),
    }
    fme.ensure_built()
    for call, spec in calls.values():
        for moved in range(1, len(spec)):
            if spec[moved][0] == "=y":  # an output: after the stream's device is looked up, which needs a GPU
                continue
            args, kwargs = arguments([s for s in spec if s[0] != "=y"],
                                     lambda i: 1 if i == moved - sum(s[0] == "=y" for s in spec[:moved]) else 0)
            with pytest.raises(ValueError, match=rf"{spec[moved][0].lstrip('=')} is on cuda:1, {spec[0][0]} on cuda:0"):
                call(*args, **kwargs)


@pytest.mark.gpu
def test_binding_refusals_on_the_gpu():
    import torch

    fme.ensure_built()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="not contiguous"):
        fme.grouped_gemm_fwd_bf16(bf(4, 256)[:, :128], bf(2, 64, 128), off)
    with pytest.raises(ValueError, match="x must be"):
        fme.grouped_gemm_fwd_bf16(bf(4, 64), bf(2, 64, 128), off)
    with pytest.raises(ValueError, match="offsets must be"):
        fme.grouped_gemm_fwd_bf16(bf(4, 128), bf(2, 64, 128), off[:2])
    with pytest.raises(ValueError, match="w must be"):
        fme.grouped_gemm_dgrad_bf16(bf(4, 64), torch.zeros((2, 64, 128), device="cuda"), off)
    with pytest.raises(ValueError, match="dw must be"):
        fme.grouped_gemm_wgrad_bf16(bf(4, 64), bf(4, 128), off, dw=bf(2, 128, 64))
    with pytest.raises(ValueError, match="h must be"):
        fme.swiglu(bf(4, 128), h=bf(4, 128))
    with pytest.raises(ValueError, match="gate_up must be"):
        fme.swiglu(bf(4, 127))
    with pytest.raises(ValueError, match="src_row must be"):
        fme.moe_permute(bf(4, 64), off, 2)
    codes, sf, scale = fme.quantize_nvfp4_pertoken(bf(256, 128))
    with pytest.raises(ValueError, match="w_sf must have at least"):
        fme.grouped_gemv_nvfp4(bf(4, 128), codes, sf[:-16], scale, off)
    with pytest.raises(ValueError, match="w_scale must be"):
        fme.grouped_gemv_nvfp4(bf(4, 128), codes, sf, scale[:-1], off)
    with pytest.raises(ValueError, match="w_codes must be"):
        fme.grouped_gemv_nvfp4(bf(4, 256), codes, sf, scale, off)
    with pytest.raises(fme.FmeError) as e:
        fme.grouped_gemv_nvfp4_swiglu(bf(4, 128), codes, sf, scale, off)  # n = 128: no multiple of 256
    assert e.value.status == SHAPE
    with pytest.raises(fme.FmeError) as e:
        fme.grouped_gemm_fwd_bf16(bf(4, 12), bf(2, 64, 12), off)
    assert e.value.status == SHAPE
    torch.cuda.synchronize()
