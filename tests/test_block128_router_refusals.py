"""What the FP8 block-128 and router calls refuse, on the host and before any launch (no GPU needed)."""
import pytest

import fp8_moe_expert_gb300 as fme

INVALID, MISALIGNED, SHAPE = fme.ERR_INVALID_ARGUMENT, fme.ERR_MISALIGNED, fme.ERR_UNSUPPORTED_SHAPE
P = 0x1000  # an aligned address that is never used: the checks come first
ODD = 0x1008


@pytest.fixture(scope="module")
def lib():
    fme.ensure_built()
    return fme.lib()


def test_quantizers(lib):
    q = lib.quantize_fp8_block128
    assert q(P, -1, 128, 0, None, 1, P, P, None, None, None) == INVALID
    assert q(P, 4, 128, 2, None, 1, P, P, None, None, None) == INVALID          # axis
    assert q(P, 4, 128, 0, None, 2, P, P, None, None, None) == INVALID          # groups without offsets
    assert q(P, 4, 128, 0, None, 1, P, P, P, None, None) == INVALID             # padded offsets of a row-wise call
    assert q(P, 4, 128, 1, None, 1, P, P, None, None, None) == INVALID          # none of a column-wise one
    assert q(P, 4, 128, 0, P, 1025, P, P, None, None, None) == INVALID
    for cols in (0, 8, 24, 130, 65552):
        assert q(P, 4, cols, 0, None, 1, P, P, None, None, None) == SHAPE
        assert q(P, 4, cols, 1, None, 1, P, P, P, None, None) == SHAPE
        assert lib.permute_quantize_fp8_block128(P, 4, cols, P, 2, P, P, None, None) == SHAPE
    assert q(P, 1 << 31, 128, 0, None, 1, P, P, None, None, None) == SHAPE
    assert q(None, 4, 128, 0, None, 1, P, P, None, None, None) == INVALID
    for i in (0, 6, 7):
        a = [P, 4, 128, 0, None, 1, P, P, None, None, None]
        a[i] = ODD
        assert q(*a) == MISALIGNED
    assert q(None, 0, 128, 0, None, 1, None, None, None, None, None) == fme.OK  # no rows: nothing to do
    assert lib.quantize_fp8_block128_rowcol(P, 4, 128, None, 1, None, P, P, P, P, None, None) == INVALID
    assert lib.permute_quantize_fp8_block128(P, 4, 128, P, 0, P, P, None, None) == INVALID
    assert lib.permute_quantize_fp8_block128(P, 4, 128, P, 65, P, P, None, None) == INVALID
    assert lib.permute_quantize_fp8_block128(P, 4, 128, None, 2, P, P, None, None) == INVALID
    assert lib.quantize_fp8_block128_weights(P, 0, 128, 128, P, P, None) == INVALID
    assert lib.quantize_fp8_block128_weights(P, 2, 120, 128, P, P, None) == SHAPE
    assert lib.quantize_fp8_block128_weights(P, 2, 128, 128, ODD, P, None) == MISALIGNED


@pytest.mark.parametrize("name", ["grouped_gemm_fwd_fp8_block128", "grouped_gemm_dgrad_fp8_block128"])
def test_row_products(lib, name):
    f = getattr(lib, name)

    def call(**kw):
        a = dict(a=P, sa=P, w=P, sw=P, off=P, e=4, m=8, n=128, k=256, y=P)
        a.update(kw)
        return f(a["a"], a["sa"], a["w"], a["sw"], a["off"], a["e"], a["m"], a["n"], a["k"], a["y"], None, None)

    assert call(m=-1) == INVALID and call(e=0) == INVALID and call(e=1025) == INVALID and call(off=None) == INVALID
    for bad in (0, 8, 100, 65552):
        assert call(n=bad) == SHAPE and call(k=bad) == SHAPE
    assert call(m=(1 << 31) - 200) == SHAPE
    assert call(m=0, a=None, y=None) == fme.OK
    for name_ in ("a", "sa", "w", "sw", "y"):
        assert call(**{name_: None}) == INVALID and call(**{name_: ODD}) == MISALIGNED
    assert call(off=ODD) == MISALIGNED


def test_weight_gradient(lib):
    def call(**kw):
        a = dict(d=P, sd=P, x=P, sx=P, pos=256, po=P, e=2, n=128, k=256, dw=P, mode=0)
        a.update(kw)
        return lib.grouped_gemm_wgrad_fp8_block128(a["d"], a["sd"], a["x"], a["sx"], a["pos"], a["po"], a["e"], a["n"],
                                                   a["k"], a["dw"], a["mode"], None, None)

    assert call(mode=3) == INVALID and call(pos=-128) == INVALID and call(po=None) == INVALID and call(dw=None) == INVALID
    assert call(pos=100) == SHAPE and call(n=24) == SHAPE and call(k=8) == SHAPE
    for name in ("d", "sd", "x", "sx", "dw", "po"):
        assert call(**{name: ODD}) == MISALIGNED
    for name in ("d", "sd", "x", "sx"):
        assert call(**{name: None}) == INVALID


def test_router(lib):
    def gate(**kw):
        a = dict(l=P, dt=1, t=4, e=8, k=2, s=0, ids=P, w=P, b=None)
        a.update(kw)
        return lib.moe_gate(a["l"], a["dt"], a["t"], a["e"], a["k"], a["s"], 1, 1.0, a["b"], a["ids"], a["w"], None)

    assert gate(t=-1) == INVALID and gate(e=0) == INVALID and gate(k=0) == INVALID and gate(k=9) == INVALID
    assert gate(dt=2) == INVALID and gate(s=2) == INVALID
    assert gate(e=1025) == SHAPE and gate(e=64, k=33) == SHAPE and gate(t=1 << 31) == SHAPE
    assert gate(l=None) == INVALID and gate(ids=None) == INVALID and gate(w=ODD) == MISALIGNED and gate(b=ODD) == MISALIGNED
    assert gate(t=0, l=None) == fme.OK
    assert lib.moe_gate_backward(P, 1, P, None, 4, 8, 2, 0, 1, 1.0, P, None, None) == INVALID
    assert lib.moe_gate_backward(P, 1, P, P, 4, 8, 9, 0, 1, 1.0, P, None, None) == INVALID
    assert lib.moe_gate_backward(P, 1, ODD, P, 4, 8, 2, 0, 1, 1.0, P, None, None) == MISALIGNED

    def balance(**kw):
        a = dict(l=P, t=100, e=8, k=2, so=None, s=1, loss=P, c=P, n=P, ws=P, wb=1 << 20)
        a.update(kw)
        return lib.moe_balance_loss(a["l"], 1, P, a["t"], a["e"], a["k"], 0, 1.0, a["so"], a["s"], None, a["loss"], a["c"],
                                    a["n"], a["ws"], a["wb"], None, None)

    assert balance(s=0) == INVALID and balance(s=2) == INVALID  # two sequences need offsets
    assert balance(so=P, s=1 << 25) == SHAPE
    assert balance(ws=None) == INVALID and balance(loss=None) == INVALID and balance(c=None) == INVALID
    assert balance(wb=fme.balance_workspace_bytes(100, 1, 8) - 1) == INVALID
    assert balance(ws=ODD) == MISALIGNED
    assert fme.balance_workspace_bytes(-1, 1, 8) == 0 and fme.balance_workspace_bytes(0, 1, 8) >= 16
    assert lib.moe_balance_loss_backward(P, 1, P, P, P, 100, 8, 2, 0, 1.0, None, 2, None, P, 0, None) == INVALID
    assert lib.moe_balance_loss_backward(P, 1, P, P, None, 100, 8, 2, 0, 1.0, None, 1, None, P, 0, None) == INVALID


def test_combine_backward(lib):
    f = lib.moe_combine_backward
    assert f(P, P, 8, P, P, -1, 2, 64, P, P, None, None) == INVALID
    assert f(P, P, 8, P, P, 4, 0, 64, P, P, None, None) == INVALID
    assert f(P, P, 8, P, P, 4, 65, 64, P, P, None, None) == INVALID
    assert f(P, P, 8, P, P, 4, 2, 60, P, P, None, None) == SHAPE
    assert f(P, P, 8, P, P, 1 << 31, 2, 64, P, P, None, None) == SHAPE
    assert f(P, P, 8, None, P, 4, 2, 64, P, P, None, None) == INVALID
    assert f(ODD, P, 8, P, P, 4, 2, 64, P, P, None, None) == MISALIGNED
    assert f(None, None, 8, None, None, 0, 2, 64, None, None, None, None) == fme.OK


def test_binding_refuses_other_tensors():
    """Wrong type, place, shape or order: a ValueError that names the argument."""
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a contiguous CUDA tensor"):
        fme.quantize_fp8_block128(x)
    with pytest.raises(ValueError, match="w must be"):
        fme.quantize_fp8_block128_weights(torch.zeros((2, 16, 16)))
    with pytest.raises(ValueError, match="logits must be bfloat16 or float32"):
        fme.moe_gate(torch.zeros((4, 8), dtype=torch.float16), 2)
    with pytest.raises(ValueError, match="logits must be a contiguous CUDA tensor"):
        fme.moe_gate(torch.zeros((4, 8)), 2)
    with pytest.raises(ValueError, match="d_out must be"):
        fme.moe_combine_backward(x, x, torch.zeros((4, 1), dtype=torch.int32), torch.zeros((4, 1)))


@pytest.mark.gpu
def test_binding_refusals_on_the_gpu():
    import torch

    fme.ensure_built()
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    l = torch.zeros((4, 8), device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ValueError, match="not contiguous"):
        fme.quantize_fp8_block128(x[:, :128])
    with pytest.raises(ValueError, match="src_row must be"):
        fme.quantize_fp8_block128(x, src_row=i32(7), top_k=2)
    with pytest.raises(ValueError, match="ROWWISE only"):
        fme.quantize_fp8_block128(x, fme.COLWISE, src_row=i32(4))
    with pytest.raises(ValueError, match="offsets must be"):
        fme.quantize_fp8_block128(x, fme.COLWISE, torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="score must be"):
        fme.moe_gate(l, 2, score="tanh")
    with pytest.raises(ValueError, match="bias must be"):
        fme.moe_gate(l, 2, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError, match="token_mask must be"):
        fme.moe_balance_loss(l, ids, token_mask=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError, match="accumulate needs"):
        fme.moe_balance_loss_backward(l, i32(8).reshape(1, 8), i32(1), torch.zeros(1, device="cuda"), 2, accumulate=True)
    with pytest.raises(fme.FmeError) as e:
        fme.moe_gate(l, 9)
    assert e.value.status == INVALID
    q, s = fme.quantize_fp8_block128(x)
    w, sw = fme.quantize_fp8_block128_weights(torch.zeros((2, 128, 256), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="a_scale must be"):
        fme.grouped_gemm_fwd_fp8_block128(q, s.t().contiguous(), w, sw, i32(3))
    with pytest.raises(ValueError, match="offsets must be"):
        fme.grouped_gemm_fwd_fp8_block128(q, s, w, sw, i32(2))
    with pytest.raises(ValueError, match="accumulate into"):
        fme.grouped_gemm_wgrad_fp8_block128(q, s, q, s, i32(2), accumulate=True)
    torch.cuda.synchronize()
