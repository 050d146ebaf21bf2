"""Tensors of different devices, or of another than the current one, are refused by the FP8 block-128 and router calls
before any address is taken.  The host-side tests use tensors that have a shape, a type and a device but no memory."""
import pytest
import torch

import fp8_moe_expert_gb300 as fme


class NoMemory(torch.Tensor):
    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError("a tensor without memory was used")


def at(device, shape, dtype):
    return torch.Tensor._make_wrapper_subclass(NoMemory, shape, dtype=dtype, device=f"cuda:{device}")


U8, F32, I32, BF16, BOOL = torch.uint8, torch.float32, torch.int32, torch.bfloat16, torch.bool

# call, its tensors in order (name, shape, type); keyword arguments have a "=" in front
CALLS = {
    "rows": (lambda *a, **k: fme.quantize_fp8_block128(*a, **k), [("x", (4, 128), BF16), ("=status", (1,), I32)]),
    "gathered rows": (lambda *a, **k: fme.quantize_fp8_block128(*a, top_k=2, **k),
                      [("x", (4, 128), BF16), ("=src_row", (8,), I32)]),
    "columns": (lambda *a, **k: fme.quantize_fp8_block128(a[0], fme.COLWISE, *a[1:], **k),
                [("x", (4, 128), BF16), ("offsets", (3,), I32)]),
    "both ways": (fme.quantize_fp8_block128_rowcol, [("x", (4, 128), BF16), ("=status", (1,), I32)]),
    "forward": (fme.grouped_gemm_fwd_fp8_block128,
                [("a_codes", (4, 256), U8), ("a_scale", (2, 4), F32), ("w_codes", (2, 128, 256), U8),
                 ("w_scale", (2, 1, 2), F32), ("offsets", (3,), I32), ("=status", (1,), I32)]),
    "dgrad": (fme.grouped_gemm_dgrad_fp8_block128,
              [("dy_codes", (4, 128), U8), ("dy_scale", (1, 4), F32), ("w_codes", (2, 128, 256), U8),
               ("w_scale", (2, 1, 2), F32), ("offsets", (3,), I32), ("=status", (1,), I32)]),
    "wgrad": (fme.grouped_gemm_wgrad_fp8_block128,
              [("dy_codes", (256, 128), U8), ("dy_scale", (2, 128), F32), ("x_codes", (256, 256), U8),
               ("x_scale", (2, 256), F32), ("padded_offsets", (3,), I32), ("=status", (1,), I32)]),
    "gate": (lambda *a, **k: fme.moe_gate(*a, 2, **k), [("logits", (4, 8), F32), ("=bias", (8,), F32)]),
    "gate gradient": (fme.moe_gate_backward, [("logits", (4, 8), F32), ("ids", (4, 2), I32), ("d_weights", (4, 2), F32),
                                              ("=status", (1,), I32)]),
    "balance": (fme.moe_balance_loss, [("logits", (4, 8), F32), ("ids", (4, 2), I32), ("=token_mask", (4,), BOOL)]),
    "balance of sequences": (fme.moe_balance_loss,
                             [("logits", (4, 8), F32), ("ids", (4, 2), I32), ("=seq_offsets", (3,), I32)]),
    "balance status": (fme.moe_balance_loss, [("logits", (4, 8), F32), ("ids", (4, 2), I32), ("=status", (1,), I32)]),
    "balance gradient": (lambda *a, **k: fme.moe_balance_loss_backward(*a, 2, **k),
                         [("logits", (4, 8), F32), ("counts", (1, 8), I32), ("seq_tokens", (1,), I32),
                          ("d_loss", (1,), F32)]),
    "combine gradient": (fme.moe_combine_backward,
                         [("d_out", (4, 64), BF16), ("y", (8, 64), BF16), ("row_of", (4, 2), I32),
                          ("weights", (4, 2), F32), ("=status", (1,), I32)]),
}


def arguments(spec, device_of):
    args, kwargs = [], {}
    for i, (name, shape, dtype) in enumerate(spec):
        t = at(device_of(i), shape, dtype)
        if name[0] == "=":
            kwargs[name[1:]] = t
        else:
            args.append(t)
    return args, kwargs


@pytest.mark.parametrize("what", list(CALLS))
def test_mixed_devices_are_refused(what):
    fme.ensure_built()
    call, spec = CALLS[what]
    for moved in range(1, len(spec)):
        args, kwargs = arguments(spec, lambda i: 1 if i == moved else 0)
        with pytest.raises(ValueError, match=rf"{spec[moved][0].lstrip('=')} is on cuda:1, {spec[0][0]} on cuda:0"):
            call(*args, **kwargs)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["rows", "both ways", "forward", "dgrad", "wgrad", "gate gradient", "balance gradient",
                                  "combine gradient"])
def test_another_device_than_the_current_one_is_refused(what):
    fme.ensure_built()
    torch.cuda.init()
    call, spec = CALLS[what]
    spec = [s for s in spec if s[0] != "=status"]
    other = torch.cuda.current_device() + 1
    args, kwargs = arguments(spec, lambda i: other)
    with pytest.raises(ValueError, match=rf"{spec[0][0]} is on cuda:{other}, the current device is cuda:{other - 1}"):
        call(*args, **kwargs)


@pytest.mark.gpu
def test_outputs_of_another_device_are_refused():
    fme.ensure_built()
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda:0")
    with pytest.raises(ValueError, match="codes is on cuda:1, x on cuda:0"):
        fme.quantize_fp8_block128(x, codes=at(1, (4, 128), U8))
    l, ids = torch.zeros((4, 8), device="cuda:0"), torch.zeros((4, 2), dtype=torch.int32, device="cuda:0")
    with pytest.raises(ValueError, match="workspace is on cuda:1, logits on cuda:0"):
        fme.moe_balance_loss(l, ids, workspace=at(1, (1 << 16,), U8))
    with pytest.raises(ValueError, match="d_y is on cuda:1"):
        fme.moe_combine_backward(x, x, torch.arange(4, dtype=torch.int32, device="cuda:0").reshape(4, 1),
                                 torch.ones((4, 1), device="cuda:0"), d_y=at(1, (4, 128), BF16))
