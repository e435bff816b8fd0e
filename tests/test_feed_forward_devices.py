"""The gated and block-scaled fp8 wrappers refuse tensors that are not in the GPU's memory or not
on one device, and views whose rows overlap, before they call the library (no GPU)."""
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def z(*shape, dtype=BF, device="meta"):
    return torch.empty(shape, dtype=dtype, device=device)


def gated(device, **kw):
    args = dict(a=z(6, 8, device=device), b_gate=z(2, 8, 5, device=device), b_up=z(2, 8, 5, device=device), out=z(6, 5, device=device),
                offsets=z(3, dtype=torch.int32, device=device), pre=z(6, 10, device=device))
    args.update(kw)
    return ttc.gemm_gated, args


def grad(device, **kw):
    args = dict(a=z(6, 8, device=device), b=z(2, 8, 5, device=device), pre=z(6, 10, device=device), dpre=z(6, 10, device=device),
                out=z(6, 5, device=device), offsets=z(3, dtype=torch.int32, device=device))
    args.update(kw)
    return ttc.gemm_gated_grad, args


def quantize(device, **kw):
    args = dict(x=z(6, 200, device=device), out=z(6, 200, dtype=E4, device=device), scale=z(6, 2, dtype=F32, device=device))
    args.update(kw)
    return ttc.quantize_blocks, args


def f8(device, **kw):
    args = dict(a=z(6, 200, dtype=E4, device=device), scale_a=z(6, 2, dtype=F32, device=device), b=z(2, 5, 200, dtype=E4, device=device),
                scale_b=z(2, 5, 2, dtype=F32, device=device), out=z(6, 5, device=device), c=z(6, 5, device=device),
                bias=z(2, 5, dtype=F32, device=device), offsets=z(3, dtype=torch.int32, device=device))
    args.update(kw)
    return ttc.gemm_f8_blocks, args


CALLS = {"gated": gated, "grad": grad, "quantize": quantize, "f8": f8}


@pytest.fixture(autouse=True)
def no_calls(monkeypatch):
    def load():
        raise AssertionError("the library was called")

    monkeypatch.setattr(ttc, "load", load)


@pytest.mark.parametrize("stream", [None, 0, 1 << 40])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_host_tensors(name, stream):
    call, args = CALLS[name]("cpu")
    with pytest.raises(ValueError):
        call(**args, stream=stream)


# a device without memory stands for the GPU
@pytest.mark.parametrize("name,which", [(n, k) for n, c in sorted(CALLS.items()) for k in c("meta")[1] if k not in ("a", "x")])
def test_operands_on_other_devices(name, which):
    call, args = CALLS[name]("meta")
    args[which] = torch.empty(args[which].shape, dtype=args[which].dtype)
    with pytest.raises(ValueError, match="must be on meta"):
        call(**args, stream=0)


@pytest.mark.parametrize("name,which", [(n, k) for n, c in sorted(CALLS.items()) for k in c("meta")[1]
                                        if k not in ("offsets", "bias", "b", "b_gate", "b_up", "scale_b")])
def test_rows_that_overlap(name, which):
    call, args = CALLS[name]("meta")
    t = args[which]
    args[which] = torch.empty((1, t.shape[-1]), dtype=t.dtype, device="meta").expand(t.shape)
    with pytest.raises(ValueError):
        call(**args, stream=0)


@pytest.mark.parametrize("name,which,dtype", [("gated", "b_up", torch.float16), ("gated", "out", F32), ("gated", "pre", F32),
                                              ("grad", "pre", torch.float16), ("grad", "dpre", F32), ("grad", "out", torch.float16),
                                              ("quantize", "scale", BF), ("quantize", "out", torch.int8), ("f8", "scale_a", BF),
                                              ("f8", "scale_b", BF), ("f8", "c", F32), ("f8", "bias", BF), ("f8", "a", torch.int8),
                                              ("f8", "b", torch.int8), ("f8", "offsets", torch.int64)])
def test_types(name, which, dtype):
    call, args = CALLS[name]("meta")
    args[which] = torch.empty(args[which].shape, dtype=dtype, device="meta")
    with pytest.raises(ValueError):
        call(**args, stream=0)
