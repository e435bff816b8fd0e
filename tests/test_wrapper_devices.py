"""The torch wrappers refuse tensors that are not in the GPU's memory, whatever the
stream, before they call the library (no GPU)."""
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc

BF, I8, F32 = torch.bfloat16, torch.int8, torch.float32


def z(*shape, dtype=BF, device="cpu"):
    return torch.zeros(shape, dtype=dtype, device=device)


OFFSETS = torch.zeros(3, dtype=torch.int32)
CALLS = {
    "gemm": lambda s: ttc.gemm(z(4, 8), z(8, 5), out=z(4, 5), stream=s),
    "gemm_grouped": lambda s: ttc.gemm_grouped(z(4, 8), z(2, 8, 5), OFFSETS, z(4, 5), stream=s),
    "gemm_grouped_wgrad": lambda s: ttc.gemm_grouped_wgrad(z(4, 8), z(4, 5), OFFSETS, out=z(2, 8, 5), stream=s),
    "quantize_rows": lambda s: ttc.quantize_rows(z(4, 8), z(4, 8, dtype=I8), z(4, dtype=F32), stream=s),
    "gemm_i8_scaled": lambda s: ttc.gemm_i8_scaled(z(4, 8, dtype=I8), z(4, dtype=F32), z(5, 8, dtype=I8), z(5, dtype=F32),
                                                   z(4, 5), stream=s),
}


@pytest.fixture(autouse=True)
def no_calls(monkeypatch):
    def load():
        raise AssertionError("the library was called")

    monkeypatch.setattr(ttc, "load", load)


@pytest.mark.parametrize("stream", [None, 0, 1 << 40])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_host_tensors(name, stream):
    with pytest.raises(ValueError):
        CALLS[name](stream)


# a device without memory stands for the GPU
@pytest.mark.parametrize("kw", [dict(b=z(8, 5)), dict(c=z(4, 5), beta=1.0), dict(out=z(4, 5)), dict(bias=z(5, dtype=F32))])
def test_gemm_operands_on_other_devices(kw):
    args = dict(a=z(4, 8, device="meta"), b=z(8, 5, device="meta"), out=z(4, 5, device="meta"))
    args.update(kw)
    with pytest.raises(ValueError, match="must be on meta"):
        ttc.gemm(**args, stream=0)


@pytest.mark.parametrize("workspace", [z(64, dtype=torch.uint8), z(1, dtype=torch.uint8, device="meta").expand(1 << 20)])
def test_workspaces(workspace):
    m = lambda *shape, dtype: z(*shape, dtype=dtype, device="meta")
    with pytest.raises(ValueError, match="workspace"):
        ttc.gemm_i8_scaled(m(4, 8, dtype=I8), m(4, dtype=F32), m(5, 8, dtype=I8), m(5, dtype=F32), m(4, 5, dtype=BF),
                           workspace=workspace, stream=0)
