"""The torch wrappers work on the device of their operands, whatever the current one is: the
library, which launches on the current device, is called with theirs (no GPU)."""
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc

BF, I8, I32, F32, E4 = torch.bfloat16, torch.int8, torch.int32, torch.float32, torch.float8_e4m3fn


def z(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")  # a device without memory stands for the operands'


CALLS = {
    "ttc_gemm": lambda: ttc.gemm(z(4, 8), z(8, 5), out=z(4, 5)),
    "ttc_gemm_grouped": lambda: ttc.gemm_grouped(z(4, 8), z(2, 8, 5), z(3, dtype=I32), z(4, 5)),
    "ttc_gemm_grouped_wgrad": lambda: ttc.gemm_grouped_wgrad(z(4, 8), z(4, 5), z(3, dtype=I32), out=z(2, 8, 5)),
    "ttc_quantize_rows": lambda: ttc.quantize_rows(z(4, 8), z(4, 8, dtype=I8), z(4, dtype=F32)),
    "ttc_gemm_i8_scaled": lambda: ttc.gemm_i8_scaled(z(4, 8, dtype=I8), z(4, dtype=F32), z(5, 8, dtype=I8), z(5, dtype=F32), z(4, 5)),
    "ttc_gemm_gated": lambda: ttc.gemm_gated(z(4, 8), z(8, 5), z(8, 5), z(4, 5)),
    "ttc_gemm_gated_grad": lambda: ttc.gemm_gated_grad(z(4, 8), z(8, 5), z(4, 10), z(4, 10)),
    "ttc_quantize_blocks": lambda: ttc.quantize_blocks(z(4, 8), z(4, 8, dtype=E4), z(4, 1, dtype=F32)),
    "ttc_gemm_f8_blocks": lambda: ttc.gemm_f8_blocks(z(4, 8, dtype=E4), z(4, 1, dtype=F32), z(5, 8, dtype=E4), z(5, 1, dtype=F32),
                                                     z(4, 5)),
}


class Devices:
    """Which device is current, and a library that notes it."""

    def __init__(self, current):
        self.current, self.seen = current, []

    def device(self, other):
        devices = self

        class Current:
            def __enter__(self):
                self.before, devices.current = devices.current, other.index

            def __exit__(self, *_):
                devices.current = self.before

        return Current()

    def __getattr__(self, name):
        if not name.startswith("ttc_"):
            raise AttributeError(name)

        def call(*args):
            self.seen.append((name, self.current))
            return 0

        return call


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("current", [3, None])  # another device; that of the operands (meta has no number)
def test_current_device(name, current, monkeypatch):
    devices = Devices(current)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: devices.current)
    monkeypatch.setattr(torch.cuda, "device", devices.device)
    monkeypatch.setattr(ttc, "load", lambda: devices)
    monkeypatch.setattr(ttc, "_stream_of", lambda stream, device: 0)
    CALLS[name]()
    assert devices.seen[-1] == (name, None) and all(d is None for _, d in devices.seen)
    assert devices.current == current
