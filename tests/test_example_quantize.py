"""The example's 4-bit quantization on the CPU: weights that are all zero, or zero in a group, stay
zero, and the others come back within half a step of E2M1 (a quarter of the group's scale up to 2,
a fifth of the value above) plus the rounding of the scale, 2^-4 of the value."""
import importlib.util
import os

import torch

from conftest import ROOT


def test_quantize_keeps_zeros_and_values():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    w = torch.randn(4, 24, 64, generator=torch.Generator().manual_seed(1))
    w[1] = 0                                    # an expert that is not used
    w[2, 5] = 0
    w[2, 6, 16:32] = 0
    w[3] *= 1e-20
    codes, scales, factor = example.quantize(w)
    got = example.dequantize(codes, scales, factor)
    assert bool(torch.isfinite(got).all()) and bool(torch.isfinite(factor).all())
    assert not got[w == 0].any()
    group = scales.view(torch.float8_e4m3fn).float() * factor[:, None, None]
    step = torch.maximum(group.repeat_interleave(16, -1) / 4, w.abs() / 5)
    assert bool(((got - w).abs() <= step + w.abs() / 16 + 1e-30).all())
