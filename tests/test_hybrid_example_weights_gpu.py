"""The serving example's 8-bit weights: a channel of zeros gives zeros."""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_channel_of_zeros():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd
    spec = importlib.util.spec_from_file_location("hybrid_decode_w", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    ex = importlib.util.module_from_spec(spec)
    sys.modules["hybrid_decode_w"] = ex
    spec.loader.exec_module(ex)
    w = torch.randn(40, 64, generator=torch.Generator().manual_seed(1)).cuda()
    w[7] = 0
    packed, scale = ex.quantized(w)
    whole = packed.view(1, 4, 128, 16).transpose(1, 2).reshape(128, 64)
    assert scale[7] == 0 and not whole[7].any()
    steps = (w / (w.abs().amax(1, keepdim=True) / 127).clamp_min(1e-30)).round()
    assert torch.equal(whole[:40].float(), steps)
    y = ssd.q8_matmul(torch.ones(3, 64, dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda"), packed, scale, dtype=torch.float32)
    assert not y[:, 7].any() and torch.isfinite(y).all()
