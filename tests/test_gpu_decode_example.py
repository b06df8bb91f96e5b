"""The decode loop of examples/decode_serving.py: all its calls together, checked against a plain softmax."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_loop():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from block_scaled_quantized_tcgen05_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("decode_serving", os.path.join(ROOT, "examples", "decode_serving.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    lines = []
    assert m.main(steps=24, say=lines.append) < 0.1
    assert len(lines) == 1
