"""The decode example notices a cache that its compaction left with holes."""
import importlib.util
import os

import pytest

import block_scaled_quantized_tcgen05_gb300 as q

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("steps", [12, 24])
def test_a_compaction_that_moves_nothing_is_noticed(monkeypatch, steps):
    from block_scaled_quantized_tcgen05_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("decode_serving", os.path.join(ROOT, "examples", "decode_serving.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    monkeypatch.setattr(q, "qgemm_kv_compact", lambda *a, **k: None)
    with pytest.raises(RuntimeError, match="not compact"):
        m.main(steps=steps, say=lambda line: None)
