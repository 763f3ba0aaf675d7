"""CPU: the 8-bit operators' binding, as far as it goes without a GPU."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from dac_vocoder_decode_gb300 import binding as V
from dac_vocoder_decode_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def test_cache_tensors_are_not_exchanged():
    """The cache keeps its tensors' addresses, so another tensor in their place is refused."""
    cache = V.KVCacheFP8.empty(3, 2, 64, device="cpu")
    larger = V.KVCacheFP8.empty(5, 2, 64, device="cpu")
    for name in ("k", "v", "k_scale", "v_scale", "pages", "kv_heads", "head_dim"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(larger, name))
    assert cache.k.data_ptr() == cache._args[0] and cache.v.data_ptr() == cache._args[1]
    assert cache.k_scale.data_ptr() == cache._args[2] and cache.v_scale.data_ptr() == cache._args[3]
    cache.k_scale[1, 1] = 2  # in place is the way
    assert cache.k_scale[1, 1] == 2 and (cache.pages, cache.kv_heads, cache.head_dim) == (3, 2, 64)


def test_a_binding_that_does_not_load_leaves_the_python_way(tmp_path, monkeypatch):
    bad = tmp_path / "lm_torch.so"
    bad.write_text("not a library")
    monkeypatch.setattr(B, "torch_lib", lambda: str(bad))
    monkeypatch.setattr(V._LM, "ready", False)
    monkeypatch.setattr(V._LM, "fast", None)
    with pytest.warns(RuntimeWarning, match="does not load"):
        V._lm_setup()
    assert V._LM.fast is None and V._LM.ready
    cache = V.KVCacheFP8.empty(3, 2, 64, device="cpu")
    assert (cache.pages, cache.kv_heads, cache.head_dim, cache.device_index) == (3, 2, 64, -1)
    with pytest.raises(V.VocoderError):
        V.rows_fp8(torch.zeros(4, 8), V.VOC_LM_NONE)
