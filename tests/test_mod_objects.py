"""Rope and ScoreMod (CPU): what a call uses is what the object shows."""
import pytest
import torch

import paged_kv_cache_kvc_gb300 as kvc


def test_what_they_hold_is_what_a_call_takes():
    f, w, a, d = torch.ones(8), torch.ones(64), torch.ones(4), torch.zeros(3, dtype=torch.int32)
    rope = kvc.Rope(f, interleaved=True, q_norm=w, eps=1e-5)
    assert rope.args == (16, 1, f, w, None, 1e-5) and rope.inv_freq is f and rope.q_norm is w and rope.k_norm is None
    mod = kvc.ScoreMod(softcap=30, window=5, sink=2, alibi=a, doc_start=d)
    assert mod.args[:4] == (30.0, 5, 2, 0) and mod.alibi is a and mod.doc_start is d


@pytest.mark.parametrize("name", ["inv_freq", "q_norm", "k_norm", "eps", "interleaved"])
def test_a_rope_cannot_be_changed(name):
    """An attribute set later would change nothing in the calls, so it cannot be set."""
    with pytest.raises(AttributeError):
        setattr(kvc.Rope(torch.ones(8)), name, torch.ones(8))


@pytest.mark.parametrize("name", ["alibi", "doc_start", "softcap", "window", "sink", "prefix"])
def test_a_score_mod_cannot_be_changed(name):
    with pytest.raises(AttributeError):
        setattr(kvc.ScoreMod(doc_start=torch.zeros(3, dtype=torch.int32)), name, 5)
