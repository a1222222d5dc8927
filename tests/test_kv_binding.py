"""The descriptions of a cache and of a norm and rotation that the Python calls take (CPU only)."""
import ctypes
import dataclasses

import pytest
import torch

from nvfp4_expert_ffn_b200 import binding as B


def _prep_c(prep, D=64):
    return ctypes.cast(prep.ref(D, -1), ctypes.POINTER(B._PrepC)).contents


def _fields(c):
    return {name: getattr(c, name) for name, _ in c._fields_}


def test_a_replaced_prep_has_its_own_structure():
    w, w2, f = torch.ones(64), torch.ones(64), torch.ones(16)
    p = B.QKPrep(w, w, 1e-6, f)
    before = _fields(_prep_c(p))
    changes = dict(q_weight=(w2, "q_weight", w2.data_ptr()), k_weight=(None, "k_weight", None), eps=(1.0, "eps", 1.0),
                   inv_freq=(None, "rot_dim", 0), interleaved=(True, "interleaved", 1), rot_scale=(3.0, "rot_scale", 3.0))
    for name, (value, member, want) in changes.items():
        q = dataclasses.replace(p, **{name: value})
        got = _fields(_prep_c(q))
        assert got[member] == want and got[member] != before[member], name
        same = B.QKPrep(**{n.name: getattr(q, n.name) for n in dataclasses.fields(q) if n.init})
        assert _fields(_prep_c(same)) == got
    assert _fields(_prep_c(p)) == before  # and the first one is as it was
    again = dataclasses.replace(p)
    assert _fields(_prep_c(again)) == before and again.ref(64, -1) is not p.ref(64, -1)
    with pytest.raises(ValueError, match="q_weight"):  # the new object's tensors are checked too
        dataclasses.replace(p, q_weight=torch.ones(32)).ref(64, -1)


def test_a_replaced_cache_has_its_own_structure():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    c = B.KVCache(u8(3, 2, 16, 64), u8(3, 2, 16, 8), u8(3, 2, 16, 64), u8(3, 2, 16, 8), torch.ones(2), None)
    before = _fields(c._c)
    ts = torch.ones(2)
    d = dataclasses.replace(c, v_ts=ts)
    got = _fields(ctypes.cast(d.ref, ctypes.POINTER(B._CacheC)).contents)
    assert got["v_ts"] == ts.data_ptr() and _fields(c._c) == before and before["v_ts"] is None
    with pytest.raises(ValueError, match="k_scales"):
        dataclasses.replace(c, k_scales=u8(3, 2, 16, 4))
