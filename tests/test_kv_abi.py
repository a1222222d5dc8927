"""Refusals of the cache and attention calls: on the host, before any device call (CPU only)."""
import ctypes

import pytest
import torch

from nvfp4_expert_ffn_b200 import binding as B

OK, INV, SHAPE, CUDA, WS = 0, 1, 2, 3, 5
P = 0x10000
p = ctypes.c_void_p(P)


def _cache(n_pages=4, page=64, Hkv=2, D=128, ptrs=(P, P, P, P), ts=(P, P)):
    return B._CacheC(n_pages, page, Hkv, D, *ptrs, *ts)


def _prep(w=P, eps=1e-6, f=P, rot=64, inter=0, m=1.0):
    return B._PrepC(w, w, eps, f, rot, inter, m)


def _rope(T=4, Hq=4, Hkv=2, D=128, q=p, qs=512, k=p, ks=256, pos=p, prep=None, qo=p, ko=p):
    prep = _prep() if prep is None else prep
    return B.lib().moe_qk_norm_rope(q, qs, k, ks, T, Hq, Hkv, D, pos, ctypes.byref(prep), qo, ko, None)


def _append(T=4, Hq=4, q=p, qs=512, k=p, ks=256, v=p, vs=256, pos=p, slots=p, prep=None, cache=None, qo=p):
    prep = _prep() if prep is None else prep
    cache = _cache() if cache is None else cache
    return B.lib().nvfp4_kv_append(q, qs, k, ks, v, vs, T, Hq, pos, slots, ctypes.byref(prep), ctypes.byref(cache), qo, None)


def _read(n=4, slots=p, kind=0, k=p, v=p, cache=None):
    cache = _cache() if cache is None else cache
    return B.lib().nvfp4_kv_read(ctypes.byref(cache), slots, n, kind, k, v, None)


def _attn(T=4, Hq=4, q=p, qs=512, cu=p, ctx=p, table=p, n=2, pages=3, max_q=4, cache=None, scale=0.1, out=p, lse=p, ws=p,
          ws_bytes=1 << 40):
    cache = _cache() if cache is None else cache
    return B.lib().nvfp4_kv_attention(q, qs, T, Hq, cu, ctx, table, n, pages, max_q, ctypes.byref(cache), scale, 1, out, lse,
                                      ws, ws_bytes, None)


def test_caches_that_are_refused():
    odd = ctypes.c_void_p(P + 8)
    for cache, want in ((_cache(D=96), SHAPE), (_cache(page=48), SHAPE), (_cache(page=8), SHAPE), (_cache(page=2048), SHAPE),
                        (_cache(n_pages=0), INV), (_cache(Hkv=0), INV), (_cache(n_pages=1 << 30), SHAPE),
                        (_cache(ptrs=(P, P, None, P)), INV), (_cache(ptrs=(P, P + 8, P, P)), INV), (_cache(ts=(P + 2, P)), INV)):
        assert _append(cache=cache, ks=4096, vs=4096, qs=4096) == want
        assert _read(cache=cache) == want
        assert _attn(cache=cache, qs=4096) == want
    assert B.lib().nvfp4_kv_append(p, 512, p, 256, p, 256, 4, 4, p, p, ctypes.byref(_prep()), None, p, None) == INV
    assert odd.value % 16


@pytest.mark.parametrize("call", [_rope, _append])
def test_norm_rope_and_append_refusals(call):
    assert call(T=-1) == INV and call(Hq=-1) == INV
    assert call(Hq=2000, qs=1 << 20) == SHAPE
    assert call(prep=_prep(rot=24)) == SHAPE and call(prep=_prep(rot=256)) == SHAPE and call(prep=_prep(rot=-16)) == SHAPE
    assert call(prep=_prep(f=None)) == INV and call(pos=None) == INV
    assert call(prep=_prep(eps=-1.0)) == INV and call(prep=_prep(eps=float("nan"))) == INV
    assert call(prep=_prep(w=P + 2)) == INV and call(pos=ctypes.c_void_p(P + 1)) == INV
    assert call(q=None) == INV and call(k=None) == INV
    assert call(q=ctypes.c_void_p(P + 8)) == INV and call(k=ctypes.c_void_p(P + 2)) == INV
    assert call(qs=504) == INV and call(qs=516) == INV and call(ks=255) == INV  # too small, not a multiple of 8
    assert call(qo=None) == INV and call(qo=ctypes.c_void_p(P + 8)) == INV
    assert call(T=0, q=None, k=None, pos=None) == OK


def test_more_refusals():
    assert _rope(D=100) == SHAPE and _rope(ko=None) == INV and _rope(Hq=0, Hkv=0) == OK
    assert _append(v=None) == INV and _append(vs=100) == INV and _append(slots=None) == INV
    assert _append(slots=ctypes.c_void_p(P + 2)) == INV
    assert _read(n=-1) == INV and _read(kind=2) == INV and _read(slots=None) == INV and _read(k=None, v=None) == INV
    assert _read(k=ctypes.c_void_p(P + 4)) == INV and _read(n=0, slots=None) == OK
    assert _read(n=1 << 41) == SHAPE


def test_attention_refusals():
    assert _attn(T=-1) == INV and _attn(n=-1) == INV and _attn(pages=-1) == INV and _attn(max_q=-1) == INV
    assert _attn(Hq=3) == SHAPE and _attn(Hq=0) == SHAPE and _attn(Hq=2048, qs=1 << 20) == SHAPE
    assert _attn(n=70000) == SHAPE and _attn(T=1 << 30) == SHAPE
    assert _attn(scale=float("nan")) == INV and _attn(max_q=0) == INV
    assert _attn(q=None) == INV and _attn(qs=500) == INV and _attn(qs=256) == INV
    assert _attn(cu=None) == INV and _attn(ctx=None) == INV and _attn(table=None) == INV and _attn(out=None) == INV
    assert _attn(cu=ctypes.c_void_p(P + 2)) == INV and _attn(out=ctypes.c_void_p(P + 8)) == INV
    assert _attn(lse=ctypes.c_void_p(P + 1)) == INV
    assert _attn(T=0) == OK and _attn(n=0) == OK
    need = B.lib().nvfp4_kv_attention_workspace
    assert need(4, 2, 4, 4, 2, 128) > 0
    assert need(4, 2, 4, 5, 2, 128) == 0 and need(4, 2, 4, 4, 2, 96) == 0 and need(-1, 2, 4, 4, 2, 128) == 0


def test_attention_sizes_past_the_limits():
    """Key positions are 32-bit with room for a step past the end; the workspace size says so too."""
    assert _attn(pages=(1 << 26) + 1, cache=_cache(page=16)) == SHAPE
    assert _attn(pages=(1 << 20) + 1, cache=_cache(page=1024)) == SHAPE
    need = B.lib().nvfp4_kv_attention_workspace
    assert need(4, 65537, 4, 4, 2, 128) == 0 and need(4, 2, 4, 2048, 2, 128) == 0 and need(1 << 30, 2, 4, 4, 2, 128) == 0
    assert need(1 << 20, 65536, 1 << 20, 1024, 8, 64) > 0


def test_binding_checks_types_shapes_and_devices():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    c = B.KVCache(u8(3, 2, 16, 64), u8(3, 2, 16, 8), u8(3, 2, 16, 64), u8(3, 2, 16, 8), torch.ones(2), None)
    assert (c.n_pages, c.Hkv, c.page_size, c.D) == (3, 2, 16, 128)
    with pytest.raises(ValueError, match="k_scales"):
        B.KVCache(u8(3, 2, 16, 64), u8(3, 2, 16, 4), u8(3, 2, 16, 64), u8(3, 2, 16, 8))
    with pytest.raises(ValueError, match="v_ts"):
        B.KVCache(u8(3, 2, 16, 64), u8(3, 2, 16, 8), u8(3, 2, 16, 64), u8(3, 2, 16, 8), None, torch.ones(3))
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    prep = B.QKPrep()
    q, k = bf(5, 4, 128), bf(5, 2, 128)
    with pytest.raises(ValueError, match="CUDA"):  # all else is right: only the device is not
        B.nvfp4_kv_append(q, k, k, i32(5), i32(5), prep, c, torch.empty_like(q))
    with pytest.raises(ValueError, match="slots"):
        B.nvfp4_kv_append(q, k, k, i32(5), i32(4), prep, c, torch.empty_like(q))
    with pytest.raises(ValueError, match="slots"):
        B.nvfp4_kv_append(q, k, k, i32(5), i32(5).long(), prep, c, torch.empty_like(q))
    with pytest.raises(ValueError, match="contiguous heads"):
        B.moe_qk_norm_rope(bf(4, 5, 128).transpose(0, 1), None, i32(5), prep, q, None)
    with pytest.raises(ValueError, match="bf16"):
        B.moe_qk_norm_rope(q.float(), None, i32(5), prep, q, None)
    with pytest.raises(ValueError, match="q_weight"):
        B.moe_qk_norm_rope(q, None, i32(5), B.QKPrep(q_weight=torch.ones(64)), q, None)
    with pytest.raises(ValueError, match="k and v"):
        B.nvfp4_kv_append(None, k[:, :1], k[:, :1], i32(5), i32(5), prep, c, None)
    with pytest.raises(ValueError, match="k_out"):
        B.nvfp4_kv_read(c, i32(5), bf(5, 2, 64), None)
    with pytest.raises(ValueError, match="bf16 or float32"):
        B.nvfp4_kv_read(c, i32(5), bf(5, 2, 128).double(), None)
    with pytest.raises(ValueError, match="cu_q"):
        B.nvfp4_kv_attention(q, i32(2), i32(2), i32(2, 3), 5, c, 0.1, True, q, None, u8(1024))
    with pytest.raises(ValueError, match="heads of"):
        B.nvfp4_kv_attention(bf(5, 4, 64), i32(3), i32(2), i32(2, 3), 5, c, 0.1, True, q, None, u8(1024))
