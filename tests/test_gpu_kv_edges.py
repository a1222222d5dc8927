"""The cache and attention calls at values and indices that ordinary data does not have: page
numbers that a kernel might take for a mark of its own, weights far below the largest."""
import numpy as np
import pytest
import torch

from oracle import kv as okv
from nvfp4_expert_ffn_b200 import binding as B
from test_gpu_kv_cache import Case, _attn_bounds, _bf16, _gpu, _np

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- page numbers

@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("n", [1, 60])
@pytest.mark.parametrize("bad", [-1, -2, -3, -2 ** 31, 2 ** 31 - 1])
def test_any_page_number_outside_the_cache_counts_as_zeros(n, bad, page):
    """In both kernels, with one or two pages to a stage of 32 keys, for the first, a middle and the
    last page of a context. The calls before leave rows with NaN scales where the keys would lie."""
    c = Case(128, 1, 4, page, [n], [7 * page + 5], 20 + page)
    c.run(causal=False)
    for at in (0, 3, 7):
        table = c.args[2].clone()
        table[0, at] = bad
        args, c.args = c.args, (c.args[0], c.args[1], table)
        out, lse = c.run(causal=False)
        c.args = args
        assert B.moe_get_device_status() == B.MOE_ERR_INVALID_ARG, (bad, at)
        k, v = c.cache.read("k", c.slots[0]), c.cache.read("v", c.slots[0])
        for rows in (k, v):
            rows[at * page:(at + 1) * page] = 0.0
        for t in {0, n - 1}:
            ref, e, w, s = okv.attention(c.q[t:t + 1], k, v, c.D ** -0.5, False)
            tol, tol_e = _attn_bounds(ref, w, s, e, len(k), np.abs(v).max(), c.D)
            assert np.all(np.abs(_np(out)[t] - ref[0]) <= tol[0]) and np.all(np.abs(lse.cpu().numpy()[t] - e[0]) <= tol_e[0])


# ---------------------------------------------------------------- weights far below the largest

@pytest.mark.parametrize("D,Hkv,G", [(64, 1, 2), (128, 2, 4), (256, 1, 3)])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("gap", [9.0, 14.0, 17.0, 18.2])
def test_many_small_weights_beside_a_dominant_one(D, Hkv, G, n, gap):
    """Every 16th key leads the others by `gap` and has a value of zero (an attention sink), so the
    output is what the others contribute, 10^-4 to 10^-8 of the weight each. A weight is held in float16
    relative to a maximum that weighs 2^7 at least: 2^-11 relative, 2^-25 absolute below 2^-14, which
    is 2^-32 of the largest weight."""
    ctx = 333
    c = Case(D, Hkv, G, 16, [n], [ctx], D + n)
    sink = np.arange(ctx) % 16 == 5
    k, v = np.zeros((ctx, Hkv, D)), _bf16(c.rng, ctx, Hkv, D, spread=0.2)
    c.q[:] = 1.0
    k[sink] = gap / np.sqrt(D)  # the score of a query of ones: D k / sqrt(D)
    v[sink] = 0.0
    v = np.abs(v)
    for name, rows in (("k", k), ("v", v)):
        c.cache.write(name, okv.to_bf16(rows), c.slots[0])
    g = c.cache
    c.gcache = B.KVCache(_gpu(g.codes["k"]), _gpu(g.scales["k"]), _gpu(g.codes["v"]), _gpu(g.scales["v"]), c.gcache.k_ts, c.gcache.v_ts)
    kk, vv = g.read("k", c.slots[0]), g.read("v", c.slots[0])
    assert np.all(kk[~sink] == 0) and np.all(vv[sink] == 0) and np.abs(np.sqrt(D) * kk[sink].mean(axis=-1) / gap - 1).max() < 0.1
    ref, e, w, s = okv.attention(c.q[:1], kk, vv, D ** -0.5, False)
    # a float16 weight is off by 2^-25 at most where it is subnormal, the sum of a part's weights is
    # 2^7 at least, and the exponential's rounding and the scores' error dS move each by its share
    dS = s * (D * 2.0 ** -23 + 2.0 ** -21) + 2.0 ** -21
    tol = (2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * dS[..., None] + ctx * 2.0 ** -24) * w
           + ctx * 2.0 ** -32 / max(1, sink.sum() / 2) * np.abs(vv).max()) * 1.01
    out, lse = c.run(causal=False)
    assert np.all(np.abs(_np(out) - ref) <= tol), (np.abs(_np(out) - ref) / ref).max()
    assert np.all(np.abs(lse.cpu().numpy() - e) <= dS + ctx * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(e)))


# ---------------------------------------------------------------- copies that land in another order

@pytest.mark.parametrize("D,G,n,ctx", [(128, 4, 40, 20011), (128, 4, 25, 40000), (64, 3, 100, 20011), (256, 4, 40, 20011)])
def test_a_split_context_gives_the_same_bits_whatever_lies_in_the_caches(D, G, n, ctx):
    """Blocks of one to four key tiles, started on keys that are in L2 and on keys that a large write has
    driven out of it, so that a block's first copies land late and in any order."""
    c = Case(D, 1, G, 64, [n], [ctx], D + n)
    q = _gpu(c.q).bfloat16()
    want, lse = c.run(q=q)
    sweep = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(60):
        if i % 2:
            sweep.fill_(i)
        out, e = c.run(q=q)
        assert torch.equal(out, want) and torch.equal(e, lse), i
    assert B.moe_get_device_status() == 0
