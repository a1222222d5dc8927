"""The cache and attention calls at values and indices that ordinary data does not have: page
numbers that a kernel might take for a mark of its own, weights far below the largest, infinities
and NaN in queries, keys and scales, scores of any size."""
import numpy as np
import pytest
import torch

from oracle import kv as okv
from oracle import nvfp4 as onv
from nvfp4_expert_ffn_b200 import binding as B
from test_gpu_kv_cache import Case, _attn_bounds, _bf16, _gpu, _np

pytestmark = pytest.mark.gpu

DEV = "cuda"


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


# ---------------------------------------------------------------- keys and queries that are not finite

@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (64, 64, True), (128, 32, False), (128, 96, True), (256, 0, False)])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T", [6, 700])
def test_infinities_and_nan_in_queries_and_keys(D, rot, inter, norm, T):
    """Where the formula gives NaN or an infinity so do both, and where it gives a number so do they:
    through a rotation without a norm an element that is not finite reaches its partner, through a
    norm an infinity makes zeros of its row's numbers and NaN makes all of it NaN."""
    rng = np.random.default_rng(D + rot + T)
    x = _bf16(rng, T, 5, D)
    odd = np.array([np.inf, -np.inf, np.nan, 3.0e38, -1e-39], np.float32)
    for h in range(1, 5):  # (head 0 stays ordinary)
        for _ in range(h - 1 or 1):
            x[np.arange(T), h, rng.integers(0, D, T)] = odd[rng.integers(0, 5, T)]
    x[::3, 4, 0], x[::3, 4, 1], x[1::3, 4, rot // 2] = np.inf, -np.inf, np.nan
    x = _np(_gpu(x).bfloat16())
    pos = rng.integers(0, 1 << 17, T).astype(np.int32)
    pos[::4] = 0
    f = (1e4 ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32)
    w = rng.uniform(0.5, 1.5, D).astype(np.float32) if norm else None
    wg = None if w is None else _gpu(w)
    prep = B.QKPrep(wg, wg, 1e-6, _gpu(f) if rot else None, inter, 1.0)
    xg = _gpu(x).bfloat16()
    bits = xg.view(torch.int16)
    bits[1::2][torch.isnan(xg[1::2])] = -63  # 0xFFC1: NaN with its sign set
    qo, ko = torch.empty_like(xg), torch.empty_like(xg)
    B.moe_qk_norm_rope(xg, xg, _gpu(pos), prep, qo, ko)
    with np.errstate(all="ignore"):
        ref = okv.norm_rope(x, pos, w, 1e-6, f if rot else None, inter, 1.0)
        fin = np.isfinite(ref) & (np.abs(ref) < 3.38e38)  # (the largest numbers may round up to an infinity)
        rms = np.where(np.isfinite(x), np.abs(x), 0).astype(np.float64).max(axis=-1, keepdims=True)
        pair = 2.0 ** -24 * (D / 16 + 16) * np.sqrt(2) * 1.5 * (np.sqrt(D) if norm else rms)  # as in test_norm_rope
        for got, err in ((qo, pair), (ko, 0.0)):
            got = _np(got).astype(np.float64)
            assert np.array_equal(np.isnan(got), np.isnan(ref))
            inf = np.isinf(ref)
            assert np.array_equal(got[inf], ref[inf]) and not np.isinf(got[np.isfinite(ref) & fin]).any()
            assert np.all((np.abs(got - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -23) + err + 1e-37)[fin])
    # and what the cache then holds is the quantiser's
    cache = B.KVCache.allocate(-(-T // 16), 16, 5, D)
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    B.nvfp4_kv_append(None, xg, xg, _gpu(pos), slots, prep, cache, None)
    for src, codes, scales in ((ko, cache.k_codes, cache.k_scales), (xg, cache.v_codes, cache.v_scales)):
        qc, qs = torch.empty(T * 5, D // 2, dtype=torch.uint8, device=DEV), torch.empty(T * 5, D // 16, dtype=torch.uint8, device=DEV)
        B.nvfp4_quantize_act(src.reshape(T * 5, D), qc, qs, torch.empty(1, device=DEV), torch.ones(1, device=DEV))
        for got, want in ((codes, qc), (scales, qs)):
            got = got.transpose(1, 2).reshape(-1, 5, got.shape[-1])[:T].reshape(T * 5, -1)
            assert torch.equal(got, want)
    assert B.moe_get_device_status() == 0


# ---------------------------------------------------------------- scales that are NaN

def test_a_scale_that_is_nan_reads_as_nan():
    """E4M3's 0x7F and 0xFF are NaN for the reader as they are for attention; a negative scale is a
    negative number."""
    cache = B.KVCache.allocate(1, 16, 2, 64)
    rng = np.random.default_rng(0)
    for t in (cache.k_codes, cache.v_codes):
        t.copy_(_gpu(rng.integers(0, 256, tuple(t.shape)).astype(np.uint8)))
    scales = rng.integers(0, 256, tuple(cache.k_scales.shape)).astype(np.uint8)
    scales.reshape(-1)[:4] = 0x7F, 0xFF, 0x7E, 0xFE
    cache.k_scales.copy_(_gpu(scales))
    cache.v_scales.copy_(_gpu(scales[:, :, ::-1].copy()))
    slots = torch.tensor(list(range(16)) + [-1], dtype=torch.int32, device=DEV)
    for dtype, eps in ((torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)):
        ko, vo = (torch.empty(17, 2, 64, dtype=dtype, device=DEV) for _ in range(2))
        B.nvfp4_kv_read(cache, slots, ko, vo)
        for got, codes, sc in ((ko, cache.k_codes, cache.k_scales), (vo, cache.v_codes, cache.v_scales)):
            ref = np.stack([onv.dequantize(codes[0, h].cpu().numpy(), sc[0, h].cpu().numpy(), 1.0) for h in range(2)], 1)
            assert np.isnan(ref).any()
            got = _np(got)
            assert np.array_equal(np.isnan(got[:16]), np.isnan(ref)) and not got[16].any()
            ok = ~np.isnan(ref)
            assert np.all(np.abs(got[:16][ok] - ref[ok]) <= np.abs(ref[ok]) * eps)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [2, 70])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_tensor_scales_that_are_not_finite_reach_every_query_that_sees_a_key(D, n, bad):
    """A NaN or infinite scale of a head's keys makes that head's rows NaN in both kernels (infinities of
    both signs are among an infinite key's products), one of its values leaves nothing finite in them;
    rows that see no key stay at 0 and -infinity, and the other head as it was."""
    c = Case(D, 2, 4, 16, [n, n], [60, n - 1], 31)
    want, lse0 = c.run()
    ts = {"k": c.gcache.k_ts, "v": c.gcache.v_ts}
    g = c.gcache
    for name in "kv":
        t = dict(ts)
        t[name] = t[name].clone()
        t[name][1] = bad
        c.gcache = B.KVCache(g.k_codes, g.k_scales, g.v_codes, g.v_scales, t["k"], t["v"])
        out, lse = c.run()
        assert torch.equal(out[:, :4], want[:, :4]) and torch.equal(lse[:, :4], lse0[:, :4])
        none = torch.isneginf(lse0[:, 4:])  # queries before the first key
        assert none[n].all() and int(none.sum()) == 4 * (1 + max(0, n - 60))
        assert not out[:, 4:][none].any() and torch.isneginf(lse[:, 4:][none]).all()
        seen = out[:, 4:][~none]
        if name == "k":
            assert torch.isnan(seen).all() and torch.isnan(lse[:, 4:][~none]).all()
        else:
            assert not torch.isfinite(seen).any() and torch.equal(lse, lse0)
            assert torch.isnan(seen).all() or bad == float("inf")
    assert B.moe_get_device_status() == 0


# ---------------------------------------------------------------- scores of any size

@pytest.mark.parametrize("D,Hkv,G", [(64, 1, 2), (128, 2, 4), (256, 1, 3)])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 22, 2.0 ** 26, 2.0 ** 29, 2.0 ** 40, 2.0 ** 90])
def test_scores_far_past_one_give_the_largest_keys_value(D, Hkv, G, n, size):
    """Scores up to 10^27: where the first key leads the second by more than the scores' float32
    error, the output is its value, rounded to bf16 after a weight rounded to float16; the others weigh
    e^-60 at most."""
    c = Case(D, Hkv, G, 16, [n, n], [300, 65], D + n, qscale=size)
    out, lse = c.run(causal=False)
    out, lse = _np(out), lse.cpu().numpy()
    clear = 0
    for b in range(2):
        k, v = c.cache.read("k", c.slots[b]), c.cache.read("v", c.slots[b])
        for t in range(c.cu[b], c.cu[b + 1]):
            for h in range(c.Hq):
                s = D ** -0.5 * (k[:, h // G] @ c.q[t, h].astype(np.float64))
                logit = D ** -0.5 * (np.abs(k[:, h // G]) @ np.abs(c.q[t, h].astype(np.float64))).max()
                dS = logit * (D * 2.0 ** -23 + 2.0 ** -21) + 2.0 ** -21
                assert np.isfinite(out[t, h]).all() and abs(lse[t, h] - s.max()) <= dS + 2.0 ** -22 * abs(s.max()) + np.log(len(k))
                first, second = np.sort(s)[:-3:-1]
                if first - second > 2 * dS + 60:
                    clear += 1
                    top = v[s.argmax(), h // G]
                    assert np.all(np.abs(out[t, h] - top) <= np.abs(top) * (2.0 ** -8 + 2.0 ** -10) + len(k) * np.exp(-60.0) * np.abs(v).max())
    assert clear >= 0.8 * 2 * n * c.Hq
    assert B.moe_get_device_status() == 0


# ---------------------------------------------------------------- offsets that do not ascend

def test_offsets_that_go_back_are_reported_and_stay_inside_the_workspace():
    """Offsets that name the same 2000 tokens 40 times make 1280 tiles of rows, nine times what a
    workspace of 2000 tokens lists: the rest is left out, the status says so, and what lies behind
    the workspace and the next call's results are as they were."""
    T, page = 2000, 16
    c = Case(64, 1, 4, page, [T], [T], 41)
    seqs = 80
    need = B.nvfp4_kv_attention_workspace(T, seqs, T, c.Hq, c.gcache)
    buf = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device=DEV)
    c.ws = buf[:need]
    good, lse = c.run()
    assert B.moe_get_device_status() == 0
    args = c.args
    c.args = (torch.tensor([0, T] * 40 + [0], dtype=torch.int32, device=DEV),
              torch.full((seqs,), 16, dtype=torch.int32, device=DEV), args[2].repeat(seqs, 1))
    c.run()
    assert B.moe_get_device_status() == B.MOE_ERR_INVALID_ARG
    assert torch.all(buf[need:] == 0xA5)
    c.args = args
    again, lse2 = c.run()
    assert B.moe_get_device_status() == 0
    assert torch.equal(again, good) and torch.equal(lse2, lse)


# ---------------------------------------------------------------- the smoke run

def test_the_smoke_run_launches_both_attention_kernels_and_both_writers(tmp_path):
    import json

    import __graft_entry__ as entry
    from torch.profiler import ProfilerActivity, profile
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        assert entry._smoke_attention(DEV) <= 5e-3
        torch.cuda.synchronize()
    p.export_chrome_trace(str(tmp_path / "trace.json"))
    runs = {(e["name"].split("<")[0].split("::")[-1], e["args"]["block"][0])
            for e in json.loads((tmp_path / "trace.json").read_text())["traceEvents"] if e.get("cat") == "kernel"}
    names = {n for n, _ in runs}
    for kernel in ("kv_attn_tc_kernel", "kv_attn_tc_join_kernel", "kv_attn_dec_kernel", "kv_attn_join_kernel"):
        assert kernel in names, runs
    # the writer of few tokens has blocks of eight warps, that of many blocks of four
    assert {b for n, b in runs if n == "qkv_prep_kernel"} == {128, 256}, runs
