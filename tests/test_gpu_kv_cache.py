"""Norm, rotation, the quantised cache write, the read back and attention over the NVFP4 cache,
against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import kv as okv
from nvfp4_expert_ffn_b200 import binding as B
from nvfp4_expert_ffn_b200 import layer as L

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def _bf16(rng, *shape, spread=1.0):
    """bf16 values as float32, rows of different size."""
    x = rng.standard_normal(shape) * np.exp2(rng.uniform(-spread, spread, shape[:-1] + (1,)))
    return okv.to_bf16(x)


def _np(t):
    return t.float().cpu().numpy()


def _attn_bounds(ref, weight, logit, lse, n_keys, vmax, D):
    """Largest error of out and lse. out: half a bf16 step; the weights' float16 rounding 2^-11 of
    sum p|v| (and 2^-25 absolute per key where they are subnormal); the scores' error dS, which
    moves every weight by dS, twice (numerator and sum). dS: float32 accumulation over D products
    of at most `logit` in sum, at 2^-23 a step on the tensor core, the factor's and the
    exponential's roundings (2^-21 of the score's size, 2^-22)."""
    dS = logit * (D * 2.0 ** -23 + 2.0 ** -21) + 2.0 ** -21
    out = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * dS[..., None] + n_keys * 2.0 ** -24) * weight + n_keys * 2.0 ** -25 * vmax
    return out * 1.01 + 1e-30, dS + n_keys * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))


# ---------------------------------------------------------------- norm and rotation

@pytest.mark.parametrize("D,Hq,Hkv,rot,inter", [(64, 3, 1, 64, False), (64, 14, 2, 32, True), (128, 4, 4, 128, True),
                                                (128, 7, 1, 96, False), (128, 2, 3, 0, False), (256, 16, 2, 64, False),
                                                (256, 5, 5, 256, True), (256, 1, 1, 16, False)])
@pytest.mark.parametrize("T", [1, 7, 1300])
def test_norm_rope(D, Hq, Hkv, rot, inter, T):
    rng = np.random.default_rng(D + rot + T)
    q, k = _bf16(rng, T, Hq, D, spread=6), _bf16(rng, T, Hkv, D, spread=6)
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    qw, kw = rng.uniform(0.5, 1.5, D).astype(np.float32), rng.uniform(-1, 1, D).astype(np.float32)
    f = (1e6 ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32)
    m = 1.2079
    prep = B.QKPrep(_gpu(qw), _gpu(kw), 1e-5, _gpu(f) if rot else None, inter, m)
    fused = torch.cat((_gpu(q.reshape(T, -1)), _gpu(k.reshape(T, -1))), 1).bfloat16()  # strided rows
    qv, kv = fused[:, :Hq * D].unflatten(1, (Hq, D)), fused[:, Hq * D:].unflatten(1, (Hkv, D))
    qo, ko = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
    B.moe_qk_norm_rope(qv, kv, _gpu(pos), prep, qo, ko)
    for got, x, w, steps in ((qo, q, qw, 8), (ko, k, kw, 0)):
        ref = okv.norm_rope(x, pos, w, 1e-5, f if rot else None, inter, m)
        # keys are float64 all the way to the roundings: half a bf16 step and half a float32 step.
        # Queries are float32: the factor (a sum of D squares, D / 8 in a row, then log2 of the lanes:
        # at most 13 steps; divide, add, root, reciprocal), two products and a sum of two rotated
        # terms, so D / 16 + 8 steps of 2^-24 of the pair's size times m
        pair = 0.0 if steps == 0 else 2.0 ** -24 * (D / 16 + 16) * m * np.sqrt(2) * np.abs(
            okv.norm_rope(np.abs(x), pos, np.abs(w), 1e-5)).max(axis=-1, keepdims=True)
        assert np.all(np.abs(_np(got) - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -23) + pair + 1e-37)
    # in place, from contiguous rows, one side at a time
    qc, kc = qv.contiguous(), kv.contiguous()
    B.moe_qk_norm_rope(qc, None, _gpu(pos), prep, qc, None)
    B.moe_qk_norm_rope(None, kc, _gpu(pos), prep, None, kc)
    assert torch.equal(qc, qo) and torch.equal(kc, ko)


def test_norm_rope_without_norm_or_rotation_copies():
    x = _gpu(_bf16(np.random.default_rng(0), 9, 4, 64)).bfloat16()
    out = torch.empty_like(x)
    B.moe_qk_norm_rope(x, None, torch.zeros(9, dtype=torch.int32, device=DEV), B.QKPrep(), out, None)
    assert torch.equal(out, x)


# ---------------------------------------------------------------- write and read

def _append_case(D, Hkv, page, T, seed, n_pages=None, Hq=4, ts=True):
    rng = np.random.default_rng(seed)
    n_pages = n_pages or -(-T // page) + 3
    kts = rng.uniform(0.8, 1.2, Hkv).astype(np.float32) * 5 / 2688 if ts else None
    vts = rng.uniform(0.8, 1.2, Hkv).astype(np.float32) * 5 / 2688 if ts else None
    slots = rng.permutation(n_pages * page)[:T].astype(np.int32)
    slots[rng.random(T) < 0.1] = -1
    return dict(rng=rng, n_pages=n_pages, kts=kts, vts=vts, slots=slots, q=_bf16(rng, T, Hq, D), k=_bf16(rng, T, Hkv, D, spread=4),
                v=_bf16(rng, T, Hkv, D, spread=4), pos=rng.integers(0, 50000, T).astype(np.int32),
                w=rng.uniform(0.5, 1.5, D).astype(np.float32), f=(1e4 ** (-np.arange(16) / 16)).astype(np.float32))


@pytest.mark.parametrize("D,Hkv,page,T,ts", [(64, 1, 16, 1, True), (64, 8, 16, 77, True), (128, 3, 32, 200, True),
                                             (128, 8, 1024, 33, False), (256, 2, 64, 1250, True), (256, 1, 128, 9, False)])
def test_append_writes_what_the_quantiser_gives_and_reads_back(D, Hkv, page, T, ts):
    c = _append_case(D, Hkv, page, T, D + T, ts=ts)
    cache = B.KVCache.allocate(c["n_pages"], page, Hkv, D, _gpu(c["kts"]) if ts else None, _gpu(c["vts"]) if ts else None)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(0x5A)  # rows that no slot names stay as they were
    prep = B.QKPrep(_gpu(c["w"]), _gpu(c["w"]), 1e-6, _gpu(c["f"]))
    k, v, q = (_gpu(c[n]).bfloat16() for n in "kvq")
    qo = torch.empty_like(q)
    B.nvfp4_kv_append(q, k, v, _gpu(c["pos"]), _gpu(c["slots"]), prep, cache, qo)
    # the same rows by the separate calls
    qn, kn = torch.empty_like(q), torch.empty_like(k)
    B.moe_qk_norm_rope(q, k, _gpu(c["pos"]), prep, qn, kn)
    assert torch.equal(qn, qo)
    oc = okv.Cache(c["n_pages"], page, Hkv, D, c["kts"], c["vts"])
    for a in (oc.codes, oc.scales):
        for n in "kv":
            a[n].fill(0x5A)
    oc.write("k", _np(kn), c["slots"])
    oc.write("v", c["v"], c["slots"])
    for n, codes, scales in (("k", cache.k_codes, cache.k_scales), ("v", cache.v_codes, cache.v_scales)):
        assert np.array_equal(codes.cpu().numpy(), oc.codes[n]) and np.array_equal(scales.cpu().numpy(), oc.scales[n])
    # read back: every written row, some twice, and padding
    live = c["slots"][c["slots"] >= 0]
    at = np.concatenate([live, live[:3], [-1, -7]]).astype(np.int32)
    for dtype, eps in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8 + 2.0 ** -23)):
        ko, vo = (torch.full((len(at), Hkv, D), 7.0, dtype=dtype, device=DEV) for _ in range(2))
        B.nvfp4_kv_read(cache, _gpu(at), ko, vo)
        for n, got in (("k", ko), ("v", vo)):
            ref = oc.read(n, np.maximum(at, 0)) * (at >= 0)[:, None, None]
            assert np.all(np.abs(_np(got) - ref) <= np.abs(ref) * eps)
        only = torch.empty_like(vo)
        B.nvfp4_kv_read(cache, _gpu(at), None, only)
        assert torch.equal(only, vo)
        B.nvfp4_kv_read(cache, _gpu(at), only, None)
        assert torch.equal(only, ko)
    assert B.moe_get_device_status() == 0


def test_append_keys_only_saturation_and_special_values():
    """Without queries; blocks of zeros, values past the largest scale, and infinities (which
    saturate) leave finite rows in the cache."""
    k = torch.zeros(4, 1, 64, dtype=torch.bfloat16, device=DEV)
    k[1, 0, 3], k[1, 0, 17], k[2, 0, 5], k[3] = 1e30, -1e-30, float("inf"), -2.0
    cache = B.KVCache.allocate(1, 16, 1, 64)
    slots = torch.arange(4, dtype=torch.int32, device=DEV)
    B.nvfp4_kv_append(None, k, k, slots, slots, B.QKPrep(), cache, None)
    out = torch.empty(4, 1, 64, dtype=torch.float32, device=DEV)
    B.nvfp4_kv_read(cache, slots, out, None)
    o = out.cpu().numpy()[:, 0]
    assert not o[0].any() and o[1, 3] == 2688 and not np.delete(o[1], 3).any() and o[2, 5] == 2688
    assert np.all(o[3] == -2.0625)  # the scale 2 / 6 rounds to the E4M3 value 11 / 32, and 6 * 11 / 32 = 2.0625


def test_slots_past_the_end_are_skipped_and_reported():
    """Checked by the kernels themselves: the access is skipped and the status set."""
    cache = B.KVCache.allocate(2, 16, 1, 64)
    k = torch.ones(3, 1, 64, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    slots = torch.tensor([0, 32, 0x7fffffff], dtype=torch.int32, device=DEV)
    B.nvfp4_kv_append(None, k, k, pos, slots, B.QKPrep(), cache, None)
    assert B.moe_get_device_status() == B.MOE_ERR_INVALID_ARG and B.moe_get_device_status() == 0
    assert int((cache.k_scales != 0).sum()) == 4
    out = torch.full((3, 1, 64), 5.0, device=DEV)
    B.nvfp4_kv_read(cache, slots, out, None)
    assert B.moe_get_device_status() == B.MOE_ERR_INVALID_ARG
    assert torch.all(out[0] == 1.03125) and not out[1:].any()  # 6 times 11 / 64, the E4M3 value next to 1 / 6


# ---------------------------------------------------------------- attention

class Case:
    """Packed sequences over a cache of random rows, with pages in random order and everything
    that no sequence owns filled with NaN scales."""

    def __init__(self, D, Hkv, G, page, q_lens, ctx, seed, qscale=1.0, extra_rows=0):
        rng = np.random.default_rng(seed)
        self.rng, self.D, self.Hkv, self.Hq, self.q_lens, self.ctx = rng, D, Hkv, Hkv * G, q_lens, ctx
        need = [-(-c // page) for c in ctx]
        n_pages, self.max_pages = sum(need) + 2, max(need + [1])
        kts, vts = (rng.uniform(0.8, 1.2, Hkv).astype(np.float32) * 5 / 2688 for _ in range(2))
        self.cache = okv.Cache(n_pages, page, Hkv, D, kts, vts)
        for n in "kv":
            self.cache.codes[n][:] = rng.integers(0, 256, self.cache.codes[n].shape)
            self.cache.scales[n][:] = 0x7F  # NaN
        order = rng.permutation(n_pages).astype(np.int32)
        # columns for 65536 keys: a table as wide as a server's, so that every kernel is used (narrow
        # ones leave short batches to one kernel: check() runs both)
        self.table = np.full((len(ctx), max(self.max_pages, 65536 // page)), 0x7ffffff0, np.int32)
        self.slots, at = [], 0
        for b, c in enumerate(ctx):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            t = np.arange(c)
            s = self.table[b][t // page].astype(np.int64) * page + t % page if c else np.zeros(0, np.int64)
            self.slots.append(s)
            for n in "kv":
                self.cache.write(n, _bf16(rng, c, Hkv, D, spread=0.5), s)
        self.cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.T = int(self.cu[-1]) + extra_rows
        self.q = okv.to_bf16(_bf16(rng, self.T, self.Hq, D, spread=1.0) * np.float32(qscale))
        c = self.cache
        self.gcache = B.KVCache(_gpu(c.codes["k"]), _gpu(c.scales["k"]), _gpu(c.codes["v"]), _gpu(c.scales["v"]), _gpu(kts), _gpu(vts))
        self.ws = torch.full((B.nvfp4_kv_attention_workspace(self.T, len(ctx), self.T, self.Hq, self.gcache),), 0xFF,
                             dtype=torch.uint8, device=DEV)
        self.args = (_gpu(self.cu), _gpu(np.asarray(ctx, np.int32)), _gpu(self.table))

    def run(self, causal=True, lse=True, q=None, stream=None, max_q=None):
        out = torch.full((self.T, self.Hq, self.D), 3.0, dtype=torch.bfloat16, device=DEV)
        e = torch.full((self.T, self.Hq), 3.0, device=DEV) if lse else None
        q = _gpu(self.q).bfloat16() if q is None else q
        B.nvfp4_kv_attention(q, *self.args, max_q or max(self.q_lens + [1]), self.gcache, self.D ** -0.5, causal, out, e, self.ws,
                             stream=stream)
        return out, e

    def check(self, causal=True, rows=None):
        """Against the oracle, with the wide block table and one of the pages in use only; rows: at
        most that many query tokens of a sequence are checked."""
        wide = self.args
        self._check(causal, rows)
        self.args = wide[:2] + (wide[2][:, :self.max_pages].contiguous(),)
        self._check(causal, rows)
        self.args = wide

    def _check(self, causal, rows):
        out, lse = self.run(causal)
        assert B.moe_get_device_status() == 0
        out, lse = _np(out), lse.cpu().numpy()
        for b, (n, c) in enumerate(zip(self.q_lens, self.ctx)):
            k, v = self.cache.read("k", self.slots[b]), self.cache.read("v", self.slots[b])
            pick = np.arange(n) if rows is None or n <= rows else np.unique(np.concatenate(
                [[0, 1, n - 2, n - 1], self.rng.integers(0, n, rows - 4)]))
            vmax = np.abs(v).max() if c else 0.0
            for i in pick:
                keys = c if not causal else min(c, max(0, c - n + i + 1))
                t = self.cu[b] + i
                ref, e, w, s = okv.attention(self.q[t:t + 1], k[:keys], v[:keys], self.D ** -0.5, False)
                tol, tol_e = _attn_bounds(ref, w, s, e, keys, vmax, self.D)
                assert np.all(np.abs(out[t] - ref[0]) <= tol[0]), (b, i, np.abs(out[t] - ref[0]).max())
                if keys == 0:
                    assert np.all(np.isneginf(lse[t])) and not out[t].any()
                else:
                    assert np.all(np.abs(lse[t] - e[0]) <= tol_e[0]), (b, i, np.abs(lse[t] - e[0]).max())
        assert np.all(out[self.cu[-1]:] == 3.0) and np.all(lse[self.cu[-1]:] == 3.0)


@pytest.mark.parametrize("D,Hkv,G", [(64, 1, 1), (64, 2, 7), (128, 8, 4), (128, 3, 8), (128, 1, 32), (256, 2, 8), (256, 1, 3),
                                     (256, 1, 17)])
@pytest.mark.parametrize("page", [16, 64])
def test_attention_single_tokens(D, Hkv, G, page):
    Case(D, Hkv, G, page, [1] * 7, [1, 2, 15, 16, 17, 129, 700], D + G + page).check()


@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 7), (128, 2, 4), (256, 1, 8)])
def test_attention_few_tokens_and_empty_sequences(D, Hkv, G):
    """Sequences without queries, without keys, with more queries than keys (the first see none)."""
    c = Case(D, Hkv, G, 16, [3, 0, 5, 2, 1, 4, 16], [3, 40, 200, 0, 0, 2, 66], D + G, extra_rows=3)
    c.check()
    c.check(causal=False)


@pytest.mark.parametrize("D,Hkv,G,page", [(64, 2, 7, 16), (64, 3, 1, 128), (128, 1, 8, 64), (128, 2, 4, 32), (256, 2, 8, 64),
                                          (256, 1, 3, 1024)])
def test_attention_prompts(D, Hkv, G, page):
    """Whole prompts, a chunk with a past, and single tokens in one call."""
    c = Case(D, Hkv, G, page, [257, 1, 100, 1, 33], [257, 300, 411, 1, 33], D + G + page, extra_rows=2)
    c.check(rows=12)
    c.check(causal=False, rows=6)


def test_attention_long_context_and_many_sequences():
    Case(128, 1, 4, 64, [1, 2], [40000, 33333], 1).check()
    Case(64, 1, 2, 16, [1] * 600, [int(x) for x in np.random.default_rng(0).integers(0, 60, 600)], 2).check()


@pytest.mark.parametrize("n", [1, 40])
def test_attention_peaked_and_extreme_scores(n):
    """Scores in the hundreds (one key takes all weight, the running maximum moves often), zero
    queries (equal weights), tiny and huge queries."""
    c = Case(128, 2, 4, 32, [n, n], [300, 65], 3, qscale=40.0)
    c.check()
    c.q[0] = 0.0
    c.q[-1] = okv.to_bf16(c.q[-1] * 1e-30)
    c.check()
    q = _gpu(c.q).bfloat16()
    q[1 if n > 1 else 0, 0, 0] = float("nan")
    out, lse = c.run(q=q)
    t = 1 if n > 1 else 0
    assert torch.isnan(out[t, 0]).all() and torch.isnan(lse[t, 0])
    assert not torch.isnan(out[t, 1:]).any() and not torch.isnan(out[t + 1:]).any()


def test_attention_bad_pages_count_as_zeros_and_are_reported():
    """Page numbers outside the cache: the kernels skip the read and set the status."""
    for n in (1, 60):
        c = Case(128, 1, 4, 16, [n], [100], 4)
        good, _ = c.run()
        table = c.args[2].clone()
        table[0, 1], table[0, 3] = -5, c.gcache.n_pages
        c.args = (c.args[0], c.args[1], table)
        out, lse = c.run(causal=False)
        assert B.moe_get_device_status() == B.MOE_ERR_INVALID_ARG
        k, v = c.cache.read("k", c.slots[0]), c.cache.read("v", c.slots[0])
        for rows in (k, v):
            rows[16:32], rows[48:64] = 0.0, 0.0
        for t in (0, n - 1):
            ref, e, w, s = okv.attention(c.q[t:t + 1], k, v, c.D ** -0.5, False)
            tol, tol_e = _attn_bounds(ref, w, s, e, 100, np.abs(v).max(), c.D)
            assert np.all(np.abs(_np(out)[t] - ref[0]) <= tol[0]) and np.all(np.abs(lse.cpu().numpy()[t] - e[0]) <= tol_e[0])
        # lengths past the table and offsets past the queries are clamped to them
        c.args = (c.args[0] * 1000, c.args[1] * 1000, table.clamp(0, c.gcache.n_pages - 1))
        c.run()
        # offsets that go back and forth name the same rows many times: refused on the device
        many = torch.tensor([0, n] * 40 + [0], dtype=torch.int32, device=DEV)
        c.args = (many, torch.full((80,), 16, dtype=torch.int32, device=DEV), table[:1].clamp(0, 1).repeat(80, 1))
        c.ws = torch.zeros(B.nvfp4_kv_attention_workspace(c.T, 80, c.T, c.Hq, c.gcache), dtype=torch.uint8, device=DEV)
        c.run()
        torch.cuda.synchronize()
        B.moe_get_device_status()
        assert good.isfinite().all()


@pytest.mark.parametrize("q_lens,ctx", [([1] * 5, [700, 3, 256, 1000, 64]), ([200, 1, 30], [300, 500, 30])])
def test_attention_streams_graphs_strides_and_repeats(q_lens, ctx):
    """Captured and replayed on another stream with the workspace of eager calls, from strided
    rows, without lse: the same bits every time."""
    c = Case(128, 2, 4, 32, q_lens, ctx, 5)
    want, lse = c.run()
    again, lse2 = c.run()
    assert torch.equal(want, again) and torch.equal(lse, lse2)
    wide = torch.randn(c.T, c.Hq * c.D + 64, device=DEV).bfloat16()
    wide[:, :c.Hq * c.D] = _gpu(c.q.reshape(c.T, -1)).bfloat16()
    q = wide[:, :c.Hq * c.D].unflatten(1, (c.Hq, c.D))
    assert torch.equal(c.run(q=q, lse=False)[0], want)
    assert torch.equal(c.run(max_q=c.T)[0], want)  # a loose bound on the query counts
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, e = torch.empty_like(want), torch.empty_like(lse)
    g = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in g:  # two graphs share one workspace
        with torch.cuda.graph(graph, stream=s):
            B.nvfp4_kv_attention(q, *c.args, max(q_lens), c.gcache, c.D ** -0.5, True, out, e, c.ws)
    for graph in (g[0], g[1], g[0]):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(e, lse)


# ---------------------------------------------------------------- together

def test_steps_through_the_cache_match_one_prompt():
    """A prompt in one call, then single-token steps replayed from one CUDA graph with changing
    device arrays, against the oracle's attention over the rows the oracle quantises itself."""
    D, Hkv, Hq, page, n0, steps = 256, 2, 16, 64, 150, 6
    rng = np.random.default_rng(7)
    n = n0 + steps
    qkv = _bf16(rng, n, (Hq + 2 * Hkv) * D)
    f, m = L.rope_frequencies(64, 1e6, factor=4.0, trained=4096)
    w = _gpu(rng.uniform(0.5, 1.5, D).astype(np.float32))
    ts = torch.full((Hkv,), 5.0 / 2688, device=DEV)
    cache = B.KVCache.allocate(5, page, Hkv, D, ts, ts)
    att = L.CachedAttention(cache, B.QKPrep(w, w, 1e-6, f, False, m), Hq, n0, 1)
    table = torch.tensor([[3, 0, 4, 1]], dtype=torch.int32, device=DEV)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731

    def split(x):
        return (x[:, :Hq * D].unflatten(1, (Hq, D)), x[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D)),
                x[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D)))

    t = torch.arange(n, device=DEV)
    slots = (table[0][t // page] * page + t % page).int()
    x = _gpu(qkv).bfloat16()
    outs = [att.forward(*split(x[:n0]), t[:n0].int(), slots[:n0], i32(0, n0), i32(n0), table, n0).clone()]
    xb, pos, sl, ctx, cu = x[n0:n0 + 1].clone(), i32(n0), slots[n0:n0 + 1].clone(), i32(n0 + 1), i32(0, 1)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = att.forward(*split(xb), pos, sl, cu, ctx, table, 1)
    for j in range(steps):
        xb.copy_(x[n0 + j:n0 + j + 1])
        pos.fill_(n0 + j)
        sl.copy_(slots[n0 + j:n0 + j + 1])
        ctx.fill_(n0 + j + 1)
        g.replay()
        outs.append(out.clone())
    got = _np(torch.cat(outs))
    assert B.moe_get_device_status() == 0
    q, k, v = (a.reshape(n, -1, D) for a in np.split(qkv, [Hq * D, (Hq + Hkv) * D], axis=1))
    fn, wn = f.cpu().numpy(), w.cpu().numpy()
    p = np.arange(n)
    qr, kr = (okv.to_bf16(okv.norm_rope(a, p, wn, 1e-6, fn, False, m)) for a in (q, k))
    oc = okv.Cache(5, page, Hkv, D, ts.cpu().numpy(), ts.cpu().numpy())
    oc.write("k", kr, slots.cpu().numpy())
    oc.write("v", v, slots.cpu().numpy())
    kk, vv = oc.read("k", slots.cpu().numpy()), oc.read("v", slots.cpu().numpy())
    for i in list(range(0, n0, 29)) + list(range(n0 - 1, n)):
        ref, e, wt, s = okv.attention(qr[i:i + 1], kk[:i + 1], vv[:i + 1], D ** -0.5, False)
        tol, _ = _attn_bounds(ref, wt, s, e, i + 1, np.abs(vv).max(), D)
        assert np.all(np.abs(got[i] - ref[0]) <= tol[0]), i


# ---------------------------------------------------------------- edges of the kernels' own units

@pytest.mark.parametrize("D,Hkv,G", [(64, 1, 1), (64, 1, 14), (128, 2, 4), (128, 1, 5), (256, 2, 8), (256, 1, 3)])
@pytest.mark.parametrize("past", [0, 1, 126, 127, 128, 300])
def test_attention_around_tiles_of_rows_and_keys(D, Hkv, G, past):
    """Rows a key head just below, at and above 32 (where the other kernel takes over), 128 and 256
    (row tiles), contexts around multiples of 64 and 128, in one call."""
    q_lens = sorted({max(1, r // G + e) for r in (32, 128, 256) for e in (0, 1)})
    c = Case(D, Hkv, G, 16, q_lens, [n + past for n in q_lens], D + G + past, extra_rows=1)
    c.check(rows=5)


def test_attention_few_rows_over_a_long_cache_are_split():
    """One row tile whose keys go to many blocks, with 100, 160 and 300 rows."""
    for D, G, n in ((128, 4, 25), (128, 4, 40), (64, 3, 100), (256, 4, 40)):
        Case(D, 1, G, 64, [n], [20011], D + n).check(rows=4)


def test_attention_more_sequences_than_the_plan_takes_at_once():
    rng = np.random.default_rng(7)
    n = 1100  # the plan scans 1024 at a time
    q_lens = [int(x) for x in rng.integers(0, 3, n)]
    for b in (0, 500, 1023, 1024, 1099):
        q_lens[b] = 40
    Case(64, 1, 2, 16, q_lens, [x + int(rng.integers(0, 30)) for x in q_lens], 8).check(rows=4)


def test_attention_sequences_longer_than_max_q():
    """max_q only picks the kernels: a bound that is too low costs time, not results."""
    c = Case(128, 2, 4, 32, [3, 70], [50, 70], 9)
    want, _ = c.run()
    got, _ = c.run(max_q=1)
    assert B.moe_get_device_status() == 0
    tol = 2 * (2.0 ** -8 + 2.0 ** -9)  # both are roundings of nearly the same value: see check()
    c.check()
    assert np.all(np.abs(_np(got) - _np(want)) <= tol * np.maximum(np.abs(_np(want)), np.abs(_np(got)).max()))


@pytest.mark.parametrize("scale", [-0.11, 0.0, 3.0])
@pytest.mark.parametrize("n", [1, 50])
def test_attention_scales(n, scale):
    """A negative scale turns the order of the keys round, a scale of zero weighs them equally."""
    c = Case(64, 1, 2, 16, [n], [130], 10)
    out, lse = torch.empty(n, 2, 64, dtype=torch.bfloat16, device=DEV), torch.empty(n, 2, device=DEV)
    B.nvfp4_kv_attention(_gpu(c.q).bfloat16(), *c.args, n, c.gcache, scale, False, out, lse, c.ws)
    k, v = c.cache.read("k", c.slots[0]), c.cache.read("v", c.slots[0])
    ref, e, w, s = okv.attention(c.q, k, v, scale, False)
    tol, tol_e = _attn_bounds(ref, w, np.abs(s), e, 130, np.abs(v).max(), 64)
    assert np.all(np.abs(_np(out) - ref) <= tol) and np.all(np.abs(lse.cpu().numpy() - e) <= tol_e)


def test_attention_without_tensor_scales_and_with_negative_ones():
    for kts, vts in ((None, None), (-0.002, -0.5)):
        for n in (1, 50):
            c = Case(128, 1, 2, 16, [n], [90], 11)
            for name, ts in (("k", kts), ("v", vts)):
                c.cache.ts[name][:] = 1.0 if ts is None else ts
            g = c.gcache
            one = lambda x: None if x is None else torch.full((1,), x, device=DEV)  # noqa: E731
            c.gcache = B.KVCache(g.k_codes, g.k_scales, g.v_codes, g.v_scales, one(kts), one(vts))
            c.q = okv.to_bf16(c.q * (0.002 if kts is None else 1.0))
            c.check()


def test_attention_two_streams_at_once():
    """Two calls with a workspace each on two streams, and a small call with the workspace of a
    large one between two large ones: the same bits as alone."""
    a, b = Case(128, 2, 4, 32, [300, 1, 40], [700, 300, 40], 12), Case(128, 2, 4, 32, [1] * 9, list(range(1, 900, 100)), 13)
    want = [x.run()[0] for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for x, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(x.run()[0])
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    own, b.ws = b.ws, a.ws
    assert own.numel() <= a.ws.numel()
    for x, w in ((a, want[0]), (b, want[1]), (a, want[0])):
        assert torch.equal(x.run()[0], w)
    assert B.moe_get_device_status() == 0


def test_calls_without_tokens_or_sequences():
    cache = B.KVCache.allocate(1, 16, 1, 64)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    i = torch.empty(0, dtype=torch.int32, device=DEV)
    B.moe_qk_norm_rope(e, None, i, B.QKPrep(), e.clone(), None)
    B.nvfp4_kv_append(None, e[:, :1], e[:, :1], i, i, B.QKPrep(), cache, None)
    B.nvfp4_kv_read(cache, i, torch.empty(0, 1, 64, device=DEV), None)
    q = torch.ones(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 3.0)
    ws = torch.empty(B.nvfp4_kv_attention_workspace(3, 1, 3, 2, cache), dtype=torch.uint8, device=DEV)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    B.nvfp4_kv_attention(q, zero, zero[:1], zero[:1, None], 1, cache, 1.0, True, out, None, ws)
    assert torch.all(out == 3.0) and B.moe_get_device_status() == 0


@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -100, 2.0 ** 60])
def test_norm_of_huge_and_tiny_rows(size):
    """The sum of squares leaves float32's range; the normalised row does not."""
    rng = np.random.default_rng(14)
    x = okv.to_bf16(_bf16(rng, 6, 3, 128, spread=0) * size)
    pos = np.arange(6, dtype=np.int32) * 1000
    f = (1e4 ** (-np.arange(64) / 64)).astype(np.float32)
    w = rng.uniform(0.5, 1.5, 128).astype(np.float32)
    out, ko = (torch.empty(6, 3, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    B.moe_qk_norm_rope(_gpu(x).bfloat16(), _gpu(x).bfloat16(), _gpu(pos), B.QKPrep(_gpu(w), _gpu(w), 0.0, _gpu(f)), out, ko)
    ref = okv.norm_rope(x, pos, w, 0.0, f)
    top = np.sqrt(2) * np.abs(okv.norm_rope(np.abs(x), pos, w, 0.0)).max(axis=-1, keepdims=True)
    for got, err in ((out, 2.0 ** -24 * (128 / 16 + 16) * top), (ko, 0.0)):  # the terms of test_norm_rope
        assert np.all(np.abs(_np(got) - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -23) + err + 1e-37)


@pytest.mark.parametrize("D,Hq,Hkv,T", [(64, 14, 2, 4099), (128, 5, 3, 2053), (256, 3, 1, 1027)])
def test_many_tokens_match_few(D, Hq, Hkv, T):
    """Odd numbers of tokens through the writer of many tokens, and the same in slices of seven
    through the writer of few: the same cache bit for bit (keys and values; queries are compared
    with the oracle in test_norm_rope)."""
    c = _append_case(D, Hkv, 16, T, 15, Hq=Hq)
    ts = _gpu(c["kts"]), _gpu(c["vts"])
    prep = B.QKPrep(_gpu(c["w"]), _gpu(c["w"]), 1e-6, _gpu(c["f"]), True, 0.7)
    k, v, q = (_gpu(c[n]).bfloat16() for n in "kvq")
    pos, slots = _gpu(c["pos"]), _gpu(c["slots"])
    caches = [B.KVCache.allocate(c["n_pages"], 16, Hkv, D, *ts) for _ in range(2)]
    for x in caches:
        for t in (x.k_codes, x.k_scales, x.v_codes, x.v_scales):
            t.fill_(0x11)
    qo, qs = torch.empty_like(q), torch.empty_like(q)
    B.nvfp4_kv_append(q, k, v, pos, slots, prep, caches[0], qo)
    for i in range(0, T, 7):
        s = slice(i, min(i + 7, T))
        B.nvfp4_kv_append(q[s], k[s], v[s], pos[s], slots[s], prep, caches[1], qs[s])
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(caches[0], n), getattr(caches[1], n)), n
    # two roundings to bf16 of values that differ by float32 roundings: at most a bf16 step
    assert np.all(np.abs(_np(qo) - _np(qs)) <= 2.0 ** -7 * np.maximum(np.abs(_np(qo)), np.abs(_np(qs))) + 2.0 ** -18)
    assert B.moe_get_device_status() == 0


@pytest.mark.parametrize("ts", [0.0, 1e-38, 1e30, 3.0e38, 2.0 ** -61, 0.7, float("inf"), float("nan"), -0.02, -1e30])
def test_append_quantises_as_the_quantiser_for_any_tensor_scale(ts):
    """Tensor scales beyond the range of the fast quotients: the quantiser's bits, for rows of every
    size, zeros, subnormals, infinities among them."""
    rng = np.random.default_rng(16)
    T, D = 300, 64
    x = okv.to_bf16(rng.standard_normal((T, 1, D)) * np.exp2(rng.uniform(-130, 120, (T, 1, 1))))
    x[::7, :, ::5] = 0.0
    x[3, 0, 1], x[4, 0, 2], x[5] = np.inf, -np.inf, 0.0
    v = _gpu(x).bfloat16()
    t = torch.full((1,), ts, device=DEV)
    cache = B.KVCache.allocate(-(-T // 16), 16, 1, D, t, t)
    i32 = torch.arange(T, dtype=torch.int32, device=DEV)
    B.nvfp4_kv_append(None, v, v, i32, i32, B.QKPrep(), cache, None)
    codes, scales = torch.empty(T, D // 2, dtype=torch.uint8, device=DEV), torch.empty(T, D // 16, dtype=torch.uint8, device=DEV)
    B.nvfp4_quantize_act(v.reshape(T, D), codes, scales, torch.empty(1, device=DEV), t)
    for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        assert torch.equal(c.reshape(-1, D // 2)[:T], codes) and torch.equal(s.reshape(-1, D // 16)[:T], scales)


@pytest.mark.parametrize("D,Hkv,G", [(128, 1, 64), (64, 1, 100), (256, 2, 33)])
def test_attention_many_heads_on_one_key_head(D, Hkv, G):
    """One token is more than 32 rows: single tokens through the kernel of many rows."""
    Case(D, Hkv, G, 16, [1] * 5, [1, 17, 128, 129, 700], D + G).check()


@pytest.mark.parametrize("max_q", [1, 40])
def test_attention_when_no_sequence_has_a_query(max_q):
    c = Case(128, 1, 4, 16, [0, 0, 0], [30, 0, 200], 17, extra_rows=5)
    out, lse = c.run(max_q=max_q)
    assert torch.all(out == 3.0) and torch.all(lse == 3.0) and B.moe_get_device_status() == 0


def test_attention_one_token_over_a_very_long_cache():
    Case(64, 1, 1, 1024, [1, 1], [300001, 1], 18).check()


def test_cache_of_more_than_four_gigabytes():
    """Offsets past 32 bits: rows at the end of 2^22 + 64 tokens of 8 heads of 256."""
    D, Hkv, page = 256, 8, 64
    n_pages = (1 << 22) // page + 1
    cache = B.KVCache.allocate(n_pages, page, Hkv, D)
    assert cache.k_codes.numel() > 1 << 32
    rng = np.random.default_rng(19)
    T = 50
    k, v, q = _bf16(rng, T, Hkv, D), _bf16(rng, T, Hkv, D), _bf16(rng, T, Hkv, D)
    slots = ((n_pages - 1) * page + np.arange(T)).astype(np.int32)
    kg, vg, qg = (_gpu(x).bfloat16() for x in (k, v, q))
    B.nvfp4_kv_append(None, kg, vg, None, _gpu(slots), B.QKPrep(), cache, None)
    oc = okv.Cache(1, page, Hkv, D)
    for n, x in (("k", k), ("v", v)):
        oc.write(n, x, np.arange(T))
    out = [torch.empty(T, Hkv, D, device=DEV) for _ in range(2)]
    B.nvfp4_kv_read(cache, _gpu(slots), *out)
    kk, vv = oc.read("k", np.arange(T)), oc.read("v", np.arange(T))
    assert np.array_equal(out[0].cpu().numpy(), kk) and np.array_equal(out[1].cpu().numpy(), vv)
    assert not cache.k_codes[:T].any()  # where an offset cut to 32 bits would land
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    for n in (1, T):  # both kernels
        o, e = torch.empty(n, Hkv, D, dtype=torch.bfloat16, device=DEV), torch.empty(n, Hkv, device=DEV)
        ws = torch.empty(B.nvfp4_kv_attention_workspace(n, 1, n, Hkv, cache), dtype=torch.uint8, device=DEV)
        B.nvfp4_kv_attention(qg[T - n:], i32(0, n), i32(T), i32(n_pages - 1)[None], n, cache, D ** -0.5, False, o, e, ws)
        ref, lse, w, s = okv.attention(q[T - n:], kk, vv, D ** -0.5, False)
        tol, tol_e = _attn_bounds(ref, w, s, lse, T, np.abs(vv).max(), D)
        assert np.all(np.abs(_np(o) - ref) <= tol) and np.all(np.abs(e.cpu().numpy() - lse) <= tol_e)
