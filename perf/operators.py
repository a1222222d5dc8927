"""Cases of the cache operators of an attention layer beside the NVFP4 expert layer: the norm
and rotation of queries and keys, the quantised write of keys and values into a paged NVFP4
cache, the read of cached rows, and attention over the cache.

Each case is computed in two ways: by elementary torch operations (the plain form) and, with
``own`` set, by the library's calls. ``exact`` states the same results in 64 bits.

NVFP4 as in include/moe_nvfp4.h: E2M1 codes (element 2i in the low nibble), one E4M3 scale per
16 elements, a float32 tensor scale (here one per key/value head); the conversions are defined
on float32 quotients, rounded to nearest even.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# Head layouts: (query heads, key/value heads, head size, rotated elements, interleaved pairs)
LAYOUTS = {
    "16+2x256": (16, 2, 256, 64, False),    # wide heads, a quarter of each rotated
    "32+8x128": (32, 8, 128, 128, False),   # four queries to a key head, all of it rotated
    "32+8x128i": (32, 8, 128, 128, True),   # the same with interleaved pairs
    "14+2x64": (14, 2, 64, 32, True),       # seven queries to a key head, half rotated
    "8+8x64": (8, 8, 64, 64, False),        # every head its own keys
    "24+3x128": (24, 3, 128, 96, False),    # odd number of key heads
}


def _ints(text):
    return [int(v) for v in text.split(",")]


def _text(values):
    return ",".join(str(v) for v in values)


def listed():
    ragged8 = [16384, 16383, 15001, 12345, 16001, 9999, 16129, 14080]
    r = random.Random(64)
    ragged64 = [r.randint(2048, 8192) for _ in range(64)]
    wide_q = [512, 2048, 8192, 16384, 1, 1, 1, 1]  # the ragged prefill + decode mix of the wide expert layer
    return [
        # one decode step of 8 slots: launch and latency bound
        {"name": "norm_rope T=8", "op": "norm_rope", "layout": "16+2x256", "T": 8, "start": 30000, "scaled": False},
        # a 16K prompt, frequencies scaled for a long context, interleaved pairs
        {"name": "norm_rope T=16384", "op": "norm_rope", "layout": "32+8x128i", "T": 16384, "start": 100000, "scaled": True},
        # the cache write of one decode step of 8 slots
        {"name": "append T=8", "op": "append", "layout": "16+2x256", "T": 8, "page": 64, "start": 30000, "scaled": False},
        # an odd chunk of a prompt, small heads and small pages, no multiple of anything
        {"name": "append T=1001", "op": "append", "layout": "14+2x64", "T": 1001, "page": 16, "start": 5, "scaled": False},
        # the whole wide prefill + decode mix written in one call
        {"name": "append T=27140", "op": "append", "layout": "32+8x128", "T": 27140, "page": 64, "start": 0, "scaled": True},
        # a short prefix read back
        {"name": "read n=333", "op": "read", "layout": "14+2x64", "n": 333, "page": 16},
        # a 64K-token prefix read back
        {"name": "read n=65536", "op": "read", "layout": "16+2x256", "n": 65536, "page": 64},
        # one sequence, one token, a short context: latency alone
        {"name": "attn decode 1x1000", "op": "attn", "layout": "32+8x128", "page": 16, "q": "1", "ctx": "1000"},
        # 8 slots of one token near 16K of context
        {"name": "attn decode 8x16K", "op": "attn", "layout": "16+2x256", "page": 64, "q": _text([1] * 8), "ctx": _text(ragged8)},
        # a full batch of ragged contexts
        {"name": "attn decode 64x8K", "op": "attn", "layout": "32+8x128", "page": 64, "q": _text([1] * 64), "ctx": _text(ragged64)},
        # a whole 16K prompt
        {"name": "attn prompt 16K", "op": "attn", "layout": "16+2x256", "page": 64, "q": "16384", "ctx": "16384"},
        # the wide mix: four prompts of different lengths and four single tokens with a past, in one call
        {"name": "attn mix 27140", "op": "attn", "layout": "32+8x128", "page": 64, "q": _text(wide_q),
         "ctx": _text([512, 2048, 8192, 16384, 4000, 777, 16384, 1])},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    layout = rng.choice(sorted(LAYOUTS))
    page = rng.choice((16, 32, 64, 128))
    op = rng.choice(("norm_rope", "append", "read", "attn", "attn", "attn"))
    if op == "norm_rope":
        return {"op": op, "layout": layout, "T": _log_int(rng, 1, 16384), "start": _log_int(rng, 1, 500000), "scaled": rng.random() < 0.5}
    if op == "append":
        return {"op": op, "layout": layout, "T": _log_int(rng, 1, 16384), "page": page, "start": _log_int(rng, 1, 500000), "scaled": rng.random() < 0.5}
    if op == "read":
        return {"op": op, "layout": layout, "n": _log_int(rng, 1, 65536), "page": page}
    kind = rng.choice(("decode", "few", "prompt"))
    if kind == "decode":    # one token of each of n sequences
        n = _log_int(rng, 1, 64)
        most = _log_int(rng, 64, 8192 if n > 8 else 32768)
        q, ctx = [1] * n, [rng.randint(1, most) for _ in range(n)]
    elif kind == "few":     # a few tokens each: speculative steps, the ends of prompts
        n = _log_int(rng, 1, 16)
        most = _log_int(rng, 64, 8192)
        q = [rng.randint(1, 16) for _ in range(n)]
        ctx = [m + rng.randint(0, most) for m in q]
    else:                   # prompts and chunks of prompts with a past
        n = rng.randint(1, 4)
        q = [_log_int(rng, 17, 6000) for _ in range(n)]
        ctx = [m + (_log_int(rng, 1, 4096) if rng.random() < 0.5 else 0) for m in q]
    return {"op": op, "layout": layout, "page": page, "q": _text(q), "ctx": _text(ctx)}


# --------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _uniform(g, lo, hi, *shape):
    return torch.rand(*shape, generator=g, device=DEV) * (hi - lo) + lo


def _inv_freq(rot, scaled):
    """theta^(-2p/R); scaled: the slow frequencies divided by 8 with a ramp between, as for contexts
    beyond the trained length. Also the factor on cos and sin that goes with it."""
    p = torch.arange(rot // 2, dtype=torch.float64)
    f = 1e6 ** (-2.0 * p / rot)
    if not scaled:
        return f.float().to(DEV), 1.0
    turns = 32768.0 * f / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
    return (f * (keep + (1 - keep) / 8.0)).float().to(DEV), 0.1 * math.log(8.0) + 1.0


def _head_scales(g, heads):
    """Static tensor scales: a calibrated maximum near 5 over 6 * 448."""
    return _uniform(g, 0.8, 1.25, heads) * (5.0 / 2688.0)


def _projected(case, g):
    """Queries, keys and values as rows of one projection's output, with the norm's weights and the rotation."""
    Hq, Hkv, D, rot, inter = LAYOUTS[case["layout"]]
    T = case["T"]
    qkv = (_normal(g, T, (Hq + 2 * Hkv) * D) * _uniform(g, 0.5, 2.0, T, 1)).bfloat16()
    f, m = _inv_freq(rot, case["scaled"])
    pos = torch.arange(T, device=DEV, dtype=torch.int32) + case["start"]
    if T <= 64:  # a decode step: every row its own sequence
        pos = torch.randint(0, case["start"] + 1, (T,), generator=g, device=DEV, dtype=torch.int32)
    return {
        "q": qkv[:, : Hq * D].unflatten(1, (Hq, D)), "k": qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D)),
        "v": qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D)),
        "q_weight": _uniform(g, 0.5, 1.5, D), "k_weight": _uniform(g, 0.5, 1.5, D), "eps": 1e-6,
        "positions": pos, "inv_freq": f, "interleaved": inter, "rot_scale": m, "rot": rot,
        "q_out": torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV),
    }


def _empty_cache(g, n_pages, Hkv, page, D):
    def z(n):
        return torch.zeros(n_pages, Hkv, page, n, dtype=torch.uint8, device=DEV)
    return {"k_codes": z(D // 2), "k_scales": z(D // 16), "v_codes": z(D // 2), "v_scales": z(D // 16),
            "k_ts": _head_scales(g, Hkv), "v_ts": _head_scales(g, Hkv)}


def _filled_cache(g, n_pages, Hkv, page, D):
    """A cache whose blocks are drawn from a pool of quantised normal blocks."""
    cache = _empty_cache(g, n_pages, Hkv, page, D)
    x = _normal(g, 1 << 16, 16) * _uniform(g, 0.5, 1.5, 1 << 16, 1)
    codes, scales = _quantise(x, torch.tensor(5.0 / 2688.0, device=DEV))
    blocks = codes.view(torch.int64).view(-1)
    for name in ("k", "v"):
        c, s = cache[name + "_codes"], cache[name + "_scales"]
        at = torch.randint(0, 1 << 16, (s.numel(),), generator=g, device=DEV)
        c.view(-1).view(torch.int64).copy_(blocks[at])
        s.view(-1).copy_(scales.view(-1)[at])
    return cache


def prepare(case, seed):
    g = _gen(seed)
    Hq, Hkv, D, rot, inter = LAYOUTS[case["layout"]]
    if case["op"] == "norm_rope":
        s = _projected(case, g)
        s["k_out"] = torch.empty(case["T"], Hkv, D, dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "append":
        s = _projected(case, g)
        page, T = case["page"], case["T"]
        n_pages = -(-T // page) + 7
        s["cache"] = _empty_cache(g, n_pages, Hkv, page, D)
        order = torch.randperm(n_pages, generator=g, device=DEV)
        t = torch.arange(T, device=DEV)
        if T <= 64:  # a decode step: any distinct places
            s["slots"] = torch.randperm(n_pages * page, generator=g, device=DEV)[:T].int()
        else:
            s["slots"] = (order[t // page] * page + t % page).int()
        s["k_out"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "read":
        page, n = case["page"], case["n"]
        n_pages = -(-n // page) + 3
        order = torch.randperm(n_pages, generator=g, device=DEV)
        t = torch.arange(n, device=DEV)
        s = {"cache": _filled_cache(g, n_pages, Hkv, page, D), "slots": (order[t // page] * page + t % page).int(),
             "k_out": torch.empty(n, Hkv, D, dtype=torch.bfloat16, device=DEV),
             "v_out": torch.empty(n, Hkv, D, dtype=torch.bfloat16, device=DEV)}
    else:
        page, q, ctx = case["page"], _ints(case["q"]), _ints(case["ctx"])
        need = [-(-c // page) for c in ctx]
        n_pages, T = sum(need) + 5, sum(q)
        order = torch.randperm(n_pages, generator=g, device=DEV).int()
        table = torch.full((len(q), max(need)), -1, dtype=torch.int32, device=DEV)
        cu, at = [0], 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
            cu.append(cu[-1] + q[b])
        # the plain form takes the sequences of few tokens as one padded batch, each long one by itself
        few = [b for b in range(len(q)) if q[b] <= 16]
        s = {"q": (_normal(g, T, Hq, D) * _uniform(g, 0.5, 2.5, T, Hq, 1)).bfloat16(),
             "cache": _filled_cache(g, n_pages, Hkv, page, D), "table": table,
             "cu_q": torch.tensor(cu, dtype=torch.int32, device=DEV), "ctx": torch.tensor(ctx, dtype=torch.int32, device=DEV),
             "max_q": max(q), "scale": D ** -0.5,
             "groups": [(torch.tensor(ids, device=DEV), max(q[b] for b in ids), max(ctx[b] for b in ids))
                        for ids in ([few] if few else []) + [[b] for b in range(len(q)) if q[b] > 16]],
             "out": torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV),
             "lse": torch.empty(T, Hq, dtype=torch.float32, device=DEV)}
    s["op"] = case["op"]
    return s


# --------------------------------------------------------------------------------- plain forms

def _quantise(x, ts):
    """float32 [..., 16n] with tensor scales ts (broadcast over the last axis' blocks) -> codes, scales."""
    b = x.unflatten(-1, (-1, 16))
    s8 = (b.abs().amax(-1) / 6.0 / ts).clamp(max=448.0).to(torch.float8_e4m3fn)
    sv = s8.float()
    q = torch.where(sv[..., None] > 0, b / (sv * ts)[..., None], torch.zeros((), device=x.device))
    a = q.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
    code = code | (torch.signbit(q).byte() << 3)
    code = code.flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), s8.view(torch.uint8)


def _values(codes, scales):
    """codes [..., D/2], scales [..., D/16] -> e2m1 * e4m3 as float32 [..., D]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _rows(cache, name, page, off):
    """Cached rows of every head at the given pages and offsets: [..., Hkv, D] float32."""
    v = _values(cache[name + "_codes"][page, :, off], cache[name + "_scales"][page, :, off])
    return v * cache[name + "_ts"][:, None]


def _norm_rope(s, x, w):
    """In 64 bits: the result's bf16 value is next quantised to 4 bits, where a last bit is a whole step."""
    x = x.double()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.double()
    a = s["positions"].double()[:, None] * s["inv_freq"].double()
    c, d = (torch.cos(a) * s["rot_scale"])[:, None], (torch.sin(a) * s["rot_scale"])[:, None]
    R = s["rot"]
    if s["interleaved"]:
        lo, hi = x[..., 0:R:2], x[..., 1:R:2]
    else:
        lo, hi = x[..., : R // 2], x[..., R // 2:R]
    lo, hi = lo * c - hi * d, hi * c + lo * d
    turned = torch.stack((lo, hi), -1).flatten(-2) if s["interleaved"] else torch.cat((lo, hi), -1)
    return torch.cat((turned, x[..., R:]), -1).float().bfloat16()


def _attend(s, out, lse, ids, nq, nctx):
    """Attention of the sequences `ids`, padded to nq queries and nctx keys each."""
    cache = s["cache"]
    page = cache["k_codes"].shape[2]
    T, Hq, D = s["q"].shape
    Hkv = cache["k_codes"].shape[1]
    ctx, first, last = s["ctx"][ids].long(), s["cu_q"][ids].long(), s["cu_q"][ids + 1].long()
    j = torch.arange(nctx, device=ctx.device)
    j_ok = j < ctx[:, None]
    pages = s["table"][ids][:, j // page].long().clamp(min=0)
    off = (j % page).expand_as(pages)
    k = _rows(cache, "k", pages, off).permute(0, 2, 3, 1)                       # [n, Hkv, D, ctx]
    v = _rows(cache, "v", pages, off).masked_fill_(~j_ok[..., None, None], 0.0).permute(0, 2, 1, 3)
    i = torch.arange(nq, device=ctx.device)
    i_ok = i < (last - first)[:, None]
    t = (first[:, None] + i).clamp(max=T - 1)
    q = s["q"][t].float().unflatten(2, (Hkv, -1)).permute(0, 2, 1, 3, 4)        # [n, Hkv, nq, G, D]
    G = q.shape[3]
    p = (q.flatten(2, 3) @ k).unflatten(2, (nq, G))
    del k
    p *= s["scale"]
    at = (ctx - (last - first))[:, None] + i
    seen = (j <= at[..., None]) & j_ok[:, None]                                 # [n, nq, ctx]
    p.masked_fill_(~seen[:, None, :, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p -= m
    p.exp_()
    z = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (nq, G)) / torch.where(z > 0, z, torch.ones_like(z))
    e = (m + torch.log(z)).squeeze(-1)
    rows = t[i_ok]
    out[rows] = o.permute(0, 2, 1, 3, 4).flatten(2, 3)[i_ok].bfloat16()
    lse[rows] = e.permute(0, 2, 1, 3).flatten(2, 3)[i_ok]


def _run_plain(s):
    if s["op"] == "norm_rope":
        return {"q": _norm_rope(s, s["q"], s["q_weight"]), "k": _norm_rope(s, s["k"], s["k_weight"])}
    if s["op"] == "attn":
        out, lse = s["out"], s["lse"]
        for group in s["groups"]:
            _attend(s, out, lse, *group)
        return {"out": out, "lse": lse}
    cache, slots = s["cache"], s["slots"].long()
    page = cache["k_codes"].shape[2]
    at = (slots // page, slots % page)
    got = {}
    if s["op"] == "append":
        got["q"] = _norm_rope(s, s["q"], s["q_weight"])
        for name, x in (("k", _norm_rope(s, s["k"], s["k_weight"])), ("v", s["v"])):
            codes, scales = _quantise(x.float(), cache[name + "_ts"][:, None])
            cache[name + "_codes"][at[0], :, at[1]] = codes
            cache[name + "_scales"][at[0], :, at[1]] = scales
    got["k"], got["v"] = (_rows(cache, name, *at).bfloat16() for name in ("k", "v"))
    return got


# --------------------------------------------------------------------------------- the library

def _run_own(s):
    from nvfp4_expert_ffn_b200 import binding as B
    if "handle" not in s:  # what a program builds once: the cache's handle, the norm and rotation, the workspace
        s["handle"] = B.KVCache(**s["cache"]) if "cache" in s else None
        if "q_weight" in s:
            s["prep"] = B.QKPrep(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], inv_freq=s["inv_freq"],
                                 interleaved=s["interleaved"], rot_scale=s["rot_scale"])
        if s["op"] == "attn":
            T, Hq, _ = s["q"].shape
            n = B.nvfp4_kv_attention_workspace(T, len(s["ctx"]), s["max_q"], Hq, s["handle"])
            s["ws"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
    if s["op"] == "norm_rope":
        B.moe_qk_norm_rope(s["q"], s["k"], s["positions"], s["prep"], s["q_out"], s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if s["op"] == "attn":
        B.nvfp4_kv_attention(s["q"], s["cu_q"], s["ctx"], s["table"], s["max_q"], s["handle"], s["scale"], True,
                             s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    got = {}
    if s["op"] == "append":
        B.nvfp4_kv_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["prep"], s["handle"], s["q_out"])
        got["q"] = s["q_out"]
    B.nvfp4_kv_read(s["handle"], s["slots"], s["k_out"], s["v_out"])
    return got | {"k": s["k_out"], "v": s["v_out"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    Hq, Hkv, D, rot, inter = LAYOUTS[case["layout"]]
    cached = 2 * Hkv * D * 9 / 16  # a token's keys and values: 4 bits and a 16th of a byte each
    if case["op"] == "norm_rope":
        n = case["T"] * (Hq + Hkv) * D
        return {"bytes": 4 * n + 4 * case["T"], "flops": 9 * n}
    if case["op"] == "append":  # written, and the rows read back
        T = case["T"]
        return {"bytes": T * ((Hq + 2 * Hkv) * D * 2 + Hq * D * 2 + cached + cached + 2 * Hkv * D * 2 + 8),
                "flops": 9 * T * (Hq + 2 * Hkv) * D}
    if case["op"] == "read":
        return {"bytes": case["n"] * (cached + 2 * Hkv * D * 2 + 4), "flops": 2 * case["n"] * 2 * Hkv * D}
    q, ctx = _ints(case["q"]), _ints(case["ctx"])
    pairs = sum(n * c - n * (n - 1) // 2 for n, c in zip(q, ctx))
    return {"bytes": sum(ctx) * cached + sum(q) * Hq * (4 * D + 4), "flops": 4 * D * Hq * pairs}


# --------------------------------------------------------------------------------- in 64 bits

def _nearest(x, table):
    """Index of the table's nearest value (ascending, from 0), a tie to the even index, for x >= 0 in float64."""
    t = torch.tensor(table, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(t, x).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    a, b = x - t[lo], t[hi] - x
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def _stored(x, ts):
    """The values that a block of 16 stands for once it is in the cache: float64 of x in bf16, ts float32."""
    e4m3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
    b = x.unflatten(-1, (-1, 16))
    sb = (b.abs().amax(-1).float() / 6.0 / ts).double()
    s = torch.tensor(e4m3, dtype=torch.float64, device=x.device)[_nearest(sb, e4m3)]
    d = (s.float() * ts).double()[..., None]
    y = torch.where(d > 0, (b / d).float().double(), torch.zeros_like(b))
    v = torch.tensor(E2M1, dtype=torch.float64, device=x.device)[_nearest(y.abs(), E2M1)] * torch.sign(y)
    return (v * s[..., None] * ts.double()[..., None]).flatten(-2)


def _turned(s, x, w):
    """The norm and the rotation as a product of complex numbers."""
    x = x.double()
    x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt() * w.double()
    R = s["rot"]
    r = x[..., :R]
    pairs = r.unflatten(-1, (R // 2, 2)) if s["interleaved"] else r.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    a = torch.outer(s["positions"].double(), s["inv_freq"].double())
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(a, s["rot_scale"]), a)[:, None]
    z = torch.view_as_real(z)
    z = z.flatten(-2) if s["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat((z, x[..., R:]), -1)


def _cached(cache, name, page, off):
    """Rows of the cache in float64, by indexing a table of all 256 bytes."""
    lut = torch.tensor([[v * (1 - 2 * n) for n in (0, 1) for v in E2M1]], dtype=torch.float64, device=page.device)[0]
    byte = torch.arange(256, device=page.device)
    both = torch.stack((lut[byte % 16], lut[byte // 16]), 1)
    c = cache[name + "_codes"][page, :, off].long()
    s = cache[name + "_scales"][page, :, off].view(torch.float8_e4m3fn).double()
    x = both[c].flatten(-2).unflatten(-1, (-1, 16)) * s[..., None]
    return x.flatten(-2) * cache[name + "_ts"].double()[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return {"q": _turned(s, s["q"], s["q_weight"]), "k": _turned(s, s["k"], s["k_weight"])}
    if case["op"] == "append":
        k = _turned(s, s["k"], s["k_weight"]).float().bfloat16().double()
        return {"q": _turned(s, s["q"], s["q_weight"]), "k": _stored(k, s["cache"]["k_ts"][:, None]),
                "v": _stored(s["v"].double(), s["cache"]["v_ts"][:, None])}
    cache, page = s["cache"], case["page"]
    if case["op"] == "read":
        at = (s["slots"].long() // page, s["slots"].long() % page)
        return {"k": _cached(cache, "k", *at), "v": _cached(cache, "v", *at)}
    T, Hq, D = s["q"].shape
    Hkv = cache["k_codes"].shape[1]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    first = 0
    for b, (n, c) in enumerate(zip(_ints(case["q"]), _ints(case["ctx"]))):
        j = torch.arange(c, device=DEV)
        at = (s["table"][b].long()[j // page], j % page)
        k, v = _cached(cache, "k", *at), _cached(cache, "v", *at)
        hidden = j > (c - n + torch.arange(n, device=DEV))[:, None]
        for h in range(Hq):
            x = s["q"][first:first + n, h].double() @ k[:, h * Hkv // Hq].T * s["scale"]
            x.masked_fill_(hidden, -math.inf)
            e = torch.logsumexp(x, -1)
            out[first:first + n, h] = x.sub_(e[:, None]).exp_() @ v[:, h * Hkv // Hq]
            lse[first:first + n, h] = e
        first += n
    return {"out": out, "lse": lse}
