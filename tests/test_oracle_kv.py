"""Pins of the attention-side oracle against library routines and closed forms (CPU)."""
import numpy as np
import pytest
import torch

from oracle import kv as okv
from nvfp4_expert_ffn_b200 import layer as L


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product_and_keeps_relative_angles(interleaved):
    rng = np.random.default_rng(1)
    x, f = rng.standard_normal((5, 2, 64)), np.float32(0.3) ** np.arange(16, dtype=np.float32)
    pos = np.array([0, 1, 7, 1000, 300000])
    y = okv.norm_rope(x, pos, inv_freq=f, interleaved=interleaved)
    i, j = (np.arange(0, 32, 2), np.arange(1, 32, 2)) if interleaved else (np.arange(16), np.arange(16, 32))
    z = (x[..., i] + 1j * x[..., j]) * np.exp(1j * pos[:, None] * f.astype(np.float64))[:, None]
    assert np.allclose(y[..., i], z.real, atol=1e-10) and np.allclose(y[..., j], z.imag, atol=1e-10)
    assert np.array_equal(y[..., 32:], x[..., 32:]) and np.array_equal(y[0], x[0])
    # scores depend on the distance alone
    a, b = x[:1], x[1:2]
    s = [np.sum(okv.norm_rope(a, [p + 9], inv_freq=f, interleaved=interleaved) *
                okv.norm_rope(b, [p], inv_freq=f, interleaved=interleaved)) for p in (0, 5, 900)]
    assert np.allclose(s, s[0], atol=1e-9)


def test_norm_has_unit_mean_square_before_the_weight():
    x = np.random.default_rng(2).standard_normal((3, 4, 128)) * 7
    y = okv.norm_rope(x, [0, 1, 2], weight=np.full(128, 2.0))
    assert np.allclose(np.mean(y * y, axis=-1), 4.0)
    t = torch.nn.functional.rms_norm(torch.from_numpy(x), (128,), torch.full((128,), 2.0, dtype=torch.float64), 1e-3)
    assert np.allclose(okv.norm_rope(x, [0, 1, 2], weight=np.full(128, 2.0), eps=1e-3), t.numpy())


def test_bf16_rounding_matches_torch():
    x = np.random.default_rng(3).standard_normal(4096) * np.exp2(np.random.default_rng(4).integers(-30, 30, 4096))
    assert np.array_equal(okv.to_bf16(x), torch.from_numpy(x).float().bfloat16().float().numpy())


def test_cache_returns_what_the_codes_stand_for():
    c = okv.Cache(4, 16, 2, 64, k_ts=[0.5, 0.01])
    rows = np.zeros((3, 2, 64), np.float32)
    rows[:, :, 0], rows[:, :, 1], rows[:, 1] = 6.0, -1.5, rows[:, 1] * 0.02
    rows[:, 1, 0], rows[:, 1, 1] = 0.12, -0.03
    c.write("k", rows, [5, -1, 63])
    got = c.read("k", [5, 63, 6])
    assert np.allclose(got[0, 0, :3], [6.0, -1.5, 0.0]) and np.array_equal(got[0], got[1]) and not got[2].any()
    assert np.allclose(got[0, 1, :2], [0.12, -0.03])


@pytest.mark.parametrize("causal", [False, True])
def test_attention_matches_torch(causal):
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((7, 6, 16)), rng.standard_normal((11, 2, 16)), rng.standard_normal((11, 2, 16))
    out, lse, weight, logit = okv.attention(q, k, v, 0.3, causal)
    t = [torch.from_numpy(a).transpose(0, 1) for a in (q, k.repeat(3, 1), v.repeat(3, 1))]
    mask = torch.ones(7, 11).tril(4).bool() if causal else torch.ones(7, 11).bool()
    s = (t[0] @ t[1].mT * 0.3).masked_fill(~mask, -torch.inf)
    assert np.allclose(out, (s.softmax(-1) @ t[2]).transpose(0, 1).numpy())
    assert np.allclose(lse, s.logsumexp(-1).T.numpy())
    assert np.all(weight >= np.abs(out) - 1e-12) and np.all(logit >= np.abs(s.masked_fill(~mask, 0).amax(-1).T.numpy()) - 1e-12)


def test_attention_without_keys_is_zero():
    q = np.ones((3, 2, 16))
    out, lse, _, _ = okv.attention(q, np.ones((2, 1, 16)), np.ones((2, 1, 16)), 1.0, True)
    assert not out[0].any() and np.all(np.isinf(lse[0])) and np.allclose(out[1:], 1.0)


def test_rope_frequencies():
    f, m = L.rope_frequencies(64, 10000.0, device="cpu")
    assert m == 1.0 and f.dtype == torch.float32 and f.shape == (32,) and f[0] == 1.0
    assert np.allclose(f.numpy(), 10000.0 ** (-np.arange(32) / 32.0))
    lin, m = L.rope_frequencies(64, 10000.0, factor=4.0, device="cpu")
    assert m == 1.0 and torch.equal(lin, f / 4)
    g, m = L.rope_frequencies(64, 10000.0, factor=4.0, trained=4096, device="cpu")
    assert m == pytest.approx(0.1 * np.log(4.0) + 1.0)
    turns = 4096 * f.double() / (2 * np.pi)
    assert torch.equal(g[turns > 33], f[turns > 33]) and torch.allclose(g[turns < 0.9], f[turns < 0.9] / 4)
    assert torch.all(g <= f) and torch.all(g >= f / 4.0001)
