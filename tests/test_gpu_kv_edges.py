"""The cache and attention calls at values and indices that ordinary data does not have: page
numbers that a kernel might take for a mark of its own."""
import numpy as np
import pytest
import torch

from oracle import kv as okv
from nvfp4_expert_ffn_b200 import binding as B
from test_gpu_kv_cache import Case, _attn_bounds, _gpu, _np

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
