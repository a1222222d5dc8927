"""What the cache's and attention's kernels must not do, checked in their source (CPU only)."""
import glob
import os
import re

import pytest

from nvfp4_expert_ffn_b200 import binding as B

SRC = sorted(glob.glob(os.path.join(os.path.dirname(os.path.abspath(B.__file__)), "csrc", "kv_*")))


@pytest.mark.parametrize("path", SRC, ids=os.path.basename)
def test_no_loads_through_the_read_only_path(path):
    """These kernels start while the one before may still write their inputs (queries, slots, page
    numbers), so those are not read-only for a kernel's whole life, which __ldg and a pointer that is
    const and __restrict__ would promise."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    assert "__ldg" not in text and "__restrict__" not in text and not re.search(r"ld\.global[.\w]*\.nc", text)


def test_a_wait_shared_out_over_a_warp_ends_with_a_warp_barrier():
    """Half of the lanes wait for one barrier, half for another: what each makes visible reaches the other
    half by the warp barrier behind the vote, which orders no memory itself."""
    text = open([p for p in SRC if p.endswith("kv_attn_tc.cu")][0]).read()
    body = re.search(r"MOE_DEV bool wait_both\(.*?\n}\n", text, re.S).group(0)
    assert body.index("wait_soon(") < body.index("__syncwarp()") < body.index("return ok;")
