"""Refusals of the drafted-tree failure-path test (CPU only: the host checks return
before any CUDA call)."""
import pytest

import chunked_prefill_gqa_gb300 as cp
from chunked_prefill_gqa_gb300 import build

G = 0x10000  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.mark.parametrize("change,code", [
    (dict(B=0), cp.ATTN_EINVAL), (dict(N=0), cp.ATTN_EINVAL), (dict(withheld=0), cp.ATTN_EINVAL),
    (dict(pageType=2), cp.ATTN_EINVAL), (dict(q=None), cp.ATTN_EINVAL), (dict(maxRows=65), cp.ATTN_ERANGE),
    (dict(maxContext=65), cp.ATTN_ERANGE), (dict(out=G + 4), cp.ATTN_EALIGN),
])
def test_refusals(change, code):
    a = dict(q=G, kPages=G, vPages=G, pageType=0, table=G, ctx=G, starts=G, masks=None, out=G, B=2, N=3, maxRows=2,
             maxBlocks=4, numPages=9, maxContext=60, numSplits=0, withheld=1, ws=None, wsBytes=0, stream=None)
    a.update(change)
    assert cp.raw("attn_selftest_tree_timeout")(*a.values()) == code
