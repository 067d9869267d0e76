"""Refusals of the failure-path tests of the calls on cache weights (CPU only: the host
checks return before any CUDA call)."""
import pytest

import chunked_prefill_gqa_gb300 as cp
from chunked_prefill_gqa_gb300 import build

G = 0x10000  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


SHARED = [(dict(B=0), cp.ATTN_EINVAL), (dict(withheld=0), cp.ATTN_EINVAL), (dict(pageType=2), cp.ATTN_EINVAL),
          (dict(q=None), cp.ATTN_EINVAL), (dict(weights=None), cp.ATTN_EINVAL), (dict(decay=1.5), cp.ATTN_EINVAL),
          (dict(maxContext=65), cp.ATTN_ERANGE), (dict(weights=G + 4), cp.ATTN_EALIGN)]


@pytest.mark.parametrize("change,code", SHARED + [(dict(out=None), cp.ATTN_EINVAL)])
def test_decode_refusals(change, code):
    a = dict(q=G, kPages=G, vPages=G, pageType=0, weights=G, table=G, ctx=G, weighed=None, decay=1.0, out=G, B=2, maxBlocks=4,
             numPages=9, maxContext=60, withheld=1, ws=None, wsBytes=0, stream=None)
    a.update(change)
    assert cp.raw("attn_selftest_decode_weigh_timeout")(*a.values()) == code


@pytest.mark.parametrize("change,code", SHARED + [(dict(N=0), cp.ATTN_EINVAL), (dict(maxRows=65537), cp.ATTN_ERANGE)])
def test_weigh_refusals(change, code):
    a = dict(q=G, kPages=G, pageType=0, weights=G, table=G, ctx=G, starts=G, weighed=None, decay=1.0, B=2, N=3, maxRows=2,
             maxBlocks=4, numPages=9, maxContext=60, withheld=1, ws=None, wsBytes=0, stream=None)
    a.update(change)
    assert cp.raw("attn_selftest_weigh_timeout")(*a.values()) == code
