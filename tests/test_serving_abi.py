"""Refusals of the serving-step calls (CPU only: the host checks return before
any CUDA call) and of their binding."""
import ctypes

import pytest

import chunked_prefill_gqa_gb300 as cp
from chunked_prefill_gqa_gb300 import build as B

G = 0x10000  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def norm(**kw):
    a = dict(q=G, k=G, inType=0, qStride=2048, kStride=512, qWeight=None, kWeight=None, eps=1e-6, cosSin=G, positions=G,
             numPositions=8, pairing=0, qOut=G, kOut=G, kOutType=0, N=3, stream=None)
    a.update(kw)
    return cp.raw("attn_qk_norm_rope")(*a.values())


def append(name="attn_append_paged", **kw):
    a = dict(q=None, k=G, v=G, inType=0, qStride=0, kStride=512, vStride=512, qWeight=None, kWeight=None, eps=1e-6,
             cosSin=None, positions=None, numPositions=0, pairing=0, qOut=None, kPages=G, vPages=G, table=G, ctx=G,
             starts=G, B=2, N=3, maxBlocks=4, numPages=9, stream=None)
    a.update(kw)
    return cp.raw(name)(*a.values())


def tree(name="attn_tree_paged", **kw):
    a = dict(q=G, kPages=G, vPages=G, table=G, ctx=G, starts=G, masks=None, out=G, B=2, N=3, maxRows=2, maxBlocks=4,
             numPages=9, maxContext=60, numSplits=0, ws=None, wsBytes=0, stream=None)
    a.update(kw)
    return cp.raw(name)(*a.values())


def compact(name="attn_compact_paged", **kw):
    a = dict(kPages=G, vPages=G, table=G, ctx=G, keep=G, counts=G, B=2, maxKeep=3, maxRows=4, maxBlocks=4, numPages=9,
             stream=None)
    a.update(kw)
    return cp.raw(name)(*a.values())


def test_rope_table():
    f = cp.raw("attn_rope_table")
    freq = (ctypes.c_double * 32)()
    assert f(freq, G, -1, None) == cp.ATTN_EINVAL
    assert f(freq, G, cp.MAX_TOKENS + 1, None) == cp.ATTN_ERANGE
    assert f(None, G, 4, None) == cp.ATTN_EINVAL
    assert f(freq, None, 4, None) == cp.ATTN_EINVAL
    assert f(freq, G + 4, 4, None) == cp.ATTN_EALIGN
    assert f(None, None, 0, None) == cp.ATTN_OK


@pytest.mark.parametrize("change,code", [
    (dict(N=-1), cp.ATTN_EINVAL), (dict(N=cp.MAX_TOKENS + 1), cp.ATTN_ERANGE),
    (dict(k=None), cp.ATTN_EINVAL), (dict(kOut=None), cp.ATTN_EINVAL), (dict(qOut=None), cp.ATTN_EINVAL),
    (dict(inType=2), cp.ATTN_EINVAL), (dict(kOutType=-1), cp.ATTN_EINVAL), (dict(pairing=2), cp.ATTN_EINVAL),
    (dict(eps=-1.0), cp.ATTN_EINVAL), (dict(eps=float("nan")), cp.ATTN_EINVAL), (dict(eps=float("inf")), cp.ATTN_EINVAL),
    (dict(numPositions=0), cp.ATTN_EINVAL), (dict(positions=None), cp.ATTN_EINVAL),
    (dict(kStride=511), cp.ATTN_EINVAL), (dict(qStride=2044), cp.ATTN_EINVAL), (dict(kStride=-512), cp.ATTN_EINVAL),
    (dict(kStride=513), cp.ATTN_EALIGN), (dict(qStride=2050), cp.ATTN_EALIGN),
    (dict(inType=1, kStride=516), cp.ATTN_EALIGN),
    (dict(q=G + 8), cp.ATTN_EALIGN), (dict(k=G + 4), cp.ATTN_EALIGN), (dict(qWeight=G + 4), cp.ATTN_EALIGN),
    (dict(cosSin=G + 8), cp.ATTN_EALIGN), (dict(positions=G + 2), cp.ATTN_EALIGN), (dict(kOut=G + 2), cp.ATTN_EALIGN),
    (dict(N=0, q=None, k=None, kOut=None, qOut=None, positions=None), cp.ATTN_OK),
])
def test_norm_rope(change, code):
    assert norm(**change) == code


@pytest.mark.parametrize("name", ["attn_append_paged", "attn_append_paged_bf16kv"])
@pytest.mark.parametrize("change,code", [
    (dict(B=-1), cp.ATTN_EINVAL), (dict(N=-1), cp.ATTN_EINVAL), (dict(maxBlocks=0), cp.ATTN_EINVAL),
    (dict(numPages=0), cp.ATTN_EINVAL), (dict(B=65536), cp.ATTN_ERANGE), (dict(N=cp.MAX_TOKENS + 1), cp.ATTN_ERANGE),
    (dict(maxBlocks=cp.MAX_TOKENS // 16 + 1), cp.ATTN_ERANGE), (dict(numPages=cp.MAX_TOKENS // 16 + 1), cp.ATTN_ERANGE),
    (dict(v=None), cp.ATTN_EINVAL), (dict(vPages=None), cp.ATTN_EINVAL), (dict(kPages=None), cp.ATTN_EINVAL),
    (dict(table=None), cp.ATTN_EINVAL), (dict(ctx=None), cp.ATTN_EINVAL), (dict(starts=None), cp.ATTN_EINVAL),
    (dict(q=G, qStride=2048), cp.ATTN_EINVAL), (dict(cosSin=G), cp.ATTN_EINVAL), (dict(vStride=500), cp.ATTN_EINVAL),
    (dict(vStride=514), cp.ATTN_EALIGN), (dict(v=G + 4), cp.ATTN_EALIGN), (dict(vPages=G + 8), cp.ATTN_EALIGN),
    (dict(table=G + 1), cp.ATTN_EALIGN), (dict(pairing=7), cp.ATTN_EINVAL),
    (dict(N=0, k=None, v=None, table=None), cp.ATTN_OK), (dict(B=0, table=None, starts=None), cp.ATTN_OK),
])
def test_append(name, change, code):
    assert append(name, **change) == code


@pytest.mark.parametrize("name", ["attn_tree_paged", "attn_tree_paged_bf16kv"])
@pytest.mark.parametrize("change,code", [
    (dict(B=-1), cp.ATTN_EINVAL), (dict(maxRows=0), cp.ATTN_EINVAL), (dict(maxContext=-1), cp.ATTN_EINVAL),
    (dict(numSplits=-1), cp.ATTN_EINVAL), (dict(maxRows=65), cp.ATTN_ERANGE), (dict(maxContext=65), cp.ATTN_ERANGE),
    (dict(B=65536), cp.ATTN_ERANGE), (dict(q=None), cp.ATTN_EINVAL), (dict(out=None), cp.ATTN_EINVAL),
    (dict(vPages=None), cp.ATTN_EINVAL), (dict(starts=None), cp.ATTN_EINVAL), (dict(q=G + 4), cp.ATTN_EALIGN),
    (dict(masks=G + 4), cp.ATTN_EALIGN), (dict(starts=G + 2), cp.ATTN_EALIGN),
    (dict(B=0, q=None, out=None), cp.ATTN_OK), (dict(N=0, q=None, out=None), cp.ATTN_OK),
])
def test_tree(name, change, code):
    assert tree(name, **change) == code


def test_tree_workspace_rejects_bad_sizes():
    for a in ((0, 3, 2, 60, 0), (2, 0, 2, 60, 0), (2, 3, 0, 60, 0), (2, 3, 65, 60, 0), (2, 3, 2, -1, 0),
              (2, 3, 2, 60, -1), (70000, 3, 2, 60, 0), (2, 3, 2, cp.MAX_TOKENS + 1, 0)):
        assert cp.attn_tree_workspace_bytes(*a) == 0


@pytest.mark.parametrize("name", ["attn_compact_paged", "attn_compact_paged_bf16kv"])
@pytest.mark.parametrize("change,code", [
    (dict(B=-1), cp.ATTN_EINVAL), (dict(maxKeep=-1), cp.ATTN_EINVAL), (dict(maxRows=0), cp.ATTN_EINVAL),
    (dict(maxRows=65), cp.ATTN_ERANGE), (dict(maxKeep=5), cp.ATTN_ERANGE), (dict(keep=None), cp.ATTN_EINVAL),
    (dict(counts=None), cp.ATTN_EINVAL), (dict(kPages=None), cp.ATTN_EINVAL), (dict(keep=G + 2), cp.ATTN_EALIGN),
    (dict(kPages=G + 8), cp.ATTN_EALIGN), (dict(B=0, keep=None), cp.ATTN_OK), (dict(maxKeep=0, keep=None), cp.ATTN_OK),
])
def test_compact(name, change, code):
    assert compact(name, **change) == code


def test_binding_checks_tensors():
    torch = pytest.importorskip("torch")
    k = torch.zeros(3, 8, 64)
    with pytest.raises(ValueError):  # on the CPU
        cp.attn_qk_norm_rope(None, k, None, None, None, k)
    with pytest.raises(ValueError):  # neither fp32 nor bf16
        cp.attn_qk_norm_rope(None, k.double(), None, None, None, k)
    with pytest.raises(TypeError):
        cp.attn_qk_norm_rope(None, k.numpy(), None, None, None, k)
    pages, ints = torch.zeros(4, 16, 8, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        cp.attn_append_paged(k, k, pages, pages, ints.view(2, 1), ints, ints)
    with pytest.raises(ValueError):
        cp.attn_tree_paged(torch.zeros(3, 32, 64), pages, pages, ints.view(2, 1), ints, ints, None,
                           torch.zeros(3, 32, 64), 2, 10)
    with pytest.raises(ValueError):
        cp.attn_compact_paged(pages, pages, ints.view(2, 1), ints, ints.view(2, 1), ints, 4)
    with pytest.raises(ValueError):
        cp.attn_rope_table(torch.zeros(4, 64))


def test_header_constants_agree_with_the_binding():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                             "attn_prefill.h")).read()
    defs = dict(re.findall(r"#define (ATTN_\w+)\s+(-?\d+)", text))
    assert int(defs["ATTN_TREE_ROWS"]) == cp.TREE_ROWS
    assert (int(defs["ATTN_F32"]), int(defs["ATTN_BF16"])) == (cp.F32, cp.BF16)
    assert (int(defs["ATTN_ROPE_HALVES"]), int(defs["ATTN_ROPE_PAIRS"])) == (cp.ROPE_HALVES, cp.ROPE_PAIRS)
