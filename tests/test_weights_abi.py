"""Refusals of the calls on cache weights and on positions of several axes (CPU only:
the host checks return before any CUDA call) and of their binding."""
import ctypes
import os
import re

import pytest

import chunked_prefill_gqa_gb300 as cp
from chunked_prefill_gqa_gb300 import build as B

G = 0x10000  # never dereferenced
AXES = (ctypes.c_int * 32)(*[i % 3 for i in range(32)])
WRONG = (ctypes.c_int * 32)(*[i % 4 for i in range(32)])
NEGATIVE = (ctypes.c_int * 32)(*([0] * 31 + [-1]))


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def norm(**kw):
    a = dict(q=G, k=G, inType=0, qStride=2048, kStride=512, qWeight=None, kWeight=None, eps=1e-6, cosSin=G, positions=G,
             positionsStride=3, numAxes=3, axes=AXES, numPositions=8, pairing=0, qOut=G, kOut=G, kOutType=0, N=3,
             stream=None)
    a.update(kw)
    return cp.raw("attn_qk_norm_rope_axes")(*a.values())


def append(name, **kw):
    a = dict(q=None, k=G, v=G, inType=0, qStride=0, kStride=512, vStride=512, qWeight=None, kWeight=None, eps=1e-6,
             cosSin=G, positions=G, positionsStride=3, numAxes=3, axes=AXES, numPositions=8, pairing=0, qOut=None,
             kPages=G, vPages=G, table=G, ctx=G, starts=G, B=2, N=3, maxBlocks=4, numPages=9, stream=None)
    a.update(kw)
    return cp.raw(name)(*a.values())


def decode(name, **kw):
    a = dict(q=G, kPages=G, vPages=G, weights=G, table=G, ctx=G, weighed=None, decay=1.0, out=G, B=2, maxBlocks=4,
             numPages=9, maxContext=60, ws=None, wsBytes=0, stream=None)
    a.update(kw)
    return cp.raw(name)(*a.values())


def weigh(name, **kw):
    a = dict(q=G, kPages=G, weights=G, table=G, ctx=G, starts=G, weighed=None, decay=1.0, B=2, N=3, maxRows=2, maxBlocks=4,
             numPages=9, maxContext=60, ws=None, wsBytes=0, stream=None)
    a.update(kw)
    return cp.raw(name)(*a.values())


def evict(name, **kw):
    a = dict(kPages=G, vPages=G, weights=G, table=G, ctx=G, keep=G, first=1, last=2, B=2, maxBlocks=4, numPages=9,
             maxContext=60, ws=None, wsBytes=0, stream=None)
    a.update(kw)
    return cp.raw(name)(*a.values())


AXES_REFUSALS = [
    (dict(positions=None), cp.ATTN_EINVAL), (dict(axes=None), cp.ATTN_EINVAL), (dict(cosSin=None), cp.ATTN_EINVAL),
    (dict(numAxes=0), cp.ATTN_EINVAL), (dict(numAxes=5), cp.ATTN_ERANGE), (dict(numAxes=2), cp.ATTN_EINVAL),
    (dict(axes=WRONG), cp.ATTN_EINVAL), (dict(axes=NEGATIVE), cp.ATTN_EINVAL), (dict(positionsStride=-1), cp.ATTN_EINVAL),
    (dict(numPositions=0), cp.ATTN_EINVAL), (dict(positions=G + 2), cp.ATTN_EALIGN), (dict(k=None), cp.ATTN_EINVAL),
    (dict(kStride=513), cp.ATTN_EALIGN), (dict(pairing=2), cp.ATTN_EINVAL), (dict(N=-1), cp.ATTN_EINVAL),
    (dict(N=cp.MAX_TOKENS + 1), cp.ATTN_ERANGE), (dict(cosSin=G + 8), cp.ATTN_EALIGN),
    (dict(N=0, k=None, positions=None, axes=None, cosSin=None), cp.ATTN_OK),
]


@pytest.mark.parametrize("change,code", AXES_REFUSALS + [
    (dict(kOut=None), cp.ATTN_EINVAL), (dict(qOut=None), cp.ATTN_EINVAL), (dict(qStride=2044), cp.ATTN_EINVAL)])
def test_norm_rope_axes(change, code):
    assert norm(**change) == code


@pytest.mark.parametrize("name", ["attn_append_paged_axes", "attn_append_paged_axes_bf16kv"])
@pytest.mark.parametrize("change,code", AXES_REFUSALS + [
    (dict(B=-1), cp.ATTN_EINVAL), (dict(B=65536), cp.ATTN_ERANGE), (dict(v=None), cp.ATTN_EINVAL),
    (dict(table=None), cp.ATTN_EINVAL), (dict(maxBlocks=0), cp.ATTN_EINVAL), (dict(vPages=G + 8), cp.ATTN_EALIGN),
    (dict(q=G, qStride=2048), cp.ATTN_EINVAL)])
def test_append_axes(name, change, code):
    assert append(name, **change) == code


SHAPES = [
    (dict(B=-1), cp.ATTN_EINVAL), (dict(maxBlocks=0), cp.ATTN_EINVAL), (dict(numPages=0), cp.ATTN_EINVAL),
    (dict(maxContext=-1), cp.ATTN_EINVAL), (dict(B=65536), cp.ATTN_ERANGE), (dict(maxContext=65), cp.ATTN_ERANGE),
    (dict(maxBlocks=cp.MAX_TOKENS // 16 + 1), cp.ATTN_ERANGE), (dict(numPages=cp.MAX_TOKENS // 16 + 1), cp.ATTN_ERANGE),
    (dict(weights=None), cp.ATTN_EINVAL), (dict(kPages=None), cp.ATTN_EINVAL), (dict(table=None), cp.ATTN_EINVAL),
    (dict(ctx=None), cp.ATTN_EINVAL), (dict(weights=G + 8), cp.ATTN_EALIGN), (dict(kPages=G + 4), cp.ATTN_EALIGN),
    (dict(table=G + 1), cp.ATTN_EALIGN), (dict(ctx=G + 2), cp.ATTN_EALIGN),
]
DECAYS = [(dict(decay=x), cp.ATTN_EINVAL) for x in (-0.1, 1.5, float("nan"), float("inf"))]


@pytest.mark.parametrize("name", ["attn_decode_weigh_paged", "attn_decode_weigh_paged_bf16kv"])
@pytest.mark.parametrize("change,code", SHAPES + DECAYS + [
    (dict(q=None), cp.ATTN_EINVAL), (dict(out=None), cp.ATTN_EINVAL), (dict(vPages=None), cp.ATTN_EINVAL),
    (dict(q=G + 4), cp.ATTN_EALIGN), (dict(out=G + 8), cp.ATTN_EALIGN), (dict(weighed=G + 2), cp.ATTN_EALIGN),
    (dict(B=0, q=None, out=None, weights=None), cp.ATTN_OK)])
def test_decode_weigh(name, change, code):
    assert decode(name, **change) == code


@pytest.mark.parametrize("name", ["attn_weigh_paged", "attn_weigh_paged_bf16kv"])
@pytest.mark.parametrize("change,code", SHAPES + DECAYS + [
    (dict(q=None), cp.ATTN_EINVAL), (dict(starts=None), cp.ATTN_EINVAL), (dict(N=-1), cp.ATTN_EINVAL),
    (dict(N=cp.MAX_TOKENS + 1), cp.ATTN_ERANGE), (dict(maxRows=0), cp.ATTN_EINVAL), (dict(maxRows=65537), cp.ATTN_ERANGE),
    (dict(starts=G + 2), cp.ATTN_EALIGN), (dict(weighed=G + 2), cp.ATTN_EALIGN),
    (dict(B=0, q=None, weights=None), cp.ATTN_OK), (dict(N=0, q=None, weights=None), cp.ATTN_OK)])
def test_weigh(name, change, code):
    assert weigh(name, **change) == code


@pytest.mark.parametrize("name", ["attn_evict_paged", "attn_evict_paged_bf16kv"])
@pytest.mark.parametrize("change,code", SHAPES + [
    (dict(keep=None), cp.ATTN_EINVAL), (dict(vPages=None), cp.ATTN_EINVAL), (dict(first=-1), cp.ATTN_EINVAL),
    (dict(last=-1), cp.ATTN_EINVAL), (dict(first=cp.MAX_TOKENS + 1), cp.ATTN_ERANGE),
    (dict(last=cp.MAX_TOKENS + 1), cp.ATTN_ERANGE), (dict(keep=G + 2), cp.ATTN_EALIGN), (dict(vPages=G + 8), cp.ATTN_EALIGN),
    (dict(B=0, keep=None, weights=None), cp.ATTN_OK), (dict(maxContext=0, keep=None), cp.ATTN_OK)])
def test_evict(name, change, code):
    assert evict(name, **change) == code


def test_workspaces_reject_bad_sizes():
    for a in ((0, 60), (-1, 60), (65536, 60), (2, -1), (2, cp.MAX_TOKENS + 1)):
        assert cp.attn_decode_weigh_workspace_bytes(*a) == 0
        assert cp.attn_evict_workspace_bytes(*a) == 0
    for a in ((0, 3, 2, 60), (2, 0, 2, 60), (2, 3, 0, 60), (2, 3, 65537, 60), (2, 3, 2, -1), (65536, 3, 2, 60),
              (2, 3, 2, cp.MAX_TOKENS + 1), (2, cp.MAX_TOKENS + 1, 2, 60)):
        assert cp.attn_weigh_workspace_bytes(*a) == 0


def test_eviction_workspace_holds_both_lists():
    for b, n in ((1, 1), (3, 1000), (65535, 4096)):  # one block a head: lists in shared memory
        assert cp.attn_evict_workspace_bytes(b, n) == 0
    for b, n in ((1, 4097), (3, 10001), (65535, 5000), (1, cp.MAX_TOKENS)):
        # counts, and for every head a list of at most half the tokens of each kind
        assert cp.attn_evict_workspace_bytes(b, n) >= b * 8 * 4 * (1 + 2 * (n // 2))
        assert cp.attn_evict_workspace_bytes(b, n) % 4 == 0


def test_binding_checks_tensors():
    torch = pytest.importorskip("torch")
    k, ints = torch.zeros(3, 8, 64), torch.zeros(2, dtype=torch.int32)
    pages, w = torch.zeros(4, 16, 8, 64), torch.zeros(4, 8, 16)
    with pytest.raises(ValueError):
        cp.attn_qk_norm_rope_axes(None, k, torch.zeros(3, 3, dtype=torch.int32), [0] * 32, k.view(24, 64), None, k)
    with pytest.raises(ValueError):
        cp.attn_append_paged_axes(k, k, pages, pages, ints.view(2, 1), ints, ints, k.view(24, 64), ints, [0] * 32)
    with pytest.raises(ValueError):
        cp.attn_decode_weigh_paged(torch.zeros(2, 32, 64), pages, pages, w, ints.view(2, 1), ints, torch.zeros(2, 32, 64), 10)
    with pytest.raises(ValueError):
        cp.attn_weigh_paged(torch.zeros(3, 32, 64), pages, w, ints.view(2, 1), ints, torch.zeros(3, dtype=torch.int32), 2, 10)
    with pytest.raises(ValueError):
        cp.attn_evict_paged(pages, pages, w, ints.view(2, 1), ints, ints, 10)
    with pytest.raises(TypeError):
        cp.attn_evict_paged(pages.numpy(), pages, w, ints.view(2, 1), ints, ints, 10)


def test_header_constants_agree_with_the_binding():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                             "attn_prefill.h")).read()
    defs = dict(re.findall(r"#define (ATTN_\w+)\s+(-?\d+)", text))
    assert (int(defs["ATTN_ROPE_AXES"]), int(defs["ATTN_WEIGH_ROWS"])) == (cp.ROPE_AXES, cp.WEIGH_ROWS)
