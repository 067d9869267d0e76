"""Failure detection of the drafted-tree kernels without a GPU fault: the first keys of
some segments are never loaded, their blocks' waits run out after 20 ms, ATTN_ETIMEOUT
is recorded, and the segments count as empty. Every kernel, as one segment, as a cluster
(whose blocks all have to meet, whatever failed) and merged through memory."""
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402
from test_gpu_tree import check, queries, run  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


def without_first(b, cut, q, masks):
    """The reference over the keys behind the first `cut` (whole pages) of one sequence."""
    (c, t), = b["lens"]
    return R.tree_reference(q, dict(b, lens=[(c - cut, t)], table=b["table"][:, cut // 16:]), masks)


@pytest.mark.parametrize("bf16,rows", [(False, 3), (False, 20), (True, 3), (True, 7), (True, 20)])
@pytest.mark.parametrize("splits", [1, 4, 20])
@pytest.mark.parametrize("withheld", [1, 64])
def test_an_expired_wait_is_reported_and_its_segment_is_empty(cp, bf16, rows, splits, withheld):
    context = 2900
    lens = [(context, rows)]
    b = R.make_batch(lens, bf16=bf16, seed=150)
    masks, q = R.tree_masks(lens, seed=1), queries(rows, seed=151)
    m = torch.from_numpy(masks).cuda()
    need = cp.attn_tree_workspace_bytes(1, rows, rows, context, splits)
    assert (need > 0) == (splits == 20)
    ws = torch.full((max(need, 16),), 0, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"))
    args = (q, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], m, out, rows, context, splits, ws)
    assert cp.attn_get_device_error() == 0
    (cp.attn_tree_paged_bf16kv if bf16 else cp.attn_tree_paged)(*args)  # finite partials in the workspace
    want, tol = R.tree_reference(q, b, masks)
    check(out, want, tol)
    out.fill_(float("nan"))
    cp.attn_selftest_tree_timeout(*args, withheld=withheld)
    assert cp.attn_get_device_error() == cp.ATTN_ETIMEOUT
    assert cp.attn_get_device_error() == 0
    if splits == 1:
        assert torch.isnan(out).all()  # left unwritten
    elif withheld == 64:
        assert torch.equal(out, torch.zeros_like(out))
    else:
        cut = ((context + rows + splits - 1) // splits + 127) // 128 * 128
        check(out, *without_first(b, cut, q, masks))
    check(run(cp, b, q, masks, bf16, splits), want, tol)  # the next call is right
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("bf16,rows", [(False, 3), (False, 20), (True, 3), (True, 7), (True, 20)])
@pytest.mark.parametrize("splits", [1, 4, 20])
def test_sequences_shorter_than_their_segments(cp, bf16, rows, splits):
    """A few tiles, one tile and no context beside a long sequence: a block's loads may
    all have been issued, and its warps have nothing else to wait for, when the wait for
    the first runs out."""
    context = 2900
    lens = [(context, rows), (300, rows), (20, rows), (0, rows)]
    b = R.make_batch(lens, bf16=bf16, seed=152)
    masks, q = R.tree_masks(lens, seed=2), queries(4 * rows, seed=153)
    need = cp.attn_tree_workspace_bytes(4, 4 * rows, rows, context, splits)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"))
    assert cp.attn_get_device_error() == 0
    cp.attn_selftest_tree_timeout(q, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"],
                                  torch.from_numpy(masks).cuda(), out, rows, context, splits, ws, withheld=64)
    assert cp.attn_get_device_error() == cp.ATTN_ETIMEOUT
    if splits == 4:
        assert torch.equal(out, torch.zeros_like(out))
    else:  # sequences in one segment are left unwritten, merged ones have no keys
        assert (torch.isnan(out) | (out == 0)).all() and torch.isnan(out[2 * rows:]).all()
    check(run(cp, b, q, masks, bf16, splits), *R.tree_reference(q, b, masks))
    assert cp.attn_get_device_error() == 0
