"""The workspace of the drafted-tree attention over the life of a server: fewer
sequences may be cut into more segments, so a smaller batch may want more of it."""
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402
from test_gpu_tree import check, queries  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows,context", [(1, 4000), (6, 4000), (32, 12000)])
@pytest.mark.parametrize("share", [0.0, 0.4, 1.0])
def test_a_batch_that_shrinks_on_one_workspace(cp, bf16, rows, context, share):
    """One buffer for 16 sequences, 4 and 1: none, some, or as much as any of
    them asks for. Every call runs and is right, with segments that fit."""
    sizes = (16, 4, 1)
    asked = [cp.attn_tree_workspace_bytes(B, B * rows, rows, context) for B in sizes]
    assert max(asked) > asked[0], "the shapes of this test no longer ask for more as the batch shrinks"
    room = int(max(asked) * share) // 16 * 16
    buf = torch.full((room + 64,), 0x7f, dtype=torch.uint8, device="cuda")
    ws = buf[:room] if room else None
    call = cp.attn_tree_paged_bf16kv if bf16 else cp.attn_tree_paged
    for B in sizes:
        lens = [(context - 37 * b, rows) for b in range(B)]
        batch = R.make_batch(lens, bf16=bf16, seed=B)
        masks, q = R.tree_masks(lens, seed=B), queries(batch["n"], seed=B)
        out = torch.full_like(q, float("nan"))
        call(q, batch["kp"], batch["vp"], batch["table"], batch["ctx"], batch["starts"],
             torch.from_numpy(masks).cuda(), out, rows, context, workspace=ws)
        check(out, *R.tree_reference(q, batch, masks))
        assert (buf[room:] == 0x7f).all(), "written past the workspace"
    assert cp.attn_get_device_error() == 0


def test_a_stated_number_of_segments_still_needs_its_workspace(cp):
    lens = [(3000, 2)]
    b, q = R.make_batch(lens, seed=73), queries(2)
    out = torch.empty_like(q)
    with pytest.raises(cp.AttnError) as e:
        cp.attn_tree_paged(q, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], None, out, 2, 3000, num_splits=20)
    assert e.value.code == cp.ATTN_ESPACE
