"""Lengths that a kernel in front of the attention has just written: a serving loop
advances contextLens and rowStart on the device between its steps."""
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


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows,splits", [(3, 1), (3, 6), (3, 24), (7, 24), (20, 24)])
def test_lengths_written_by_the_kernel_before(cp, captured, bf16, rows, splits):
    """Calls one after another in a stream, each right behind the copies that set its
    lengths: contexts and rows grow and shrink, and so do the segments that a merge
    through memory counts. Beside them an append, which waits and starts in the same way."""
    full = [(2900, rows), (1800, rows)]
    b = R.make_batch(full, bf16=bf16, seed=140)
    n, q = 2 * rows, queries(2 * rows, seed=141)
    lens = [[(2900, rows), (1800, rows)], [(10, 1), (1500, rows)], [(2900, rows), (0, 1)], [(130, 2), (2, 2)],
            [(2800, 1), (1799, rows)]]
    ctxs = [torch.tensor([c for c, _ in x], dtype=torch.int32, device="cuda") for x in lens]
    starts = [torch.tensor([0, x[0][1], x[0][1] + x[1][1]], dtype=torch.int32, device="cuda") for x in lens]
    need = cp.attn_tree_workspace_bytes(2, n, rows, 2900, splits)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.full_like(q, float("nan")) for _ in lens]
    call = cp.attn_tree_paged_bf16kv if bf16 else cp.attn_tree_paged
    append = cp.attn_append_paged_bf16kv if bf16 else cp.attn_append_paged
    spare = R.make_batch(full, bf16=bf16, seed=142)
    k = torch.randn(n, 8, 64, device="cuda")
    slow = torch.randn(2048, 2048, device="cuda")

    def steps():
        for c, s, o in zip(ctxs, starts, outs):
            x = slow @ slow  # so that what follows is enqueued while this runs
            b["ctx"].copy_(c).add_((x[0, 0] * 0).int())
            b["starts"].copy_(s)
            append(k, k, spare["kp"], spare["vp"], b["table"], b["ctx"], b["starts"])
            call(q, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], None, o, rows, 2900, splits, ws)

    if captured:
        steps()
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(float("nan"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            steps()
        g.replay()
    else:
        steps()
    torch.cuda.synchronize()
    for x, o in zip(lens, outs):
        now = dict(b, lens=x, n=sum(t for _, t in x))
        want, tol = R.tree_reference(q[:now["n"]], now, R.tree_masks(x, "chain"))
        check(o[:now["n"]], want, tol)
        assert torch.isnan(o[now["n"]:]).all()
    assert cp.attn_get_device_error() == 0
