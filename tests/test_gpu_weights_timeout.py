"""Failure detection of the calls on cache weights without a GPU fault: the first keys of
some segments are never loaded, their blocks' waits run out after 20 ms, ATTN_ETIMEOUT is
recorded, the segments count as empty and their tokens' weights stay. Every form: one
launch in a cluster, two launches."""
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402
import weights_ref as W  # noqa: E402
from test_gpu_weights import bits, check_weights, decode, inside, weigh, workspace  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


def untouched(w, b, n):
    """Tokens in front whose weights, NaN before, were not written; all others were, of every head."""
    still = torch.isnan(W.get_weights(w, b, 0, n))
    cut = int(still[:, 0].sum())
    assert still[:cut].all() and not still[cut:].any()
    return cut


def behind(b, cut):
    """The sequence without its first `cut` tokens (whole pages)."""
    assert cut % 16 == 0
    (c, t), = b["lens"]
    return dict(b, lens=[(c - cut, t)], table=b["table"][:, cut // 16:].contiguous())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("context", [1000, 30000])  # a cluster; merged through memory
@pytest.mark.parametrize("withheld", [1, 64])
def test_decode(cp, bf16, context, withheld):
    b = R.make_batch([(context, 0)], bf16=bf16, seed=160)
    q = torch.randn(1, 32, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(161))
    need = cp.attn_decode_weigh_workspace_bytes(1, context)
    assert (need > 0) == (context == 30000)
    ws, out = workspace(need).fill_(0), torch.full_like(q, float("nan"))
    w = torch.full_like(W.weight_pool(b), float("nan"))
    before = w.clone()
    assert cp.attn_get_device_error() == 0
    decode(cp, b, q, w.clone(), 0.0, ws=ws)  # finite partials in the workspace
    cp.attn_selftest_decode_weigh_timeout(q, b["kp"], b["vp"], w, b["table"], b["ctx"], out, context, 0.0, workspace=ws,
                                          withheld=withheld)
    assert cp.attn_get_device_error() == cp.ATTN_ETIMEOUT
    assert cp.attn_get_device_error() == 0
    if withheld == 64:
        assert torch.equal(bits(w), bits(before)) and torch.equal(out, torch.zeros_like(out))
    else:
        cut = untouched(w, b, context)
        assert 0 < cut < context
        rest = behind(b, cut)
        want, o, tol = W.weigh_reference(q, rest, before, [0], 0.0, decode=True)
        check_weights(w, before, rest, want)
        inside(out, o, tol)
    w = before.clone()
    out = decode(cp, b, q, w, 0.0, ws=ws)  # the next call is right
    want, o, tol = W.weigh_reference(q, b, before, [0], 0.0, decode=True)
    check_weights(w, before, b, want)
    inside(out, o, tol)
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("context,rows", [(1000, 8), (1000, 40), (1000, 70), (30000, 64)])
@pytest.mark.parametrize("withheld", [1, 64])
def test_weigh(cp, bf16, context, rows, withheld):
    b = R.make_batch([(context, rows)], bf16=bf16, seed=162)
    q = torch.randn(rows, 32, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(163))
    need = cp.attn_weigh_workspace_bytes(1, rows, rows, context)
    ws = workspace(need).fill_(0)
    w = torch.full_like(W.weight_pool(b), float("nan"))
    before = w.clone()
    assert cp.attn_get_device_error() == 0
    cp.attn_selftest_weigh_timeout(q, b["kp"], w, b["table"], b["ctx"], b["starts"], rows, context, 0.0, workspace=ws,
                                   withheld=withheld)
    assert cp.attn_get_device_error() == cp.ATTN_ETIMEOUT
    assert cp.attn_get_device_error() == 0
    if withheld == 64:
        assert torch.equal(bits(w), bits(before))
    elif need:  # the passes' segments differ: the rows' sums lack other keys than those that stay
        assert not torch.isnan(W.get_weights(w, b, 0, context + rows)[-1]).any()
    else:
        rest = behind(b, untouched(w, b, context + rows))
        check_weights(w, before, rest, W.weigh_reference(q, rest, before, [0], 0.0))
    w = before.clone()
    weigh(cp, b, q, w, 0.0, ws=ws)
    check_weights(w, before, b, W.weigh_reference(q, b, before, [0], 0.0))
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("bf16", [False, True])
def test_lengths_of_all_kinds(cp, bf16):
    """A few keys, none, and no rows beside a long sequence: what has nothing to load ends as ever."""
    lens = [(2000, 5), (20, 3), (0, 1), (500, 0)]
    b = R.make_batch(lens, bf16=bf16, seed=164)
    q = torch.randn(9, 32, 64, device="cuda")
    w = torch.full_like(W.weight_pool(b), float("nan"))
    before = w.clone()
    ws = workspace(cp.attn_weigh_workspace_bytes(4, 9, 5, 2000))
    cp.attn_selftest_weigh_timeout(q, b["kp"], w, b["table"], b["ctx"], b["starts"], 5, 2000, 0.0, workspace=ws, withheld=64)
    assert cp.attn_get_device_error() == cp.ATTN_ETIMEOUT
    assert torch.equal(bits(w), bits(before))
    out, ws = torch.full((4, 32, 64), float("nan"), device="cuda"), workspace(cp.attn_decode_weigh_workspace_bytes(4, 2000))
    cp.attn_selftest_decode_weigh_timeout(q[:4], b["kp"], b["vp"], w, b["table"], b["ctx"], out, 2000, 0.0,
                                          workspace=ws, withheld=64)
    assert cp.attn_get_device_error() == cp.ATTN_ETIMEOUT
    assert torch.equal(bits(w), bits(before)) and torch.equal(out, torch.zeros_like(out))
    weigh(cp, b, q, w, 0.0)
    check_weights(w, before, b, W.weigh_reference(q, b, before, [0, 0, 0, 0], 0.0))
    assert cp.attn_get_device_error() == 0
