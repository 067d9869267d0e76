"""The failure test of a window in two launches, whose passes cut the keys differently: the
rows' sums lack the rows pass's first segment, the weights of the keys pass's first
segment stay, and every other token's weight is what the rows' remaining sums give to it."""
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402
import weights_ref as W  # noqa: E402
from test_gpu_weights import check_weights, weigh, workspace  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


def reference(q, b, summed, first):
    """(weights, tolerance) of tokens `first` and on, rows' sums over the tokens from `summed` on."""
    (c, t), = b["lens"]
    n = c + t
    k, tok = R.gather(b["kp"], b["table"][0], n), torch.arange(n, device="cuda")
    seen = tok[None] <= (c + torch.arange(t, device="cuda"))[:, None]
    w, tol = torch.zeros(n, 8, dtype=torch.float64, device="cuda"), torch.zeros(n, 8, dtype=torch.float64, device="cuda")
    for h in range(32):
        _, rel = W.softmax_reference(q[:, h].double(), k[:, h // 4], seen)  # over all keys: no smaller than over some
        s = (q[:, h].double() @ k[:, h // 4].T / 8).masked_fill(~seen, float("-inf"))
        total = torch.logsumexp(s.masked_fill(tok < summed, float("-inf")), -1, keepdim=True)
        p = torch.exp(s - total).masked_fill(torch.isneginf(total), 0.0)  # no key left: such a row gives nothing
        w[:, h // 4] += p.sum(0)
        tol[:, h // 4] += (p * rel).sum(0)
    tol += (70 + t / 32) * 2.0 ** -24 * w
    return w[first:], tol[first:]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("context,rows", [(1000, 70), (30000, 64), (0, 1500), (500, 400)])
def test_what_the_other_segments_give(cp, bf16, context, rows):
    b = R.make_batch([(context, rows)], bf16=bf16, seed=51)
    q = torch.randn(rows, 32, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(52))
    need = cp.attn_weigh_workspace_bytes(1, rows, rows, context)
    assert need > 0 and need % (rows * 32 * 8) == 0
    splits, n = need // (rows * 32 * 8), context + rows  # a float2 for each row, head and segment of the rows pass
    summed = -(-(-(-n // splits)) // 128) * 128
    w = torch.full_like(W.weight_pool(b), float("nan"))
    before = w.clone()
    ws = workspace(need)
    assert cp.attn_get_device_error() == 0
    cp.attn_selftest_weigh_timeout(q, b["kp"], w, b["table"], b["ctx"], b["starts"], rows, context, 0.0, workspace=ws,
                                   withheld=1)
    assert cp.attn_get_device_error() == cp.ATTN_ETIMEOUT
    got = W.get_weights(w, b, 0, n)
    cut = int(torch.isnan(got[:, 0]).sum())
    assert cut % 128 == 0 and cut > 0 and got[:cut].isnan().all() and not got[cut:].isnan().any()
    rest = dict(b, lens=[(context - cut, rows)], table=b["table"][:, cut // 16:].contiguous())
    if context < cut:  # (the rows' own tokens are what is left)
        rest["lens"] = [(n - cut, 0)]
    check_weights(w, before, rest, [reference(q, b, summed, cut)])
    w = before.clone()
    weigh(cp, b, q, w, 0.0, ws=ws)
    check_weights(w, before, b, W.weigh_reference(q, b, before, [0], 0.0))
    assert cp.attn_get_device_error() == 0
