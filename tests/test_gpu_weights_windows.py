"""Windows of many row tiles (attn_weigh_paged, both page types): prompts weighed whole, and
segments of keys that a window's first row tiles do not see, against the plain form in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402
import weights_ref as W  # noqa: E402
from test_gpu_weights import check_weights, ints, weigh  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


# Two row tiles, whose first one does not see the last segment; then three and more.
WINDOWS = {
    "segment behind the first tile": [(90, 64)], "segment at its end": [(96, 64)], "one row in the second": [(127, 33)],
    "two, and an empty segment": [(60, 64)], "two of several": [(0, 64), (100, 64), (2000, 50)],
    "three": [(0, 70), (128, 65)], "ten": [(0, 300), (500, 200)], "a prompt": [(0, 2000), (300, 900), (40, 0)],
    "a long prompt": [(0, 5000), (700, 2500)],
}


@pytest.mark.parametrize("name", WINDOWS)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("bound", [None, 3000, 30000])
def test_row_tiles_without_keys(cp, name, bf16, bound):
    lens = WINDOWS[name]
    bound = bound and max([bound] + [c for c, _ in lens])
    b = R.make_batch(lens, bf16=bf16, seed=21, extra_blocks=(bound or 0) // 16 + 1)
    weighed = [c // 2 for c, _ in lens]
    w = W.weight_pool(b, known=weighed)
    q = torch.randn(b["n"], 32, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(22))
    before = w.clone()
    weigh(cp, b, q, w, 0.9, ints(weighed), bound=bound)
    assert cp.attn_get_device_error() == 0
    check_weights(w, before, b, W.weigh_reference(q, b, before, weighed, 0.9))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens", [[(90, 64)], [(0, 64)], [(0, 300)], [(0, 2000)]])
def test_lost_segments_of_such_windows(cp, bf16, lens):
    """The failure test's waits run out in segments that only later row tiles see, too; the next call is right."""
    b = R.make_batch(lens, bf16=bf16, seed=23)
    n, (c, t) = b["n"], lens[0]
    q = torch.randn(n, 32, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(24))
    w = torch.full_like(W.weight_pool(b), float("nan"))
    before = w.clone()
    ws = torch.zeros(max(16, cp.attn_weigh_workspace_bytes(1, n, t, c)), dtype=torch.uint8, device="cuda")
    assert cp.attn_get_device_error() == 0
    cp.attn_selftest_weigh_timeout(q, b["kp"], w, b["table"], b["ctx"], b["starts"], t, c, 0.0, workspace=ws, withheld=64)
    assert cp.attn_get_device_error() == cp.ATTN_ETIMEOUT
    assert torch.equal(w.view(torch.int32), before.view(torch.int32))
    weigh(cp, b, q, w, 0.0, ws=ws)
    assert cp.attn_get_device_error() == 0
    check_weights(w, before, b, W.weigh_reference(q, b, before, [0], 0.0))
