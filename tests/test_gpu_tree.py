"""attn_tree_paged and attn_tree_paged_bf16kv (drafted rows over a paged cache)
against the plain form in 64 bits, element by element, and the whole serving step."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


def queries(n, seed=0, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, 32, 64, generator=g, device="cuda") * scale


def run(cp, b, q, masks, bf16, splits=0, max_rows=None, max_context=None, pad=0, stream=None):
    """The call on poisoned outputs and a poisoned workspace, with guard rows behind."""
    mr, mc = max_rows or b["max_rows"], b["max_context"] if max_context is None else max_context
    n = b["n"] + pad
    if pad:
        q = torch.cat([q, torch.full((pad, 32, 64), float("nan"), device="cuda")])
        masks = None if masks is None else np.concatenate([masks, np.full(pad, -1)])
    buf = torch.full((n + 2, 32, 64), float("nan"), device="cuda")
    out = buf[1:n + 1]
    m = None if masks is None else torch.from_numpy(masks).cuda()
    need = cp.attn_tree_workspace_bytes(b["ctx"].shape[0], n, mr, mc, splits)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None
    call = cp.attn_tree_paged_bf16kv if bf16 else cp.attn_tree_paged
    call(q, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], m, out, mr, mc, num_splits=splits, workspace=ws,
         stream=stream)
    torch.cuda.synchronize()
    assert torch.isnan(buf[0]).all() and torch.isnan(buf[b["n"] + 1:]).all(), "rows of no sequence were written"
    return out[:b["n"]]


def check(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() / tol.clamp(min=1e-300)).max()))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 33, 64])
@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 129, 1000])
def test_sizes(cp, bf16, rows, ctx):
    lens = [(ctx, rows)]
    b = R.make_batch(lens, bf16=bf16, seed=rows * 7 + ctx)
    q, masks = queries(rows, seed=ctx), R.tree_masks(lens, seed=rows)
    check(run(cp, b, q, masks, bf16), *R.tree_reference(q, b, masks))
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows", [5, 8, 9, 16, 17, 31, 33, 64])
@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 129, 1000])
@pytest.mark.parametrize("splits", [1, 5])
def test_sizes_below_a_long_bound(cp, bf16, rows, ctx, splits):
    """The kernels of calls that allow long contexts, at the short ones."""
    lens = [(ctx, rows)]
    b = R.make_batch(lens, bf16=bf16, seed=rows * 7 + ctx, extra_blocks=1100)
    q, masks = queries(rows, seed=ctx), R.tree_masks(lens, seed=rows)
    check(run(cp, b, q, masks, bf16, splits, max_context=17000), *R.tree_reference(q, b, masks))
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", ["tree", "chain", "self", "empty", "mixed", "null"])
@pytest.mark.parametrize("splits", [0, 1, 3, 8, 64])
def test_ragged_batch_masks_and_splits(cp, bf16, kind, splits):
    lens = [(700, 5), (0, 12), (33, 0), (1, 1), (2500, 12), (128, 7), (0, 1), (255, 2)]
    b = R.make_batch(lens, bf16=bf16, seed=11)
    masks = R.tree_masks(lens, "chain" if kind == "null" else kind, seed=12)
    q = queries(b["n"], seed=13)
    got = run(cp, b, q, None if kind == "null" else masks, bf16, splits, pad=3)
    check(got, *R.tree_reference(q, b, masks))
    if kind == "empty":  # no context and no drafted row to see
        assert torch.equal(got[5:17], torch.zeros_like(got[5:17]))
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("bf16", [False, True])
def test_loose_bounds_change_nothing_but_the_segments(cp, bf16):
    """maxRows and maxContext above what the batch has (64 and the whole table)."""
    lens = [(300, 3), (77, 6)]
    b = R.make_batch(lens, bf16=bf16, seed=21, extra_blocks=500)
    masks, q = R.tree_masks(lens, seed=2), queries(9, seed=3)
    check(run(cp, b, q, masks, bf16, max_rows=64, max_context=8000), *R.tree_reference(q, b, masks))


LOOSE = {
    "ragged": [((137 * i) % 900, (11 * i) % 65) for i in range(40)],
    "short": [(3 * i, 1 + i % 7) for i in range(20)],
    "one long": [(0, 0)] * 9 + [(9000, 33)] + [(1, 1), (0, 2)] * 6,
    "alike": [(1024, 32)] * 24,
}


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", ["tree", "empty", "mixed"])
@pytest.mark.parametrize("batch", list(LOOSE))
def test_batches_far_below_their_bounds(cp, bf16, kind, batch):
    """64 rows and 30000 tokens as bounds: most segments are empty, and a sequence
    may end in any of them."""
    lens = LOOSE[batch]
    b = R.make_batch(lens, bf16=bf16, seed=17, extra_blocks=2000)
    masks, q = R.tree_masks(lens, kind, seed=18), queries(b["n"], seed=19)
    got = run(cp, b, q, masks, bf16, max_rows=64, max_context=30000, pad=2)
    check(got, *R.tree_reference(q, b, masks))
    again = run(cp, b, q, masks, bf16, max_rows=64, max_context=30000)
    assert torch.equal(got, again)
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows", [1, 6, 20])
def test_long_context(cp, bf16, rows):
    lens = [(40000, rows), (9000, rows)]
    b = R.make_batch(lens, bf16=bf16, seed=31)
    masks, q = R.tree_masks(lens, seed=2), queries(2 * rows, seed=3)
    check(run(cp, b, q, masks, bf16), *R.tree_reference(q, b, masks))


@pytest.mark.parametrize("bf16", [False, True])
def test_one_row_a_sequence_is_a_decode_step(cp, bf16):
    """Against attn_decode_paged on the same fp32 cache (a chain of one row sees
    its context and itself)."""
    lens = [(999, 1), (0, 1), (4095, 1), (64, 1)]
    b = R.make_batch(lens, bf16=bf16, seed=41)
    q = queries(4, seed=1)
    got = run(cp, b, q, None, bf16)
    k, v = b["kp"].float(), b["vp"].float()
    out, ctx = torch.empty_like(q), b["ctx"] + 1
    need = cp.attn_decode_workspace_bytes(4, 4096, 0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    cp.attn_decode_paged(q, k, v, b["table"], ctx, out, 4096, 0, ws)
    _, tol = R.tree_reference(q, b, R.tree_masks(lens, "chain"))
    check(got, out.double(), 2 * tol)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows", [4, 7, 30])
def test_planted_scores(cp, bf16, rows):
    """Scores of 128 and -128 next to small ones, rising along the keys, so the
    reference maximum moves in late pages; and a row of equal scores."""
    lens = [(530, rows)]
    b = R.make_batch(lens, bf16=bf16, seed=51)
    for t in (5, 100, 400, 529, 531):
        b["kp"][b["table"][0, t // 16].long(), t % 16] = 4.0 if t % 2 else -4.0
    q = queries(rows, seed=4)
    q[0] = 4.0
    q[1] = 0.0
    masks = R.tree_masks(lens, "chain")
    check(run(cp, b, q, masks, bf16), *R.tree_reference(q, b, masks))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("rows", [3, 8, 24])
def test_what_a_row_does_not_see_has_no_influence(cp, bf16, value, rows):
    """A drafted row whose key and value are not finite reaches the rows that see
    it and no other."""
    lens = [(70, rows)]
    b = R.make_batch(lens, bf16=bf16, seed=61)
    masks = R.tree_masks(lens, "self")
    masks[2] = 0b101
    q = queries(rows, seed=5)
    want, tol = R.tree_reference(q, b, masks)  # row 0 is poisoned after this
    kv = b["kp"].clone(), b["vp"].clone()
    page, slot = b["table"][0, 70 // 16].long(), 70 % 16
    b["vp"][page, slot, :, 5] = value
    got = run(cp, b, q, masks, bf16)
    blind = [i for i in range(rows) if i not in (0, 2)]
    check(got[blind], want[blind], tol[blind])
    assert not torch.isfinite(got[[0, 2]][:, :, 5]).any()
    rest = [d for d in range(64) if d != 5]
    check(got[[0, 2]][:, :, rest], want[[0, 2]][:, :, rest], tol[[0, 2]][:, :, rest])
    b["kp"], b["vp"] = kv
    b["kp"][page, slot] = value
    got = run(cp, b, q, masks, bf16)
    check(got[blind], want[blind], tol[blind])


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows", [4, 5, 20])
@pytest.mark.parametrize("splits", [1, 3, 20])
def test_a_query_that_is_nan_stays_in_its_row(cp, bf16, rows, splits):
    lens = [(3000, rows)]
    b = R.make_batch(lens, bf16=bf16, seed=62)
    masks, q = R.tree_masks(lens, "chain"), queries(rows, seed=5)
    want, tol = R.tree_reference(q, b, masks)
    q[3, 7, 0] = float("nan")
    got = run(cp, b, q, masks, bf16, splits)
    assert torch.isnan(got[3, 7]).all()
    got[3, 7] = want[3, 7].float()
    check(got, want, tol + 1e-7)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows", [3, 7, 40])
@pytest.mark.parametrize("splits", [1, 4, 20])
def test_out_may_be_q(cp, bf16, rows, splits):
    lens = [(3000, rows), (200, rows)]
    b = R.make_batch(lens, bf16=bf16, seed=65)
    masks, q = R.tree_masks(lens, seed=1), queries(2 * rows, seed=6)
    want = run(cp, b, q, masks, bf16, splits)
    need = cp.attn_tree_workspace_bytes(2, 2 * rows, rows, 3000, splits)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    call = cp.attn_tree_paged_bf16kv if bf16 else cp.attn_tree_paged
    call(q, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], torch.from_numpy(masks).cuda(), q, rows, 3000, splits,
         ws)
    assert torch.equal(q, want)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("splits", [1, 3])
def test_bad_pages_read_as_zeros(cp, bf16, splits):
    lens = [(500, 6), (40, 2)]
    b = R.make_batch(lens, bf16=bf16, seed=71)
    masks, q = R.tree_masks(lens, "chain"), queries(8, seed=6)
    good = b["table"].clone()
    zero = dict(b)
    zero["kp"], zero["vp"], zero["table"] = b["kp"].clone(), b["vp"].clone(), good
    for s, j in ((0, 3), (0, 20), (1, 0)):
        zero["kp"][good[s, j].long()] = 0
        zero["vp"][good[s, j].long()] = 0
    want, tol = R.tree_reference(q, zero, masks)
    b["table"][0, 3], b["table"][0, 20], b["table"][1, 0] = b["kp"].shape[0], -1, 2 ** 30
    assert cp.attn_get_device_error() == 0
    got = run(cp, b, q, masks, bf16, splits)
    assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    check(got, want, tol + 1e-6)
    b["table"] = good
    got = run(cp, b, q, masks, bf16, splits)
    assert cp.attn_get_device_error() == 0
    check(got, *R.tree_reference(q, b, masks))


def test_lengths_out_of_range_are_recorded(cp):
    """Contexts and row counts past the stated bounds: recorded and clamped, the
    other sequences unharmed."""
    lens = [(100, 3), (60, 4), (90, 2)]
    b = R.make_batch(lens, seed=72)
    masks, q = R.tree_masks(lens, "chain"), queries(9, seed=7)
    want, tol = R.tree_reference(q, b, masks)
    b["ctx"][1] = -3
    assert cp.attn_get_device_error() == 0
    got = run(cp, b, q, masks, False)
    assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    check(got[[0, 1, 2, 7, 8]], want[[0, 1, 2, 7, 8]], tol[[0, 1, 2, 7, 8]])
    b["ctx"][1] = 60
    got = run(cp, b, q, masks, False, max_rows=3)  # sequence 1 has four
    assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    check(got[[0, 1, 2, 7, 8]], want[[0, 1, 2, 7, 8]], tol[[0, 1, 2, 7, 8]])


def test_workspace_is_checked(cp):
    lens = [(3000, 2)]
    b = R.make_batch(lens, seed=73)
    q, out = queries(2), torch.empty(2, 32, 64, device="cuda")
    need = cp.attn_tree_workspace_bytes(1, 2, 2, 3000, 20)
    assert need > 0
    for ws in (None, torch.empty(need - 16, dtype=torch.uint8, device="cuda")):
        with pytest.raises(cp.AttnError) as e:
            cp.attn_tree_paged(q, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], None, out, 2, 3000, 20, ws)
        assert e.value.code == cp.ATTN_ESPACE


def test_workspace_of_the_longest_context(cp):
    """attn_tree_paged takes a bound of ATTN_MAX_TOKENS; the size is there for it too."""
    assert cp.attn_tree_workspace_bytes(2, 9, 5, cp.MAX_TOKENS, 20) == 9 * 32 * 20 * 66 * 4


def test_pools_past_32_bit_offsets(cp):
    """Pages whose bytes lie past 4 GiB of their pool."""
    lens = [(200, 5)]
    b = R.make_batch(lens, bf16=False, seed=81, num_pages=140000)
    masks, q = R.tree_masks(lens, seed=1), queries(5, seed=8)
    k, v = torch.randn(5, 8, 64, device="cuda"), torch.randn(5, 8, 64, device="cuda")
    cp.attn_append_paged(k, v, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"])
    tok = torch.arange(200, 205, device="cuda")
    page = b["table"].long()[0, tok // 16]
    assert int(page.min()) * 16 * 512 * 4 > 2 ** 32
    assert torch.equal(b["kp"][page, tok % 16], k) and torch.equal(b["vp"][page, tok % 16], v)
    check(run(cp, b, q, masks, False), *R.tree_reference(q, b, masks))
    keep = torch.tensor([[1, 4]], dtype=torch.int32, device="cuda")
    cp.attn_compact_paged(b["kp"], b["vp"], b["table"], b["ctx"], keep,
                          torch.tensor([2], dtype=torch.int32, device="cuda"), 5)
    assert torch.equal(b["kp"][page[:2], tok[:2] % 16], k[[1, 4]])
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("splits", [0, 12])
def test_streams_and_graph_replay(cp, bf16, splits):
    """Two captured graphs with a workspace each, replayed on two streams at once,
    after the inputs have changed; and an eager call on another stream."""
    lens = [(2000, 9), (700, 4)]
    made = []
    for s in range(2):
        b = R.make_batch(lens, bf16=bf16, seed=90 + s)
        masks = torch.from_numpy(R.tree_masks(lens, seed=s)).cuda()
        q, out = queries(13, seed=s), torch.empty(13, 32, 64, device="cuda")
        need = cp.attn_tree_workspace_bytes(2, 13, 9, 2000, splits)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        call = cp.attn_tree_paged_bf16kv if bf16 else cp.attn_tree_paged
        args = (q, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], masks, out, 9, 2000)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            call(*args, num_splits=splits, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            call(*args, num_splits=splits, workspace=ws)
        q.copy_(queries(13, seed=s + 10))
        out.fill_(float("nan"))
        made.append((b, masks, q, out, g, st, ws))
    torch.cuda.synchronize()
    for _ in range(3):
        for *_, g, st, _ws in made:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for b, masks, q, out, *_ in made:
        check(out, *R.tree_reference(q, b, masks.cpu().numpy()))
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("rows,splits", [(3, 0), (7, 20), (20, 0)])
def test_each_call_sees_what_ran_before_it(cp, captured, rows, splits):
    """A call may be prepared while what is before it in the stream still runs: a
    long kernel, a copy, a fill, another stream's work joined by an event, and its
    own predecessors, whose results it reads and overwrites."""
    lens = [(900, rows), (300, rows)]
    n = 2 * rows
    b = R.make_batch(lens, seed=130)
    kp0, vp0 = b["kp"].clone(), b["vp"].clone()
    masks = R.tree_masks(lens, "chain")
    table = cp.attn_rope_table(torch.empty(1024, 64, device="cuda"))
    sets = [[torch.randn(n, h, 64, device="cuda") for h in (32, 8, 8)] for _ in range(3)]
    q, k, v, qo, out = (torch.empty(n, h, 64, device="cuda") for h in (32, 8, 8, 32, 32))
    keep = torch.tensor([[rows - 1]] * 2, dtype=torch.int32, device="cuda")
    cnt = torch.empty(2, dtype=torch.int32, device="cuda")
    need = cp.attn_tree_workspace_bytes(2, n, rows, 900, splits)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    slow = torch.randn(2048, 2048, device="cuda")
    outs, sides = [torch.empty_like(out) for _ in sets], torch.cuda.Stream()

    def step():
        for (q1, k1, v1), o in zip(sets, outs):
            q.copy_(q1)                      # copies
            x = slow @ slow                  # a kernel that takes a while
            k.copy_(k1).add_(x[0, 0] * 0)
            sides.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(sides):   # work of another stream
                v.copy_((slow @ slow)[0, 0] * 0 + v1)
            torch.cuda.current_stream().wait_stream(sides)
            cp.attn_append_paged(k, v, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], table, q=q, qOut=qo)
            cp.attn_tree_paged(qo, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], None, out, rows, 900, splits, ws)
            o.copy_(out)                     # and what follows a call
            out.zero_()
            cnt.fill_(1)
            cp.attn_compact_paged(b["kp"], b["vp"], b["table"], b["ctx"], keep, cnt, rows)
            for pool in (q, k, v, qo, cnt):
                pool.zero_()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    for o in outs:
        o.zero_()
    b["kp"].copy_(kp0), b["vp"].copy_(vp0)
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        g.replay()
    else:
        step()
    torch.cuda.synchronize()
    assert cp.attn_get_device_error() == 0
    tok = torch.tensor([c + i for c, t in lens for i in range(t)], device="cuda")
    for (q1, k1, v1), o in zip(sets, outs):
        want = dict(b, kp=kp0.clone(), vp=vp0.clone())
        kw, kt = R.norm_rotate_reference(k1, None, tok, table, 0, 1e-6)
        qw, qt = R.norm_rotate_reference(q1, None, tok, table, 0, 1e-6)
        seq = torch.tensor([0] * rows + [1] * rows, device="cuda")
        page = b["table"].long()[seq, tok // 16]
        want["kp"][page, tok % 16], want["vp"][page, tok % 16] = kw.float(), v1
        ref, tol = R.tree_reference(qw.float(), want, masks)
        # the rotated operands' own roundings (a few 2^-24 of values around 1) next to the tolerance's 2^-19
        check(o, ref, 2 * tol)
    last = torch.tensor([rows - 1, 2 * rows - 1], device="cuda")
    first = torch.tensor([900, 300], device="cuda")
    assert torch.equal(b["vp"][b["table"].long()[[0, 1], first // 16], first % 16], sets[-1][2][last])


@pytest.mark.parametrize("bf16", [False, True])
def test_calls_from_several_threads(cp, bf16):
    """Four threads, each with its own stream, batch and workspace."""
    import threading
    lens = [(900, 6), (300, 3), (2500, 4)]
    call = cp.attn_tree_paged_bf16kv if bf16 else cp.attn_tree_paged
    need = cp.attn_tree_workspace_bytes(3, 13, 6, 2500, 12)
    made = []
    for s in range(4):
        b, masks = R.make_batch(lens, bf16=bf16, seed=110 + s), R.tree_masks(lens, seed=s)
        made.append((b, masks, torch.from_numpy(masks).cuda(), queries(13, seed=s),
                     torch.empty(13, 32, 64, device="cuda"), torch.empty(need, dtype=torch.uint8, device="cuda"),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(b, m, q, out, ws, st):
        for splits in (12, 0, 1, 12):
            call(q, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], m, out, 6, 2500, splits, ws, stream=st)

    threads = [threading.Thread(target=work, args=(b, *rest)) for b, _, *rest in made]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for b, masks, _, q, out, *_ in made:
        check(out, *R.tree_reference(q, b, masks))
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("rows", [2, 7, 20])
def test_beside_a_prefill_on_another_stream(cp, rows):
    """Blocks of the bf16 prefill and of the tree kernels share SMs, shared and tensor memory."""
    lens = [(3000, rows)] * 3
    b = R.make_batch(lens, bf16=True, seed=120)
    masks, q = R.tree_masks(lens, seed=1), queries(3 * rows, seed=2)
    m, out = torch.from_numpy(masks).cuda(), torch.empty_like(q)
    need = cp.attn_tree_workspace_bytes(3, 3 * rows, rows, 3000, 0)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    pq = torch.randn(96, 32, 64, device="cuda")
    pk, pv = (torch.randn(2096, 8, 64, device="cuda").bfloat16() for _ in range(2))
    pout, want = torch.empty_like(pq), torch.empty_like(pq)
    cp.attn_prefill_bf16kv(pq, pk, pv, want, 2000)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(40):
        cp.attn_prefill_bf16kv(pq, pk, pv, pout, 2000, stream=streams[0])
        cp.attn_tree_paged_bf16kv(q, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], m, out, rows, 3000, 0, ws,
                                  stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(pout, want)
    check(out, *R.tree_reference(q, b, masks))
    assert cp.attn_get_device_error() == 0


FIRST_CALLS = """
import torch
import chunked_prefill_gqa_gb300 as cp
F, I = dict(device="cuda"), dict(device="cuda", dtype=torch.int32)
k, q, out = torch.randn(4, 8, 64, **F), torch.randn(4, 32, 64, **F), torch.empty(4, 32, 64, **F)
kp, vp = torch.zeros(6, 16, 8, 64, **F), torch.zeros(6, 16, 8, 64, **F)
table, ctx, starts = torch.arange(6, **I).view(2, 3), torch.zeros(2, **I), torch.tensor([0, 1, 4], **I)
keep, counts, cs = torch.zeros(2, 1, **I), torch.ones(2, **I), torch.empty(8, 64, **F)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    cp.attn_rope_table(cs)
    cp.attn_append_paged(k, k, kp, vp, table, ctx, starts, cs, q=q, qOut=q)
    cp.attn_tree_paged(q, kp, vp, table, ctx, starts, None, out, 3, 20)
    cp.attn_compact_paged(kp, vp, table, ctx, keep, counts, 3)
g.replay()
torch.cuda.synchronize()
v = k[0][:, None].expand(8, 4, 64)  # one key: its value, whose product keeps all but 2^-19 of it
assert ((out[0].view(8, 4, 64) - v).abs() <= 2.0 ** -19 * v.abs()).all()
assert cp.attn_get_device_error() == 0
print("captured")
"""


def test_first_calls_inside_a_capture(cp):
    """A process whose first calls of the library are captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("pairing", [0, 1])
def test_serving_step(cp, bf16, pairing):
    """Append, tree attention, compaction and the next step, against the same step
    done plainly: what the accepted rows leave in the cache is what appending
    them one after another leaves."""
    lens = [(50, 12), (0, 7), (129, 3)]
    b = R.make_batch(lens, bf16=bf16, seed=95)
    dtype = b["kp"].dtype
    n = b["n"]
    table = cp.attn_rope_table(torch.empty(400, 64, device="cuda"))
    masks = R.tree_masks(lens, seed=6)
    depth = np.array([bin(int(m) & (1 << 64) - 1).count("1") - 1 for m in masks.view(np.uint64)])
    ctx_of = np.concatenate([[c] * t for c, t in lens])
    pos = torch.from_numpy((ctx_of + depth).astype(np.int32)).cuda()
    q, k, v = (torch.randn(n, h, 64, device="cuda") for h in (32, 8, 8))
    qw, kw = torch.randn(64, device="cuda"), torch.randn(64, device="cuda")
    qo = torch.empty_like(q)
    append = cp.attn_append_paged_bf16kv if bf16 else cp.attn_append_paged
    append(k, v, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], table, positions=pos, kWeight=kw, q=q, qOut=qo,
           qWeight=qw, pairing=pairing)
    qwant, qtol = R.norm_rotate_reference(q, qw, pos.long(), table, pairing, 1e-6)
    assert ((qo.double() - qwant).abs() <= qtol + 1e-37).all()
    out = run(cp, b, qo, masks, bf16)
    check(out, *R.tree_reference(qo, b, masks))
    # accept in each sequence the path to its last row
    keep, counts = np.zeros((3, 12), dtype=np.int32), []
    r = 0
    for s, (c, t) in enumerate(lens):
        last = int(masks.view(np.uint64)[r + t - 1])
        path = [j for j in range(t) if last >> j & 1]
        keep[s, :len(path)] = path
        counts.append(len(path))
        r += t
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    compact = cp.attn_compact_paged_bf16kv if bf16 else cp.attn_compact_paged
    compact(b["kp"], b["vp"], b["table"], b["ctx"], torch.from_numpy(keep).cuda(), cnt, 12)
    r = 0
    for s, (c, t) in enumerate(lens):
        path = torch.from_numpy(keep[s, :counts[s]].astype(np.int64)).cuda()
        kwant, ktol = R.norm_rotate_reference(k[r + path], kw, c + torch.arange(len(path), device="cuda"), table,
                                              pairing, 1e-6)
        tok = torch.arange(c, c + counts[s], device="cuda")
        page = b["table"].long()[s, tok // 16]
        assert ((b["kp"][page, tok % 16].double() - kwant).abs() <= R.stored(kwant, ktol, dtype)).all()
        assert torch.equal(b["vp"][page, tok % 16], v[r + path].to(dtype))
        r += t
    # the next token of every sequence, one row each
    b["ctx"] = b["ctx"] + cnt
    b["lens"] = [(c + m, 1) for (c, _), m in zip(lens, counts)]
    b["starts"], b["n"] = torch.arange(4, dtype=torch.int32, device="cuda"), 3
    b["max_rows"], b["max_context"] = 1, max(c for c, _ in b["lens"])
    q1, k1, v1 = (torch.randn(3, h, 64, device="cuda") for h in (32, 8, 8))
    qo1 = torch.empty_like(q1)
    append(k1, v1, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], table, kWeight=kw, q=q1, qOut=qo1, qWeight=qw,
           pairing=pairing)
    check(run(cp, b, qo1, None, bf16), *R.tree_reference(qo1, b, R.tree_masks(b["lens"], "chain")))
    assert cp.attn_get_device_error() == 0
