"""Weights of cached tokens (attn_decode_weigh_paged, attn_weigh_paged, both page types)
against plain forms in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402
import weights_ref as W  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


def inside(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() / tol.clamp(min=1e-300)).max()))


def workspace(n):
    w = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return w.fill_(0xFF)  # NaN wherever something unwritten is read


def bits(x):
    return x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)


def check_weights(got, before, batch, want):
    """The weights of the sequences, and that nothing else of the pool changed."""
    rest = before.clone()
    for b, pair in enumerate(want):
        if pair is None:
            continue
        n = pair[0].shape[0]
        inside(W.get_weights(got, batch, b, n), *pair)
        W.put_weights(rest, batch, b, W.get_weights(got, batch, b, n))
    assert torch.equal(bits(rest), bits(got))


def decode(cp, batch, q, weights, decay=1.0, weighed=None, bound=None, stream=None, ws=None):
    bound = batch["max_context"] if bound is None else bound
    call = cp.attn_decode_weigh_paged_bf16kv if batch["kp"].dtype == torch.bfloat16 else cp.attn_decode_weigh_paged
    out = torch.full_like(q, float("nan"))
    ws = workspace(cp.attn_decode_weigh_workspace_bytes(len(batch["lens"]), bound)) if ws is None else ws
    return call(q, batch["kp"], batch["vp"], weights, batch["table"], batch["ctx"], out, bound, decay=decay,
                weighedLens=weighed, workspace=ws, stream=stream)


def weigh(cp, batch, q, weights, decay=1.0, weighed=None, bound=None, rows=None, stream=None, ws=None):
    bound = batch["max_context"] if bound is None else bound
    rows = batch["max_rows"] if rows is None else rows
    call = cp.attn_weigh_paged_bf16kv if batch["kp"].dtype == torch.bfloat16 else cp.attn_weigh_paged
    if ws is None:
        ws = workspace(cp.attn_weigh_workspace_bytes(len(batch["lens"]), q.shape[0], rows, bound))
    return call(q, batch["kp"], weights, batch["table"], batch["ctx"], batch["starts"], rows, bound, decay=decay,
                weighedLens=weighed, workspace=ws, stream=stream)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


CONTEXTS = {
    "one": [1], "none": [0, 5, 0], "page": [15, 16, 17], "warps": [63, 64, 65, 48, 49],
    "segment": [255, 256, 257], "uneven": [1000, 3, 517], "long": [4097], "longer": [19999, 21, 7000], "many": [int(x) % 300 for x in
                                                                                np.random.default_rng(2).integers(0, 10 ** 6, 70)],
}


@pytest.mark.parametrize("name", CONTEXTS)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("decay,bound", [(1.0, None), (0.9, 9000), (0.0, None), (0.9, 30000)])
def test_decode(cp, name, bf16, decay, bound):
    lens = [(c, 0) for c in CONTEXTS[name]]
    bound = bound and max([bound] + CONTEXTS[name])  # of the longest context at least
    b = R.make_batch(lens, bf16=bf16, seed=4, extra_blocks=bound // 16 + 1 if bound else 0)
    weighed = [c - 1 for c, _ in lens]
    w = W.weight_pool(b, known=[max(0, n) for n in weighed]) if decay else torch.full_like(W.weight_pool(b), float("nan"))
    before = w.clone()
    q = torch.randn(len(lens), 32, 64, device="cuda") * 2
    out = decode(cp, b, q, w, decay, bound=bound)
    assert cp.attn_get_device_error() == 0
    want, ref, tol = W.weigh_reference(q, b, before, weighed, decay, decode=True)
    inside(out, ref, tol)
    check_weights(w, before, b, want)


@pytest.mark.parametrize("bf16", [False, True])
def test_decode_of_tokens_without_weights(cp, bf16):
    """weighedLens below the context: what the pool held from there on is not read."""
    lens = [(300, 0), (40, 0), (700, 0)]
    b, weighed = R.make_batch(lens, bf16=bf16, seed=5), [0, 17, 700]
    w = W.weight_pool(b, known=weighed)
    before, q = w.clone(), torch.randn(3, 32, 64, device="cuda")
    out = decode(cp, b, q, w, weighed=ints(weighed))
    want, ref, tol = W.weigh_reference(q, b, before, weighed, 1.0, decode=True)
    inside(out, ref, tol)
    check_weights(w, before, b, want)


WINDOWS = {
    "one": [(0, 1)], "first": [(0, 33), (0, 1), (0, 32)], "edges": [(127, 1), (128, 1), (129, 2), (96, 32), (95, 33)],
    "rows": [(50, 3), (300, 0), (31, 31), (0, 0), (200, 64), (17, 65)], "prompt": [(0, 300)], "long": [(4000, 7), (33, 100)],
    "many": [(int(x) % 200, int(x) % 5) for x in np.random.default_rng(3).integers(0, 10 ** 6, 90)],
}


@pytest.mark.parametrize("name", WINDOWS)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("decay,bound", [(1.0, None), (0.5, 20000), (0.0, None)])
def test_window(cp, name, bf16, decay, bound):
    lens, pad = WINDOWS[name], 3  # rows behind the last sequence
    b = R.make_batch(lens, bf16=bf16, seed=6, extra_blocks=1260 if bound else 0)
    weighed = [c for c, _ in lens]
    w = W.weight_pool(b) if decay else torch.full_like(W.weight_pool(b), float("nan"))
    before = w.clone()
    q = torch.randn(b["n"] + pad, 32, 64, device="cuda") * 2
    q[b["n"]:] = float("nan")
    assert weigh(cp, b, q, w, decay, bound=bound) is w
    assert cp.attn_get_device_error() == 0
    check_weights(w, before, b, W.weigh_reference(q, b, before, weighed, decay))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens,bound", [([(0, 1)], None), ([(100, 28)], None), ([(100, 29)], None), ([(1023, 1)], None), ([(1024, 32)], None),
                                        ([(3039, 32)], None), ([(3045, 32)], None), ([(3000, 33)], None), ([(5, 9), (0, 32), (700, 17)], 1500),
                                        ([(40 * i, 1 + i) for i in range(15)], 350), ([(0, 3), (2, 0), (1900, 8), (1300, 31)], None)])
def test_windows_whose_products_are_kept(cp, bf16, lens, bound):
    """As many keys as a cluster's tensor memory holds the products of, and a few more; segments without any."""
    bound = max(c for c, _ in lens) if bound is None else max(bound, max(c for c, _ in lens))
    b = R.make_batch(lens, bf16=bf16, seed=15, extra_blocks=bound // 16 + 2)
    weighed = [max(0, c - 5) for c, _ in lens]
    w, q = W.weight_pool(b, known=weighed), torch.randn(b["n"], 32, 64, device="cuda") * 2
    before = w.clone()
    weigh(cp, b, q, w, 0.9, ints(weighed), bound=bound)
    assert cp.attn_get_device_error() == 0
    check_weights(w, before, b, W.weigh_reference(q, b, before, weighed, 0.9))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens,bound", [([9000, 3, 0, 515, 8999] + [100 * i for i in range(11)], None),
                                        ([8192, 8191, 8177] + [31 * i for i in range(27)], None),
                                        ([16384, 16383, 12000, 5, 16000, 64, 65], 40000),
                                        ([20480, 20481, 300], 60000)])
def test_decode_of_uneven_lengths(cp, bf16, lens, bound):
    b = R.make_batch([(c, 0) for c in lens], bf16=bf16, seed=14, extra_blocks=(bound or 0) // 16)
    bound = max(lens) if bound is None else bound
    weighed = [max(0, c - 1 - 7 * (i % 3)) for i, c in enumerate(lens)]
    w, q = W.weight_pool(b, known=weighed), torch.randn(len(lens), 32, 64, device="cuda") * 2
    before = w.clone()
    out = decode(cp, b, q, w, 0.9, ints(weighed), bound=bound)
    assert cp.attn_get_device_error() == 0
    want, o, tol = W.weigh_reference(q, b, before, weighed, 0.9, decode=True)
    check_weights(w, before, b, want)
    inside(out, o, tol)


@pytest.mark.parametrize("bf16", [False, True])
def test_window_of_tokens_without_weights(cp, bf16):
    """A prompt's last rows weigh all of it for the first time."""
    lens = [(260, 40), (100, 3), (1000, 64)]
    b, weighed = R.make_batch(lens, bf16=bf16, seed=7), [0, 103, 500]
    w = W.weight_pool(b, known=weighed)
    before, q = w.clone(), torch.randn(b["n"], 32, 64, device="cuda")
    weigh(cp, b, q, w, weighed=ints(weighed))
    check_weights(w, before, b, W.weigh_reference(q, b, before, weighed, 1.0))


@pytest.mark.parametrize("bf16", [False, True])
def test_window_of_one_row_is_a_decode_step(cp, bf16):
    lens = [(77, 1), (400, 1)]
    b, q = R.make_batch(lens, bf16=bf16, seed=8), torch.randn(2, 32, 64, device="cuda")
    w0, w1 = W.weight_pool(b), W.weight_pool(b)
    weigh(cp, b, q, w0)
    grown = dict(b, ctx=b["ctx"] + 1, max_context=401, lens=[(78, 0), (401, 0)])
    decode(cp, grown, q, w1)
    before = W.weight_pool(b)
    for pool in (w0, w1):
        check_weights(pool, before, b, W.weigh_reference(q, b, before, [77, 400], 1.0))


@pytest.mark.parametrize("bf16", [False, True])
def test_probabilities_add_up(cp, bf16):
    """Set from nothing, a sequence's weights are 4 heads x rows in all."""
    lens = [(500, 9), (0, 40)]
    b, q = R.make_batch(lens, bf16=bf16, seed=9), torch.randn(49, 32, 64, device="cuda") * 4
    w = torch.full_like(W.weight_pool(b), float("nan"))
    weigh(cp, b, q, w, decay=0.0)
    for s, (c, t) in enumerate(lens):
        got = W.get_weights(w, b, s, c + t).double().sum(0)
        # each p to 2^-15 (softmax_reference's bound at these scores), the weights to 70 roundings
        assert ((got - 4 * t).abs() <= 4 * t * 2.0 ** -13).all(), got


@pytest.mark.parametrize("bf16", [False, True])
def test_scores_of_any_size(cp, bf16):
    """Scores of several hundred, a maximum in the last token, and one token that takes all."""
    lens = [(700, 0), (33, 0)]
    b = R.make_batch(lens, bf16=bf16, seed=10)
    q = torch.randn(2, 32, 64, device="cuda")
    q[0] = 30.0
    b["kp"][b["table"][0, 699 // 16].long(), 699 % 16] = 30.0  # score 64 * 900 / 8
    w = W.weight_pool(b, known=[699, 32])
    before = w.clone()
    out = decode(cp, b, q, w)
    want, ref, tol = W.weigh_reference(q, b, before, [699, 32], 1.0, decode=True)
    assert torch.isfinite(out).all() and float((out[0].double() - ref[0]).abs().max()) <= 2.0 ** -18 * float(ref[0].abs().max())
    # one token's probability is 1, the others' underflow
    got = W.get_weights(w, b, 0, 700).double()
    assert float((got[699] - 4).abs().max()) <= 4 * 2.0 ** -18
    assert torch.equal(got[:699].float(), W.get_weights(before, b, 0, 699))
    rows = dict(b, ctx=ints([699, 32]), lens=[(699, 1), (32, 1)], starts=ints([0, 1, 2]), n=2, max_rows=1)
    w = before.clone()
    weigh(cp, rows, q, w)
    got = W.get_weights(w, b, 0, 700).double()
    assert float((got[699] - 4).abs().max()) <= 4 * 2.0 ** -18
    assert torch.equal(got[:699].float(), W.get_weights(before, b, 0, 699))


@pytest.mark.parametrize("bf16", [False, True])
def test_infinities_and_nan_reach_what_they_should(cp, bf16):
    """A NaN key makes its sequence and head NaN, and no other; slots behind the last token
    are NaN throughout (make_batch) and reach nothing."""
    lens = [(40, 0), (90, 0)]
    b = R.make_batch(lens, bf16=bf16, seed=11)
    b["kp"][b["table"][1, 2].long(), 3, 5] = float("nan")  # token 35 of sequence 1, head 5
    w, q = W.weight_pool(b, known=[39, 89]), torch.randn(2, 32, 64, device="cuda")
    before = w.clone()
    out = decode(cp, b, q, w)
    assert torch.isfinite(out[0]).all() and out[1, 20:24].isnan().all()
    assert torch.isfinite(out[1, :20]).all() and torch.isfinite(out[1, 24:]).all()
    got = W.get_weights(w, b, 1, 90)
    assert got[:, 5].isnan().all() and torch.isfinite(got[:, :5]).all() and torch.isfinite(got[:, 6:]).all()
    # In a window, rows before the token do not see it: of the row at 34 alone nothing is NaN.
    for ctx, bad in ((34, False), (35, True)):
        x, w = dict(b, ctx=ints([39, ctx]), starts=ints([0, 1, 2]), max_rows=1), before.clone()
        weigh(cp, x, q, w)
        got = W.get_weights(w, b, 1, ctx + 1)
        assert bool(got[:, 5].isnan().any()) == bad and torch.isfinite(got[:, :5]).all()
        assert torch.isfinite(W.get_weights(w, b, 0, 40)).all()


def test_bad_pages_and_lengths_are_recorded(cp):
    lens = [(100, 0), (60, 0), (40, 0)]
    b, q = R.make_batch(lens, seed=12), torch.randn(3, 32, 64, device="cuda")
    w = W.weight_pool(b, known=[99, 59, 39])
    before, table = w.clone(), b["table"].clone()
    b["table"][1, 1], b["table"][0, 0] = b["kp"].shape[0], -3
    assert cp.attn_get_device_error() == 0
    out = decode(cp, b, q, w)
    assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    want, ref, tol = W.weigh_reference(q[2:], dict(b, lens=lens[2:], table=table[2:]), before, [39], 1.0, decode=True)
    inside(out[2:], ref, tol)  # the others are as ever
    good = dict(b, table=table)
    assert torch.equal(bits(W.get_weights(w, good, 1, 32)[16:]), bits(W.get_weights(before, good, 1, 32)[16:]))
    b["table"] = table
    for ctx in ([100, -1, 40], [101, 60, 40]):  # 101 is past the bound
        x = dict(b, ctx=ints(ctx))
        out = decode(cp, x, q, before.clone())
        assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
        inside(out[2:], ref, tol)
        if ctx[1] < 0:
            assert torch.equal(out[1], torch.zeros_like(out[1]))
    rows = dict(b, starts=ints([0, 1, 2, 3]), ctx=ints([99, 59, 39]), max_rows=1)
    for change in (dict(starts=ints([0, 1, 2, 9])), dict(ctx=ints([-4, 59, 39])), dict(starts=ints([0, 2, 1, 3]))):
        weigh(cp, dict(rows, **change), q, before.clone())
        assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    rows["table"] = b["table"].clone()
    rows["table"][0, 3] = 1 << 20
    w = before.clone()
    weigh(cp, rows, q, w)
    assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    assert torch.isfinite(W.get_weights(w, b, 2, 40)).all()


def test_refusals(cp):
    lens = [(100, 2), (60, 1)]
    b, q = R.make_batch(lens, seed=13, extra_blocks=1900), torch.randn(3, 32, 64, device="cuda")
    w, out = W.weight_pool(b), torch.empty(2, 32, 64, device="cuda")
    need = cp.attn_decode_weigh_workspace_bytes(2, 30000)
    for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device="cuda")):
        with pytest.raises(cp.AttnError) as e:
            cp.attn_decode_weigh_paged(q[:2], b["kp"], b["vp"], w, b["table"], b["ctx"], out, 30000, workspace=ws)
        assert e.value.code == cp.ATTN_ESPACE
    need = cp.attn_weigh_workspace_bytes(2, 3, 65, 100)  # too many rows for their sums to stay on chip
    for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device="cuda")):
        with pytest.raises(cp.AttnError) as e:
            cp.attn_weigh_paged(q, b["kp"], w, b["table"], b["ctx"], b["starts"], 65, 100, workspace=ws)
        assert e.value.code == cp.ATTN_ESPACE
    with pytest.raises(cp.AttnError) as e:
        cp.attn_weigh_paged(q, b["kp"], w, b["table"], b["ctx"], b["starts"], 65, 100, workspace=workspace(need + 16)[8:])
    assert e.value.code == cp.ATTN_EALIGN
    for bad in (w[:, :, :8], w.half(), w.cpu(), w[1:], w.transpose(1, 2)):
        with pytest.raises(ValueError):
            cp.attn_weigh_paged(q, b["kp"], bad, b["table"], b["ctx"], b["starts"], 2, 100, workspace=workspace(need))
    with pytest.raises(cp.AttnError) as e:
        decode(cp, b, q[:2], w, decay=1.5)
    assert e.value.code == cp.ATTN_EINVAL
    with pytest.raises(ValueError):
        decode(cp, b, q[:2], w, weighed=ints([1]))
    empty = torch.empty(0, 32, 64, device="cuda")
    cp.attn_weigh_paged(empty, b["kp"], w, b["table"], b["ctx"], ints([0, 0, 0]), 2, 100)  # no row: nothing to do


@pytest.mark.parametrize("bf16", [False, True])
def test_streams_and_graphs(cp, bf16):
    """Two streams at once, each with its own sequences and workspace, and a step captured
    and replayed: the weights of three passes."""
    lens = [(1500, 20), (700, 3)]
    b = R.make_batch(lens, bf16=bf16, seed=14)
    q = torch.randn(23, 32, 64, device="cuda")
    first, both = W.weight_pool(b), []
    for s, (c, t) in enumerate(lens):
        one = dict(b, lens=[lens[s]], table=b["table"][s:s + 1].contiguous(), ctx=b["ctx"][s:s + 1].contiguous(),
                   starts=ints([0, t]), n=t, max_rows=t, max_context=c)
        both.append((one, q[:20] if s == 0 else q[20:], torch.cuda.Stream()))
    w = first.clone()
    torch.cuda.synchronize()
    for one, rows, stream in both:
        with torch.cuda.stream(stream):
            weigh(cp, one, rows, w)
    torch.cuda.synchronize()
    check_weights(w, first, b, W.weigh_reference(q, b, first, [c for c, _ in lens], 1.0))
    grown = dict(b, ctx=b["ctx"] + 1, lens=[(c + 1, 0) for c, _ in lens], max_context=1501)
    qd, w = torch.randn(2, 32, 64, device="cuda"), first.clone()
    ws0 = workspace(cp.attn_decode_weigh_workspace_bytes(2, 1501))
    ws1 = workspace(cp.attn_weigh_workspace_bytes(2, 23, 20, 1500))
    graph, out = torch.cuda.CUDAGraph(), torch.empty(2, 32, 64, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        weigh(cp, b, q, w, ws=ws1)
        got = decode(cp, grown, qd, w, ws=ws0)
    reached = first.clone()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for call in (weigh(cp, b, q, reached), decode(cp, grown, qd, reached)):
            pass
    out.copy_(got)
    assert torch.equal(bits(w), bits(reached))  # the same bits: no sum goes by the order of atomics
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("bf16", [False, True])
def test_pools_past_two_to_the_31(cp, bf16):
    """Pages far behind the start of a pool of more than 2^31 values."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    lens, pages = [(70, 5), (200, 33)], (1 << 31) // (16 * 8 * 64) + 40
    b = R.make_batch(lens, bf16=bf16, seed=15, num_pages=pages)
    q = torch.randn(38, 32, 64, device="cuda")
    w = W.weight_pool(b)
    before = w.clone()
    weigh(cp, b, q, w)
    check_weights(w, before, b, W.weigh_reference(q, b, before, [70, 200], 1.0))
    grown = dict(b, lens=[(75, 0), (233, 0)], ctx=ints([75, 233]), max_context=233)
    w = W.weight_pool(grown, known=[74, 232])
    before = w.clone()
    out = decode(cp, grown, q[:2], w)
    want, ref, tol = W.weigh_reference(q[:2], grown, before, [74, 232], 1.0, decode=True)
    inside(out, ref, tol)
    check_weights(w, before, b, want)
    assert cp.attn_get_device_error() == 0
