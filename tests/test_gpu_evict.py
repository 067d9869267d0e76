"""attn_evict_paged (both page types) against the selection in whole numbers, bit by bit,
and the run of a bounded cache: append, weigh, evict, decode."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402
import weights_ref as W  # noqa: E402
from test_gpu_weights import bits, check_weights, decode, inside, ints, weigh, workspace  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


def evict(cp, b, w, keep, first=0, last=0, bound=None, ws=None):
    call = cp.attn_evict_paged_bf16kv if b["kp"].dtype == torch.bfloat16 else cp.attn_evict_paged
    bound = b["max_context"] if bound is None else bound
    ws = workspace(cp.attn_evict_workspace_bytes(len(b["lens"]), bound)) if ws is None else ws
    call(b["kp"], b["vp"], w, b["table"], b["ctx"], keep if torch.is_tensor(keep) else ints(keep), bound, keep_first=first,
         keep_last=last, workspace=ws)


def rows_of(pool, b, s, n):
    tok = torch.arange(n, device="cuda")
    return pool[b["table"][s].long()[tok // 16], tok % 16]


def check(cp, b, w, keep, first=0, last=0, bound=None, untouched=()):
    """Runs the call and compares every kept token's key, value and weight, bit by bit."""
    old = b["kp"].clone(), b["vp"].clone(), w.clone()
    evict(cp, b, w, keep, first, last, bound)
    for s, (c, _) in enumerate(b["lens"]):
        n = c if s in untouched else min(c, keep[s])
        ow, nw = W.get_weights(old[2], b, s, c), W.get_weights(w, b, s, c)
        for g in range(8):
            if s in untouched or n == c:
                source = np.arange(c)
            else:
                source = W.evict_reference(ow[:, g].cpu().numpy(), c, n, first, last)
            at = torch.from_numpy(source).cuda()
            assert torch.equal(bits(nw[:len(source), g].contiguous()), bits(ow[at, g].contiguous())), (s, g)
            for pool, before in zip((b["kp"], b["vp"]), old):
                got, want = rows_of(pool, b, s, c)[:len(source), g], rows_of(before, b, s, c)[at, g]
                assert torch.equal(bits(got.contiguous()), bits(want.contiguous())), (s, g)
        # what is left behind the kept tokens stays as it was
        for pool, before in zip((b["kp"], b["vp"]), old):
            assert torch.equal(bits(rows_of(pool, b, s, c)[n:].contiguous()), bits(rows_of(before, b, s, c)[n:].contiguous()))
    used = torch.zeros(b["kp"].shape[0], dtype=torch.bool, device="cuda")
    used[b["table"][b["table"] >= 0].long()] = True
    for pool, before in zip((b["kp"], b["vp"], w), old):
        assert torch.equal(bits(pool[~used].contiguous()), bits(before[~used].contiguous()))


CASES = {
    "small": ([20, 7, 1, 0, 33], [10, 7, 1, 0, 32], 0, 0),
    "sinks": ([100, 257], [50, 100], 4, 16),
    "all of them": ([100, 60], [100, 200], 4, 16),
    "nothing of the middle": ([100, 300], [20, 20], 4, 16),
    "to nothing": ([100, 17], [0, 0], 0, 0),
    "one leaves": ([1000, 65], [999, 64], 4, 64),
    "last ones overlap": ([1000, 900], [990, 650], 1, 300),
    "many last ones": ([3000, 1200], [1100, 1199], 0, 1000),
    "to one": ([500, 2], [1, 1], 0, 1),
    "ragged": ([int(x) % 900 + 40 for x in np.random.default_rng(1).integers(0, 10 ** 6, 60)],
               [int(x) % 500 + 40 for x in np.random.default_rng(2).integers(0, 10 ** 6, 60)], 8, 32),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("bound", [None, 5000, 40000])  # one block a head; a cluster and a second kernel
def test_evict(cp, name, bf16, bound):
    contexts, keep, first, last = CASES[name]
    b = R.make_batch([(c, 0) for c in contexts], bf16=bf16, seed=3, extra_blocks=2500 if bound else 0)
    # A sequence that has to give up tokens and cannot hold the first and last ones is refused.
    refused = [s for s, c in enumerate(contexts) if keep[s] < c and keep[s] < first + last]
    check(cp, b, W.weight_pool(b), keep, first, last, bound=bound, untouched=refused)
    assert cp.attn_get_device_error() == (cp.ATTN_EBOUNDS if refused else 0)


@pytest.mark.parametrize("kind", ["zeros", "few values", "half zeros", "nan", "signs", "infinite"])
@pytest.mark.parametrize("context,keep", [(700, 300), (4096, 3500), (5000, 4500)])
def test_equal_and_unusual_weights(cp, kind, context, keep):
    b = R.make_batch([(context, 0), (90, 0)], bf16=True, seed=4)
    rng, w = np.random.default_rng(5), W.weight_pool(b)
    for s, (c, _) in enumerate(b["lens"]):
        x = np.exp(rng.standard_normal((c, 8))).astype(np.float32)
        if kind == "zeros":
            x[:] = 0
        elif kind == "few values":
            x = rng.integers(0, 3, (c, 8)).astype(np.float32)
        elif kind == "half zeros":
            x[rng.random((c, 8)) < 0.5] = 0.0
            x[rng.random((c, 8)) < 0.1] = -0.0  # equal to the other zero
        elif kind == "nan":
            x[rng.random((c, 8)) < 0.4] = np.nan
            x[rng.random((c, 8)) < 0.2] = -np.inf
        elif kind == "signs":
            x = rng.standard_normal((c, 8)).astype(np.float32)
        else:
            x[rng.random((c, 8)) < 0.3] = np.inf
            x[rng.random((c, 8)) < 0.3] = 1e-42  # below the normal numbers
        W.put_weights(w, b, s, x)
    check(cp, b, w, [keep, 45], 3, 20)


@pytest.mark.parametrize("kind", ["zeros", "few values", "half zeros"])
@pytest.mark.parametrize("contexts,keep", [([20000], 9000), ([40000, 30, 17000], 8000)])
def test_more_equal_weights_than_are_listed(cp, kind, contexts, keep):
    """So many in the first digit's bin that a block's list of them overflows: all of its keys are looked at again."""
    b = R.make_batch([(c, 0) for c in contexts], bf16=True, seed=8)
    rng, w = np.random.default_rng(9), W.weight_pool(b)
    for s, c in enumerate(contexts):
        x = np.exp(rng.standard_normal((c, 8))).astype(np.float32)
        if kind == "zeros":
            x[:] = 0
        elif kind == "few values":
            x = rng.integers(0, 3, (c, 8)).astype(np.float32)
        else:
            x[rng.random((c, 8)) < 0.7] = 0.0
        W.put_weights(w, b, s, x)
    check(cp, b, w, [keep] * len(contexts), 4, 20)
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("contexts,keep", [([20000], 9000), ([70001], 60000), ([9000, 300, 12345], 4000)])
def test_several_blocks_a_head(cp, contexts, keep):
    b = R.make_batch([(c, 0) for c in contexts], bf16=True, seed=6)
    check(cp, b, W.weight_pool(b), [keep] * len(contexts), 4, 128)


def test_a_bound_far_above_the_lengths(cp):
    """So far that a block's tokens would not fit its shared memory: read again instead."""
    b = R.make_batch([(5000, 0), (100, 0), (0, 0)], bf16=True, seed=7, extra_blocks=30000)
    check(cp, b, W.weight_pool(b), [1234, 64, 5], 4, 32, bound=480000)
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("far", [0, 500])  # by a bound of 8000 through lists in memory
def test_refused_sequences_are_recorded_and_left(cp, far):
    lens = [(100, 0), (200, 0), (300, 0), (80, 0)]

    def fresh():
        b = R.make_batch(lens, seed=8, extra_blocks=far)
        if far:
            b["max_context"] = 8000
        return b, W.weight_pool(b)
    b, w = fresh()
    assert cp.attn_get_device_error() == 0
    check(cp, b, w, [50, 19, 100, 30], 4, 16, untouched=(1,))  # 19 < 4 + 16
    assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    b, w = fresh()
    check(cp, b, w, [50, -1, 100, 30], 4, 16, untouched=(1,))
    assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    b, w = fresh()
    check(cp, b, w, [50, 60, 100, 30], 4, 16, bound=250, untouched=(2,))  # 300 is past the bound
    assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    for entry in (0, 7, 12):  # a bad page under the first ones, the middle, the last ones of sequence 1
        for page in (-1, 1 << 20):
            b, w = fresh()
            old = b["kp"].clone(), b["vp"].clone(), w.clone()
            good = b["table"].clone()
            b["table"][1, entry] = page
            evict(cp, b, w, [50, 60, 100, 30], 4, 16)
            assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
            b["table"] = good
            for pool, before in zip((b["kp"], b["vp"]), old):
                assert torch.equal(bits(rows_of(pool, b, 1, 200)), bits(rows_of(before, b, 1, 200)))
                assert not torch.equal(bits(rows_of(pool, b, 0, 50)), bits(rows_of(before, b, 0, 50)))
    b = R.make_batch(lens, seed=8, extra_blocks=500)
    w = W.weight_pool(b)
    for ws, code in ((torch.empty(64, dtype=torch.uint8, device="cuda"), cp.ATTN_ESPACE),
                     (workspace(1 << 20)[8:], cp.ATTN_EALIGN)):
        with pytest.raises(cp.AttnError) as e:
            evict(cp, b, w, [50, 60, 100, 30], bound=8000, ws=ws)
        assert e.value.code == code
    with pytest.raises(cp.AttnError) as e:
        evict(cp, b, w, [50, 60, 100, 30], first=-1)
    assert e.value.code == cp.ATTN_EINVAL
    with pytest.raises(ValueError):
        evict(cp, b, w, ints([1, 2, 3]))


def test_graph_and_two_streams(cp):
    lens = [(900, 0), (4000, 0)]
    b, plain = R.make_batch(lens, bf16=True, seed=9), R.make_batch(lens, bf16=True, seed=9)
    w, pw = W.weight_pool(b), W.weight_pool(plain)
    keep, ws = ints([400, 1000]), workspace(cp.attn_evict_workspace_bytes(2, 4000))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        evict(cp, b, w, keep, 4, 64, ws=ws)
    graph.replay()
    keep.copy_(ints([300, 500]))
    b["ctx"].copy_(ints([400, 1000]))
    graph.replay()  # lengths are read by the call, not by the capture
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, (ctx, now) in enumerate((((900, 400), 300), ((4000, 1000), 500))):
        one = dict(plain, lens=[lens[s]], table=plain["table"][s:s + 1].contiguous(), max_context=lens[s][0])
        steps = [(ints([ctx[0]]), ints([ctx[1]])), (ints([ctx[1]]), ints([now]))]
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[s]):
            for c, k in steps:
                evict(cp, dict(one, ctx=c), pw, k, 4, 64)
    torch.cuda.synchronize()
    for got, want in ((b["kp"], plain["kp"]), (b["vp"], plain["vp"]), (w, pw)):
        assert torch.equal(bits(got), bits(want))


def test_pools_past_two_to_the_31(cp):
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    pages = (1 << 31) // (16 * 8 * 64) + 40
    b = R.make_batch([(300, 0), (100, 0)], bf16=True, seed=10, num_pages=pages)
    check(cp, b, W.weight_pool(b), [100, 60], 4, 16)


@pytest.mark.parametrize("bf16", [False, True])
def test_a_bounded_cache(cp, bf16):
    """A video's rows appended by their three positions, its last rows weighed, the cache cut
    down, then decode steps on what is left, and cut down again: each step against the
    plain form on the cache as it stands."""
    axes, video, window = [i % 3 for i in range(32)], 450, 32
    lens, n = [(0, video), (0, 130)], video + 130
    b = R.make_batch([(c, t + 40) for c, t in lens], bf16=bf16, seed=11)  # room for what is decoded
    table = cp.attn_rope_table(torch.empty(2000, 64, device="cuda"))
    act = b["kp"].dtype
    q, k, v = (torch.randn(n, h, 64, device="cuda").to(act) for h in (32, 8, 8))
    pos = torch.stack([torch.arange(n, device="cuda") // 20, torch.arange(n, device="cuda") % 20 // 5,
                       torch.arange(n, device="cuda") % 5]).to(torch.int32)
    qo, one = torch.empty(n, 32, 64, device="cuda"), torch.ones(64, device="cuda")
    ctx, starts = ints([0, 0]), ints([0, video, n])
    append = cp.attn_append_paged_axes_bf16kv if bf16 else cp.attn_append_paged_axes
    append(k, v, b["kp"], b["vp"], b["table"], ctx, starts, table, pos, axes, kWeight=one, q=q, qOut=qo, qWeight=one)
    w = torch.full((b["kp"].shape[0], 8, 16), float("nan"), device="cuda")
    rows = torch.cat([qo[video - window:video], qo[n - window:]]).contiguous()
    part = dict(b, lens=[(video - window, window), (130 - window, window)], ctx=ints([video - window, 130 - window]),
                starts=ints([0, window, 2 * window]), n=2 * window, max_rows=window, max_context=video - window)
    before = w.clone()
    weigh(cp, part, rows, w, weighed=ints([0, 0]))
    check_weights(w, before, part, W.weigh_reference(rows, part, before, [0, 0], 1.0))
    now, keep = [video, 130], [200, 130]
    at = dict(b, lens=[(c, 0) for c in now], ctx=ints(now), max_context=max(now))
    check(cp, at, w, keep, 4, 16)
    now = keep
    for step in range(6):
        t = 30 + step  # positions go on where the video ended, whatever the slots
        x = [torch.randn(2, h, 64, device="cuda").to(act) for h in (32, 8, 8)]
        qd = torch.empty(2, 32, 64, device="cuda")
        append(x[1], x[2], b["kp"], b["vp"], b["table"], ints(now), ints([0, 1, 2]), table,
               ints([[t, t]]).expand(3, 2), axes, kWeight=one, q=x[0], qOut=qd, qWeight=one)
        now = [c + 1 for c in now]
        at = dict(b, lens=[(c, 0) for c in now], ctx=ints(now), max_context=max(now))
        before = w.clone()
        out = decode(cp, at, qd, w, decay=0.95)
        want, ref, tol = W.weigh_reference(qd, at, before, [c - 1 for c in now], 0.95, decode=True)
        inside(out, ref, tol)
        check_weights(w, before, at, want)
        if step % 2:
            keep = [c - 2 for c in now]
            check(cp, at, w, keep, 4, 16)
            now = keep
    assert cp.attn_get_device_error() == 0
