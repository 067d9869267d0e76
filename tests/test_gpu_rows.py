"""attn_rope_table, attn_qk_norm_rope, attn_append_paged and attn_compact_paged
(and the bf16 forms) against plain forms in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


def make_table(cp, n, **kw):
    return cp.attn_rope_table(torch.empty(n, 64, device="cuda"), **kw)


def inside(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() / tol.clamp(min=1e-300)).max()))


@pytest.mark.parametrize("theta", [10000.0, 500000.0])
def test_table(cp, theta):
    n = 70001
    t = make_table(cp, n, theta=theta).double().cpu()
    pos = torch.arange(n, dtype=torch.float64)[:, None]
    ang = pos * torch.tensor([theta ** (-i / 32.0) for i in range(32)], dtype=torch.float64)
    want = torch.cat([ang.cos(), ang.sin()], 1)
    # one rounding to fp32, and the frequency's own half step in double times the position
    assert float((t - want).abs().max()) <= 2.0 ** -24 + n * 2.0 ** -52


def test_table_takes_scaled_frequencies(cp):
    freq = [1.0 / (8.0 ** (i / 7.0)) for i in range(32)]
    t = make_table(cp, 513, invFreq=freq).double().cpu()
    ang = torch.arange(513, dtype=torch.float64)[:, None] * torch.tensor(freq, dtype=torch.float64)
    assert float((t - torch.cat([ang.cos(), ang.sin()], 1)).abs().max()) <= 2.0 ** -24 + 513 * 2.0 ** -52
    with pytest.raises(ValueError):
        make_table(cp, 4, invFreq=freq[:-1])


@pytest.mark.parametrize("n", [1, 2, 7, 33, 300])
@pytest.mark.parametrize("act,out", [(F, F), (F, BF), (BF, F), (BF, BF)])
@pytest.mark.parametrize("pairing,normed", [(0, True), (1, True), (0, False), (1, False)])
def test_norm_rope(cp, n, act, out, pairing, normed):
    gen = torch.Generator(device="cuda").manual_seed(n * 8 + pairing)
    wide = torch.randn(n, 50, 64, generator=gen, device="cuda").to(act)
    q, k = wide[:, 1:33], wide[:, 40:48]  # views with 50 heads between rows
    table = make_table(cp, 5000)
    pos = torch.randint(0, 5000, (n,), generator=gen, device="cuda").to(torch.int32)
    pos[0] = 4999
    qw = torch.randn(64, generator=gen, device="cuda") if normed else None
    kw = torch.randn(64, generator=gen, device="cuda") if normed else None
    qo = torch.full((n, 32, 64), float("nan"), device="cuda")
    ko = torch.full((n, 8, 64), float("nan"), device="cuda", dtype=out)
    cp.attn_qk_norm_rope(q, k, pos, table, qo, ko, qWeight=qw, kWeight=kw, eps=1e-5, pairing=pairing)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        want, tol = R.norm_rotate_reference(x, w, pos.long(), table, pairing, 1e-5)
        inside(got, want, R.stored(want, tol, got.dtype))
    assert cp.attn_get_device_error() == 0


def test_norm_only_rotation_only_and_keys_only(cp):
    n = 19
    q, k = torch.randn(n, 32, 64, device="cuda"), torch.randn(n, 8, 64, device="cuda")
    w = torch.randn(64, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    cp.attn_qk_norm_rope(q, k, None, None, qo, ko, qWeight=w)  # q normed, k copied
    want, tol = R.norm_rotate_reference(q, w, None, None, 0, 1e-6)
    inside(qo, want, tol)
    assert torch.equal(ko, k)
    table, pos = make_table(cp, 64), torch.arange(n, dtype=torch.int32, device="cuda")
    ko.fill_(float("nan"))
    cp.attn_qk_norm_rope(None, k, pos, table, None, ko, kWeight=w, pairing=1)
    want, tol = R.norm_rotate_reference(k, w, pos.long(), table, 1, 1e-6)
    inside(ko, want, tol)


def test_zero_rows_zero_eps_and_extreme_heads(cp):
    """A head of zeros under a norm stays zeros (eps > 0); tiny and large heads
    come out at rms 1."""
    k = torch.zeros(3, 8, 64, device="cuda")
    k[1] = 1e-12
    k[2] = 1e12
    w, ko = torch.ones(64, device="cuda"), torch.empty_like(k)
    cp.attn_qk_norm_rope(None, k, None, None, None, ko, kWeight=w, eps=1e-30)
    assert torch.equal(ko[0], torch.zeros_like(ko[0]))
    want, tol = R.norm_rotate_reference(k[1:], w, None, None, 0, 1e-30)
    inside(ko[1:], want, tol)
    empty = torch.empty(0, 8, 64, device="cuda")
    cp.attn_qk_norm_rope(None, empty, None, None, None, torch.empty_like(empty), kWeight=w)


def test_in_place(cp):
    n = 11
    q, k = torch.randn(n, 32, 64, device="cuda"), torch.randn(n, 8, 64, device="cuda")
    q0, k0 = q.clone(), k.clone()
    table, pos = make_table(cp, 64), torch.arange(n, dtype=torch.int32, device="cuda") + 7
    w = torch.randn(64, device="cuda")
    cp.attn_qk_norm_rope(q, k, pos, table, q, k, qWeight=w, kWeight=w)
    for got, x in ((q, q0), (k, k0)):
        want, tol = R.norm_rotate_reference(x, w, pos.long(), table, 0, 1e-6)
        inside(got, want, tol)


def test_positions_out_of_range_are_recorded_and_clamped(cp):
    k = torch.randn(3, 8, 64, device="cuda")
    table, ko = make_table(cp, 10), torch.empty(3, 8, 64, device="cuda")
    pos = torch.tensor([-5, 3, 10], dtype=torch.int32, device="cuda")
    assert cp.attn_get_device_error() == 0
    cp.attn_qk_norm_rope(None, k, pos, table, None, ko)
    assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    want, tol = R.norm_rotate_reference(k, None, torch.tensor([0, 3, 9], device="cuda"), table, 0, 1e-6)
    inside(ko, want, tol)


BATCHES = {
    "decode": [(0, 1), (15, 1), (16, 1), (1000, 1)],
    "trees": [(5, 7), (0, 3), (31, 0), (17, 64), (100, 1)],
    "chunk": [(100, 300)],
    "many": [(int(x) % 70, int(x) % 3) for x in np.random.default_rng(5).integers(0, 1000, 1100)],
}


@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("with_q", [False, True])
def test_append(cp, name, bf16, with_q):
    lens = BATCHES[name]
    b = R.make_batch(lens, bf16=bf16, seed=3)
    before = b["kp"].clone(), b["vp"].clone()
    n, pad = b["n"], 5  # rows behind the last sequence
    act = BF if bf16 else F
    kv = torch.randn(n + pad, 16, 64, device="cuda").to(act)
    k, v = kv[:, :8], kv[:, 8:]
    q = torch.randn(n + pad, 32, 64, device="cuda").to(act) if with_q else None
    qo = torch.full((n + pad, 32, 64), float("nan"), device="cuda") if with_q else None
    w = torch.randn(64, device="cuda")
    table = make_table(cp, 1200)
    far = torch.randint(0, 1200, (n + pad,), device="cuda").to(torch.int32) if with_q else None
    call = cp.attn_append_paged_bf16kv if bf16 else cp.attn_append_paged
    call(k, v, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], table, positions=far, kWeight=w, q=q, qOut=qo,
         qWeight=w, pairing=1)
    assert cp.attn_get_device_error() == 0
    seq = torch.tensor([s for s, (_, t) in enumerate(lens) for _ in range(t)], device="cuda")
    tok = torch.tensor([c + i for c, t in lens for i in range(t)], device="cuda")
    page, slot = b["table"].long()[seq, tok // 16], tok % 16
    pos = tok if far is None else far[:n].long()
    want, tol = R.norm_rotate_reference(k[:n], w, pos, table, 1, 1e-6)
    dtype = b["kp"].dtype
    inside(b["kp"][page, slot], want, R.stored(want, tol, dtype))
    assert torch.equal(b["vp"][page, slot], v[:n].to(dtype))
    # everything else in the pools is as it was
    for pool, old in zip((b["kp"], b["vp"]), before):
        pool[page, slot] = old[page, slot]
        assert torch.equal(pool.view(torch.int16 if bf16 else torch.int32), old.view(torch.int16 if bf16 else torch.int32))
    if with_q:
        want, tol = R.norm_rotate_reference(q[:n], w, pos, table, 1, 1e-6)
        inside(qo[:n], want, tol)
        assert torch.isnan(qo[n:]).all()


def test_append_rounds_fp32_rows_to_bf16_once(cp):
    b = R.make_batch([(3, 4)], bf16=True)
    k = torch.randn(4, 8, 64, device="cuda")
    v = k * (1 + 2.0 ** -9)
    cp.attn_append_paged_bf16kv(k, v, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"])
    page, slot = b["table"][0, 0].long(), torch.arange(3, 7, device="cuda")
    assert torch.equal(b["kp"][page, slot], k.to(BF)) and torch.equal(b["vp"][page, slot], v.to(BF))


def test_append_skips_what_is_out_of_range(cp):
    """A row past the table, a page past the pool, a negative page and a negative
    context are recorded and not stored; the other rows are."""
    b = R.make_batch([(14, 4), (16, 2), (0, 2), (3, 1)], spare=2)
    table = b["table"].clone()[:, :1].contiguous()  # tokens 16 .. have no entry
    table[2, 0] = b["kp"].shape[0]
    ctx = b["ctx"].clone()
    ctx[3] = -4
    before = b["kp"].clone(), b["vp"].clone()
    k, v = torch.randn(9, 8, 64, device="cuda"), torch.randn(9, 8, 64, device="cuda")
    assert cp.attn_get_device_error() == 0
    cp.attn_append_paged(k, v, b["kp"], b["vp"], table, ctx, b["starts"])
    assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    page = b["table"][0, 0].long()
    for pool, old, src in ((b["kp"], before[0], k), (b["vp"], before[1], v)):
        assert torch.equal(pool[page, 14:16], src[0:2])
        pool[page, 14:16] = old[page, 14:16]
        assert torch.equal(pool.view(torch.int32), old.view(torch.int32))


def test_append_with_a_row_start_far_below_zero(cp):
    """Rows 2^31 and more behind their sequence's first: past the table, recorded, not stored."""
    b = R.make_batch([(0, 3)])
    before = b["kp"].clone()
    k = torch.randn(3, 8, 64, device="cuda")
    starts = torch.tensor([-2 ** 31, 3], dtype=torch.int32, device="cuda")
    assert cp.attn_get_device_error() == 0
    cp.attn_append_paged(k, k, b["kp"], b["vp"], b["table"], b["ctx"], starts)
    assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    assert torch.equal(b["kp"].view(torch.int32), before.view(torch.int32))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens", [[(0, 1)], [(5, 64), (16, 17), (0, 33), (100, 2), (7, 0)],
                                  [(40, 20)] * 37])
def test_compact(cp, bf16, lens):
    b = R.make_batch(lens, bf16=bf16, seed=4)
    rng = np.random.default_rng(len(lens))
    width = b["max_rows"]
    keep = np.full((len(lens), width), -1, dtype=np.int32)  # entries past a count are not read
    counts = []
    for s, (_, t) in enumerate(lens):
        n = int(rng.integers(0, t + 1)) if s % 3 else t
        keep[s, :n] = np.sort(rng.permutation(t)[:n])
        counts.append(n)
    want = b["kp"].clone(), b["vp"].clone()
    for s, (c, _) in enumerate(lens):
        for i in range(counts[s]):
            a, z = c + int(keep[s, i]), c + i
            for pool in want:
                pool[b["table"][s, z // 16].long(), z % 16] = pool[b["table"][s, a // 16].long(), a % 16].clone()
    call = cp.attn_compact_paged_bf16kv if bf16 else cp.attn_compact_paged
    call(b["kp"], b["vp"], b["table"], b["ctx"], torch.from_numpy(keep).cuda(),
         torch.tensor(counts, dtype=torch.int32, device="cuda"), b["max_rows"])
    assert cp.attn_get_device_error() == 0
    raw = torch.int16 if bf16 else torch.int32
    assert torch.equal(b["kp"].view(raw), want[0].view(raw)) and torch.equal(b["vp"].view(raw), want[1].view(raw))


@pytest.mark.parametrize("what", ["falling", "equal", "negative", "past", "count", "page", "context"])
def test_compact_leaves_a_bad_sequence_alone(cp, what):
    b = R.make_batch([(10, 8), (20, 8)])
    keep = torch.tensor([[1, 3, 5, 7], [1, 3, 5, 7]], dtype=torch.int32, device="cuda")
    counts = torch.tensor([4, 4], dtype=torch.int32, device="cuda")
    table, ctx = b["table"].clone(), b["ctx"].clone()
    if what == "falling":
        keep[0, 2] = 2
    elif what == "equal":
        keep[0, 1] = 1
    elif what == "negative":
        keep[0, 0] = -1
    elif what == "past":
        keep[0, 3] = 8
    elif what == "count":
        counts[0] = 5
    elif what == "page":
        table[0, 1] = -1
    else:
        ctx[0] = -1
    want = b["kp"].clone(), b["vp"].clone()
    for i, r in enumerate((1, 3, 5, 7)):
        a, z = 20 + r, 20 + i
        for pool in want:
            pool[table[1, z // 16].long(), z % 16] = pool[table[1, a // 16].long(), a % 16].clone()
    assert cp.attn_get_device_error() == 0
    cp.attn_compact_paged(b["kp"], b["vp"], table, ctx, keep, counts, 8)
    assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    assert torch.equal(b["kp"].view(torch.int32), want[0].view(torch.int32))
    assert torch.equal(b["vp"].view(torch.int32), want[1].view(torch.int32))
