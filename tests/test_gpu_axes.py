"""attn_qk_norm_rope_axes and attn_append_paged_axes (both page types) against plain forms
in 64 bits, and bit by bit against the calls with one position a row."""
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
LAYOUTS = {
    "sections": [0] * 8 + [1] * 12 + [2] * 12,
    "odd sections": [0] * 11 + [1] * 11 + [2] * 10,
    "interleaved": [i % 3 for i in range(32)],
    "one": [0] * 32,
    "four": [(7 * i) % 4 for i in range(32)],
}


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


def make_table(cp, n):
    return cp.attn_rope_table(torch.empty(n, 64, device="cuda"))


def inside(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() / tol.clamp(min=1e-300)).max()))


def reference(x, weight, positions, axes, table, pairing, eps):
    """Each pair of dims by its own axis: columns of the one-position form's results."""
    want = tol = None
    for a in sorted(set(axes)):
        y, t = R.norm_rotate_reference(x, weight, positions[a].long(), table, pairing, eps)
        if want is None:
            want, tol = y.clone(), t.clone()
        for i in range(32):
            if axes[i] == a:
                dims = [i, i + 32] if pairing == 0 else [2 * i, 2 * i + 1]
                want[..., dims], tol[..., dims] = y[..., dims], t[..., dims]
    return want, tol


@pytest.mark.parametrize("n", [1, 2, 33, 300])
@pytest.mark.parametrize("act,out", [(F, F), (F, BF), (BF, F), (BF, BF)])
@pytest.mark.parametrize("pairing", [0, 1])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_norm_rope_axes(cp, n, act, out, pairing, layout):
    axes, gen = LAYOUTS[layout], torch.Generator(device="cuda").manual_seed(n * 8 + pairing)
    count = max(axes) + 1
    wide = torch.randn(n, 50, 64, generator=gen, device="cuda").to(act)
    q, k = wide[:, 1:33], wide[:, 40:48]  # views with 50 heads between rows
    table = make_table(cp, 5000)
    pos = torch.randint(0, 5000, (count, n + 3), generator=gen, device="cuda").to(torch.int32)[:, :n]
    pos[:, 0] = 4999
    qw, kw = (torch.randn(64, generator=gen, device="cuda") for _ in range(2))
    qo = torch.full((n, 32, 64), float("nan"), device="cuda")
    ko = torch.full((n, 8, 64), float("nan"), device="cuda", dtype=out)
    cp.attn_qk_norm_rope_axes(q, k, pos, axes, table, qo, ko, qWeight=qw, kWeight=kw, eps=1e-5, pairing=pairing)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        want, tol = reference(x, w, pos, axes, table, pairing, 1e-5)
        inside(got, want, R.stored(want, tol, got.dtype))
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("pairing", [0, 1])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_equal_positions_are_one_position(cp, pairing, layout):
    """Rows of text, by an expanded tensor (all axes share one array): the same bits."""
    n, axes = 41, LAYOUTS[layout]
    q, k = torch.randn(n, 32, 64, device="cuda"), torch.randn(n, 8, 64, device="cuda")
    table, pos = make_table(cp, 900), torch.randint(0, 900, (n,), device="cuda").to(torch.int32)
    w, outs = torch.randn(64, device="cuda"), []
    for call in (lambda a, b: cp.attn_qk_norm_rope(q, k, pos, table, a, b, qWeight=w, pairing=pairing),
                 lambda a, b: cp.attn_qk_norm_rope_axes(q, k, pos.expand(max(axes) + 1, n), axes, table, a, b, qWeight=w,
                                                        pairing=pairing)):
        a, b = torch.empty_like(q), torch.empty_like(k)
        call(a, b)
        outs.append((a, b))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_in_place_and_keys_only(cp):
    n, axes = 19, LAYOUTS["interleaved"]
    k = torch.randn(n, 8, 64, device="cuda")
    k0, table = k.clone(), make_table(cp, 64)
    pos = torch.randint(0, 64, (3, n), device="cuda").to(torch.int32)
    cp.attn_qk_norm_rope_axes(None, k, pos, axes, table, None, k)
    want, tol = reference(k0, None, pos, axes, table, 0, 1e-6)
    inside(k, want, tol)


def test_positions_out_of_range_are_recorded_and_clamped(cp):
    k, axes = torch.randn(3, 8, 64, device="cuda"), LAYOUTS["sections"]
    table, ko = make_table(cp, 10), torch.empty(3, 8, 64, device="cuda")
    pos = torch.tensor([[1, 3, 10], [-5, 0, 9], [2, 2, 2147483647]], dtype=torch.int32, device="cuda")
    assert cp.attn_get_device_error() == 0
    cp.attn_qk_norm_rope_axes(None, k, pos, axes, table, None, ko)
    assert cp.attn_get_device_error() == cp.ATTN_EBOUNDS
    want, tol = reference(k, None, pos.clamp(0, 9), axes, table, 0, 1e-6)
    inside(ko, want, tol)


@pytest.mark.parametrize("lens", [[(0, 1), (15, 1), (1000, 1)], [(5, 7), (31, 0), (17, 64), (100, 1)], [(100, 300)]])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("layout,pairing", [("sections", 0), ("interleaved", 0), ("odd sections", 1)])
def test_append_axes(cp, lens, bf16, layout, pairing):
    axes, b, pad = LAYOUTS[layout], R.make_batch(lens, bf16=bf16, seed=3), 5  # rows behind the last sequence
    before, n, act = (b["kp"].clone(), b["vp"].clone()), b["n"], BF if bf16 else F
    kv = torch.randn(n + pad, 16, 64, device="cuda").to(act)
    k, v, q = kv[:, :8], kv[:, 8:], torch.randn(n + pad, 32, 64, device="cuda").to(act)
    qo = torch.full((n + pad, 32, 64), float("nan"), device="cuda")
    w, table = torch.randn(64, device="cuda"), make_table(cp, 700)
    pos = torch.randint(0, 700, (3, n + pad), device="cuda").to(torch.int32)
    call = cp.attn_append_paged_axes_bf16kv if bf16 else cp.attn_append_paged_axes
    call(k, v, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], table, pos, axes, kWeight=w, q=q, qOut=qo, qWeight=w,
         pairing=pairing)
    assert cp.attn_get_device_error() == 0
    assert qo[n:].isnan().all()
    want, tol = reference(q[:n], w, pos[:, :n], axes, table, pairing, 1e-6)
    inside(qo[:n], want, tol)
    want, tol = reference(k[:n], w, pos[:, :n], axes, table, pairing, 1e-6)
    tol, r = R.stored(want, tol, b["kp"].dtype), 0
    for s, (c, t) in enumerate(lens):
        tok = torch.arange(c, c + t, device="cuda")
        page, slot = b["table"][s].long()[tok // 16], tok % 16
        inside(b["kp"][page, slot], want[r:r + t], tol[r:r + t])
        assert torch.equal(b["vp"][page, slot], v[r:r + t].to(b["vp"].dtype))
        for pool, old in zip((b["kp"], b["vp"]), before):
            pool[page, slot] = old[page, slot]
        r += t
    for pool, old in zip((b["kp"], b["vp"]), before):  # and nothing else was written
        bits = torch.int16 if bf16 else torch.int32
        assert torch.equal(pool.view(bits), old.view(bits))


def test_refusals(cp):
    k, table = torch.randn(3, 8, 64, device="cuda"), make_table(cp, 8)
    pos, ko = torch.zeros(3, 3, dtype=torch.int32, device="cuda"), torch.empty(3, 8, 64, device="cuda")
    ok = LAYOUTS["sections"]
    for p, a, wrong in ((pos[:, :2], ok, ValueError), (pos[0], ok, ValueError), (pos.T.contiguous().T, ok, ValueError),
                        (pos.long(), ok, ValueError), (pos.cpu(), ok, ValueError), (pos, ok[:31], ValueError),
                        (pos, 3, TypeError), (pos, [0.5] * 32, TypeError), (None, ok, TypeError)):
        with pytest.raises(wrong):
            cp.attn_qk_norm_rope_axes(None, k, p, a, table, None, ko)
    for p, a, code in ((pos[:2], ok, cp.ATTN_EINVAL), (pos, [-1] * 32, cp.ATTN_EINVAL),
                       (torch.zeros(5, 3, dtype=torch.int32, device="cuda"), ok, cp.ATTN_ERANGE)):
        with pytest.raises(cp.AttnError) as e:
            cp.attn_qk_norm_rope_axes(None, k, p, a, table, None, ko)
        assert e.value.code == code
    with pytest.raises(cp.AttnError):
        cp.attn_qk_norm_rope_axes(None, k, pos, ok, None, None, ko)
    empty = torch.empty(0, 8, 64, device="cuda")
    cp.attn_qk_norm_rope_axes(None, empty, torch.zeros(3, 0, dtype=torch.int32, device="cuda"), ok, table, None, empty)
