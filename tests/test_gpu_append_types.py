"""Appends whose rows and pages are of either type each, against the plain form in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402
from test_gpu_rows import inside, make_table  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


@pytest.mark.parametrize("act", [F, BF])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("with_q", [False, True])
@pytest.mark.parametrize("pairing", [0, 1])
def test_append_of_either_type(cp, act, bf16, with_q, pairing):
    lens = [(5, 7), (0, 3), (31, 0), (100, 41)]
    b = R.make_batch(lens, bf16=bf16, seed=5)
    raw = torch.int16 if bf16 else torch.int32
    before = b["kp"].clone(), b["vp"].clone()
    n = b["n"]
    kv = torch.randn(n, 16, 64, device="cuda").to(act)
    k, v = kv[:, :8], kv[:, 8:]
    q = torch.randn(n, 33, 64, device="cuda").to(act)[:, 1:] if with_q else None
    qo = torch.full((n, 32, 64), float("nan"), device="cuda") if with_q else None
    w, table = torch.randn(64, device="cuda"), make_table(cp, 200)
    call = cp.attn_append_paged_bf16kv if bf16 else cp.attn_append_paged
    call(k, v, b["kp"], b["vp"], b["table"], b["ctx"], b["starts"], table, kWeight=w, q=q, qOut=qo, qWeight=w,
         pairing=pairing)
    assert cp.attn_get_device_error() == 0
    seq = torch.tensor([s for s, (_, t) in enumerate(lens) for _ in range(t)], device="cuda")
    tok = torch.tensor([c + i for c, t in lens for i in range(t)], device="cuda")
    page, slot = b["table"].long()[seq, tok // 16], tok % 16
    want, tol = R.norm_rotate_reference(k, w, tok, table, pairing, 1e-6)
    inside(b["kp"][page, slot], want, R.stored(want, tol, b["kp"].dtype))
    assert torch.equal(b["vp"][page, slot], v.to(b["vp"].dtype))
    for pool, old in zip((b["kp"], b["vp"]), before):  # everything else is as it was
        pool[page, slot] = old[page, slot]
        assert torch.equal(pool.view(raw), old.view(raw))
    if with_q:
        want, tol = R.norm_rotate_reference(q, w, tok, table, pairing, 1e-6)
        inside(qo, want, tol + 1e-37)
