"""Cache weights where the numbers are large: scores in the hundreds from ordinary values, whose
products round, and finite operands next to their type's largest number. Decode step and
window, one launch and two, both page types, against the plain forms in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402
import weights_ref as W  # noqa: E402
from test_gpu_weights import check_weights, decode, inside, ints, weigh  # noqa: E402

pytestmark = pytest.mark.gpu
F32_MAX, BF16_MAX = torch.finfo(torch.float32).max, torch.finfo(torch.bfloat16).max


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


def queries(n, seed):
    return torch.randn(n, 32, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))


def check_decode(cp, b, q, bound=None):
    weighed = [max(0, c - 3) for c, _ in b["lens"]]
    w = W.weight_pool(b, known=weighed)
    before = w.clone()
    out = decode(cp, b, q, w, 0.9, ints(weighed), bound=bound)
    assert cp.attn_get_device_error() == 0
    want, ref, tol = W.weigh_reference(q, b, before, weighed, 0.9, decode=True)
    inside(out, ref, tol)
    check_weights(w, before, b, want)


def check_window(cp, b, q, bound=None):
    weighed = [max(0, c - 3) for c, _ in b["lens"]]
    w = W.weight_pool(b, known=weighed)
    before = w.clone()
    weigh(cp, b, q, w, 0.9, ints(weighed), bound=bound)
    assert cp.attn_get_device_error() == 0
    check_weights(w, before, b, floored(W.weigh_reference(q, b, before, weighed, 0.9), b))


def floored(want, b):
    """A probability below 2^-126 may come out as 0: 4 heads of each row, that much each."""
    return [pair and (pair[0], pair[1] + 4 * t * 2.0 ** -126) for pair, (_, t) in zip(want, b["lens"])]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("size", [30, 150])  # scores of up to 100 and 500
@pytest.mark.parametrize("bound", [None, 30000])
def test_scores_in_the_hundreds(cp, bf16, size, bound):
    extra = 2000 if bound else 0
    b = R.make_batch([(700, 0), (33, 0), (2000, 0)], bf16=bf16, seed=41, extra_blocks=extra)
    q = queries(3, 42) * size
    weighed = [700, 33, 2000]  # all have a weight, which the smallest probabilities vanish in
    w = W.weight_pool(b)
    before = w.clone()
    out = decode(cp, b, q, w, 1.0, ints(weighed), bound=bound)
    want, ref, tol = W.weigh_reference(q, b, before, weighed, 1.0, decode=True)
    inside(out, ref, tol)
    check_weights(w, before, b, want)
    for lens in ([(700, 8)], [(2500, 32)], [(700, 40), (100, 8)], [(3000, 70), (0, 20)]):
        b = R.make_batch(lens, bf16=bf16, seed=43, extra_blocks=extra)
        check_window(cp, b, queries(b["n"], 44) * size, bound)


FAR = [(False, F32_MAX), (False, -F32_MAX), (False, 2.0 ** 128 - 2.0 ** 115), (True, BF16_MAX), (True, -BF16_MAX)]
SHAPES = [([(70, 3)], None), ([(70, 8)], 30000), ([(500, 40)], None), ([(70, 70)], None)]


def place(b, token):
    return b["table"][0, token // 16].long(), token % 16


@pytest.mark.parametrize("bf16,value", FAR)
@pytest.mark.parametrize("lens,bound", SHAPES)
def test_a_largest_key(cp, bf16, value, lens, bound):
    """One dim of a key, met by queries of zero there; and one of 2^101 met by 2^-100 (a score of 1/4)."""
    b = R.make_batch(lens, bf16=bf16, seed=45, extra_blocks=2000 if bound else 0)
    page, slot = place(b, 20)
    b["kp"][page, slot, :, 5] = value
    b["kp"][..., 6] = 0.0
    page, slot = place(b, 33)
    b["kp"][page, slot, :, 6] = 2.0 ** 101 if value > 0 else -2.0 ** 101
    q = queries(b["n"], 46)
    q[:, :, 5] = 0.0
    q[:, :, 6] = 2.0 ** -100
    check_window(cp, b, q, bound)
    check_decode(cp, dict(b, lens=[(c, 0) for c, _ in lens]), q[:1].contiguous(), bound)


@pytest.mark.parametrize("bf16,value", FAR)
@pytest.mark.parametrize("bound", [None, 30000])
def test_a_largest_value(cp, bf16, value, bound):
    """With queries of zero every key weighs alike, so that the weighted sum stays in range."""
    b = R.make_batch([(70, 0)], bf16=bf16, seed=47, extra_blocks=2000 if bound else 0)
    page, slot = place(b, 20)
    b["vp"][page, slot, :, ::3] = value
    check_decode(cp, b, torch.zeros(1, 32, 64, device="cuda"), bound)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("value", [F32_MAX, -F32_MAX, 2.0 ** 128 - 2.0 ** 115, 2.0 ** 128 - 2.0 ** 119])
@pytest.mark.parametrize("lens,bound", SHAPES)
def test_a_largest_query(cp, bf16, value, lens, bound):
    """One dim of the queries, met by 2^-110 in one key and zeros in the others: a score of 2^15 in
    magnitude against zeros, so that the key's probability is 1, or 0 and the others' alike."""
    b = R.make_batch(lens, bf16=bf16, seed=48, extra_blocks=2000 if bound else 0)
    b["kp"][..., 5] = 0.0
    page, slot = place(b, 33)
    b["kp"][page, slot, :, 5] = 2.0 ** -110
    c, t = lens[0]
    w = W.weight_pool(b)
    before = w.clone()
    q = torch.zeros(t, 32, 64, device="cuda")
    q[:, :, 5] = value
    weigh(cp, b, q, w, 0.0, bound=bound)
    n, i = c + t, torch.arange(t, device="cuda")
    seen = torch.arange(n, device="cuda")[None] <= (c + i)[:, None]
    p = torch.zeros(t, n, dtype=torch.float64, device="cuda")
    if value > 0:
        p[:, 33] = 1.0
    else:
        p = seen.double()
        p[:, 33] = 0.0
        p /= p.sum(-1, keepdim=True)
    want = (4 * p.sum(0))[:, None].expand(n, 8)
    # A score is a sum of q's terms times a power of two, two additions that round by 2^-23 of it in either
    # pass (zeros add exactly), and its reference is subtracted in three terms; in the exponent, times
    # log2 e. Where the key gives nothing the others' scores are exactly 0.
    rel = (2 * 2 + 3) * 2.0 ** -23 * 2.0 ** 15 * 1.4427 if value > 0 else 2.0 ** -18
    tol = want * rel + (70 + t) * 2.0 ** -24 * want
    check_weights(w, before, b, [(want, tol)])
    q1 = q[:1].contiguous()
    one = dict(b, lens=[(c, 0)], ctx=ints([c]))
    w = before.clone()
    out = decode(cp, one, q1, w, 0.0, ints([0]), bound=bound)
    v = R.gather(b["vp"], b["table"][0], c)
    ref = v[33] if value > 0 else (v.sum(0) - v[33]) / (c - 1)
    ref = ref.repeat_interleave(4, 0)[None]
    inside(out, ref, 2.0 ** -17 * v.abs().amax(0).repeat_interleave(4, 0)[None])
    assert cp.attn_get_device_error() == 0
