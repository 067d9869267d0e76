"""Finite operands at the edge of their type's range through the drafted-tree
attention: what a row does not see has no influence on it, and what it sees gives
the formula's finite value. The term splits round, and a rounded first term of
such a value would be infinite."""
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402
from test_gpu_tree import check, queries, run  # noqa: E402

pytestmark = pytest.mark.gpu
F32_MAX, BF16_MAX = torch.finfo(torch.float32).max, torch.finfo(torch.bfloat16).max


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


def far(bf16):
    """The type's largest value, and on fp32 pages the least whose 11 upper bits round up to infinity."""
    return [BF16_MAX, -BF16_MAX] if bf16 else [F32_MAX, -F32_MAX, 2.0 ** 128 - 2.0 ** 115, 2.0 ** 115 - 2.0 ** 128]


CASES = [(bf16, value) for bf16 in (False, True) for value in far(bf16)]
# (rows, stated bound of the context, segments): each kernel of a page type, whole and cut
SHAPES = [(3, 70, 0), (8, 70, 0), (8, 17000, 1), (24, 17000, 1), (24, 17000, 5), (8, 17000, 40)]


def place(b, token):
    return b["table"][0, token // 16].long(), token % 16


@pytest.mark.parametrize("bf16,value", CASES)
@pytest.mark.parametrize("rows,bound,splits", SHAPES)
def test_a_largest_value_reaches_the_rows_that_see_it(cp, bf16, value, rows, bound, splits):
    """A drafted row's value is hidden from all rows but two, whose queries are zero:
    every key weighs 1, so that the weighted sum itself stays in range."""
    lens = [(70, rows)]
    b = R.make_batch(lens, bf16=bf16, seed=61, extra_blocks=1100)
    masks = R.tree_masks(lens, "self")
    masks[2] = 0b101
    q = queries(rows, seed=5)
    q[[0, 2]] = 0.0
    b["vp"][place(b, 70)] = value
    check(run(cp, b, q, masks, bf16, splits, max_context=bound), *R.tree_reference(q, b, masks))
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("bf16,value", CASES)
@pytest.mark.parametrize("rows,bound,splits", SHAPES)
def test_a_largest_value_of_the_context(cp, bf16, value, rows, bound, splits):
    lens = [(70, rows)]
    b = R.make_batch(lens, bf16=bf16, seed=63, extra_blocks=1100)
    masks, q = R.tree_masks(lens), torch.zeros(rows, 32, 64, device="cuda")
    page, slot = place(b, 20)
    b["vp"][page, slot, :, ::3] = value
    check(run(cp, b, q, masks, bf16, splits, max_context=bound), *R.tree_reference(q, b, masks))
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("bf16,value", CASES)
@pytest.mark.parametrize("rows,bound,splits", SHAPES)
def test_a_largest_key(cp, bf16, value, rows, bound, splits):
    """One dim of a key in the context, met by queries of 2^-125 there (a score of +-1, and
    a power of two: one term); and a whole drafted key that all rows but one are blind to."""
    lens = [(70, rows)]
    b = R.make_batch(lens, bf16=bf16, seed=64, extra_blocks=1100)
    masks, q = R.tree_masks(lens, "self"), queries(rows, seed=6)
    q[:, :, 5] = 2.0 ** -125
    page, slot = place(b, 20)
    b["kp"][page, slot, :, 5] = value
    want, tol = R.tree_reference(q, b, masks)
    page, slot = place(b, 71)  # row 1's
    b["kp"][page, slot] = value
    got = run(cp, b, q, masks, bf16, splits, max_context=bound)
    blind = [i for i in range(rows) if i != 1]
    check(got[blind], want[blind], tol[blind])
    assert cp.attn_get_device_error() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("value", [F32_MAX, -F32_MAX, 2.0 ** 128 - 2.0 ** 115, 2.0 ** 128 - 2.0 ** 119])
@pytest.mark.parametrize("rows,bound,splits", SHAPES)
def test_a_largest_query(cp, bf16, value, rows, bound, splits):
    """One dim of a query, met by 2^-110 in one key and zeros in the others: all of its
    weight is on that key, or none."""
    lens = [(70, rows)]
    b = R.make_batch(lens, bf16=bf16, seed=66, extra_blocks=1100)
    b["kp"][..., 5] = 0.0
    page, slot = place(b, 33)
    b["kp"][page, slot, :, 5] = 2.0 ** -110
    masks, q = R.tree_masks(lens), queries(rows, seed=7)
    q[1] = 0.0
    q[1, :, 5] = value
    got = run(cp, b, q, masks, bf16, splits, max_context=bound)
    want, tol = R.tree_reference(q, b, masks)
    # row 1's score is +-2^15 against zeros: its weights are 1 and 0, or 0 and alike
    if value > 0:
        v = b["vp"][page, slot].double().repeat_interleave(4, 0)
        want[1], tol[1] = v, 2.0 ** -18 * v.abs()
    check(got, want, tol)
    assert cp.attn_get_device_error() == 0
