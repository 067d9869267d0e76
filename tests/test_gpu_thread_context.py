"""Every entry point whose kernels take tensor maps, from a host thread that has made
no CUDA call: the driver's encoder needs a context that such a thread does not have
yet. (The C interface: PyTorch's own bookkeeping would bind one.)"""
import threading

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


NAMES = ["attn_prefill", "attn_prefill_bf16x3", "attn_prefill_bf16kv", "attn_prefill_paged", "attn_decode_paged",
         "attn_tree_paged", "attn_tree_paged_bf16kv"]


@pytest.mark.parametrize("name", NAMES)
def test_a_thread_whose_first_cuda_call_it_is(cp, name):
    C, P = 4, 60
    q = torch.randn(C, 32, 64, device="cuda")
    k, v = torch.randn(P + C, 8, 64, device="cuda"), torch.randn(P + C, 8, 64, device="cuda")
    if "bf16kv" in name:
        k, v = k.bfloat16(), v.bfloat16()
    ids = torch.arange(4, dtype=torch.int32, device="cuda")
    lens = torch.tensor([P], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, C], dtype=torch.int32, device="cuda")
    outs = [torch.full((C, 32, 64), float("nan"), device="cuda") for _ in range(2)]

    def call(out):
        p = [t.data_ptr() for t in (q, k, v)]
        if name.startswith("attn_tree"):
            return cp.raw(name)(*p, ids.data_ptr(), lens.data_ptr(), starts.data_ptr(), None, out.data_ptr(), 1, C, C, 4,
                                4, P, 1, None, 0, None)
        if name == "attn_decode_paged":
            return cp.raw(name)(*p, ids.data_ptr(), lens.data_ptr(), out.data_ptr(), 1, 4, 4, P, 1, None, 0, None)
        if name == "attn_prefill_paged":
            return cp.raw(name)(*p, ids.data_ptr(), out.data_ptr(), C, P, 4, None)
        return cp.raw(name)(*p, out.data_ptr(), C, P, None)

    torch.cuda.synchronize()
    codes = [call(outs[0])]
    t = threading.Thread(target=lambda: codes.append(call(outs[1])))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert codes == [cp.ATTN_OK, cp.ATTN_OK]
    assert torch.equal(*[o.nan_to_num(nan=7.0) for o in outs]) and not torch.isnan(outs[1][0]).any()
    assert cp.attn_get_device_error() == 0
