"""The calls on cache weights from a host thread that has made no CUDA call: their kernels
take tensor maps and clusters, whose set-up needs a context. (The C interface: PyTorch's
own bookkeeping would bind one.)"""
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


@pytest.mark.parametrize("kind", ["", "_bf16kv"])
@pytest.mark.parametrize("name", ["attn_decode_weigh_paged", "attn_weigh_paged", "attn_evict_paged"])
def test_a_thread_whose_first_cuda_call_it_is(cp, name, kind):
    dtype = torch.bfloat16 if kind else torch.float32
    n, rows = 60, 4
    q = torch.randn(rows, 32, 64, device="cuda")
    pages = [torch.randn(4, 16, 8, 64, device="cuda").to(dtype) for _ in range(2)]
    weights = torch.rand(4, 8, 16, device="cuda")
    ids = torch.arange(4, dtype=torch.int32, device="cuda")
    lens, keep = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (n, 30))
    starts = torch.tensor([0, rows], dtype=torch.int32, device="cuda")

    def call(state):
        k, v, w, out = (t.data_ptr() for t in state)
        if name == "attn_decode_weigh_paged":
            return cp.raw(name + kind)(q.data_ptr(), k, v, w, ids.data_ptr(), lens.data_ptr(), None, 1.0, out, 1, 4, 4, n, None, 0,
                                       None)
        if name == "attn_weigh_paged":
            return cp.raw(name + kind)(q.data_ptr(), k, w, ids.data_ptr(), lens.data_ptr(), starts.data_ptr(), None, 1.0, 1, rows,
                                       rows, 4, 4, n, None, 0, None)
        return cp.raw(name + kind)(k, v, w, ids.data_ptr(), lens.data_ptr(), keep.data_ptr(), 2, 3, 1, 4, 4, n, None, 0, None)

    states = [[t.clone() for t in (*pages, weights)] + [torch.zeros(1, 32, 64, device="cuda")] for _ in range(2)]
    torch.cuda.synchronize()
    codes = [call(states[0])]
    t = threading.Thread(target=lambda: codes.append(call(states[1])))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert codes == [cp.ATTN_OK, cp.ATTN_OK]
    assert all(torch.equal(a, b) for a, b in zip(*states))
    assert not torch.equal(states[0][2], weights)  # something was done
    assert cp.attn_get_device_error() == 0
