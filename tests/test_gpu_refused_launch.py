"""A launch that the runtime refuses is reported by its own call and by no later one.
The refusal is made on the host: a stream whose capture has been invalidated takes
no launch."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


def runtime():
    """The CUDA runtime that PyTorch has loaded."""
    with open("/proc/self/maps") as f:
        paths = {line.split()[-1] for line in f if "libcudart" in line}
    assert paths, "no shared CUDA runtime in the process"
    return ctypes.CDLL(sorted(paths)[0])


class RefusingStream:
    """A stream in a capture that was invalidated by a wait for it."""

    def __enter__(self):
        self.rt, self.stream = runtime(), ctypes.c_void_p()
        assert self.rt.cudaStreamCreateWithFlags(ctypes.byref(self.stream), 1) == 0
        assert self.rt.cudaStreamBeginCapture(self.stream, 2) == 0  # relaxed: other streams are free
        assert self.rt.cudaStreamSynchronize(self.stream) != 0
        self.rt.cudaGetLastError()  # (PyTorch's runtime: the library has its own)
        return self.stream.value

    def __exit__(self, *exc):
        graph = ctypes.c_void_p()
        assert self.rt.cudaStreamEndCapture(self.stream, ctypes.byref(graph)) != 0 and not graph.value
        self.rt.cudaGetLastError()
        assert self.rt.cudaStreamDestroy(self.stream) == 0


def calls(cp):
    """{name: call on a given stream} of the entry points, with what they read kept alive."""
    f = dict(device="cuda")
    q, k, out = torch.randn(4, 32, 64, **f), torch.randn(4, 8, 64, **f), torch.empty(4, 32, 64, **f)
    k2 = torch.empty_like(k)
    i32 = dict(device="cuda", dtype=torch.int32)
    pages, vpages = torch.randn(300, 16, 8, 64, **f), torch.randn(300, 16, 8, 64, **f)
    table, ctx, starts = torch.arange(256, **i32).view(1, 256), torch.tensor([4000], **i32), torch.tensor([0, 4], **i32)
    keep, counts, cs = torch.zeros(1, 1, **i32), torch.ones(1, **i32), torch.empty(8, 64, **f)
    ws = torch.empty(1 << 24, dtype=torch.uint8, **f)
    long_k, long_v = torch.randn(4004, 8, 64, **f), torch.randn(4004, 8, 64, **f)
    bk, bv = long_k.bfloat16(), long_v.bfloat16()
    ids = torch.arange(251, **i32)
    tree = (q, pages, vpages, table, ctx, starts, None, out, 4, 4000)
    return {
        "attn_rope_table": lambda st=None: cp.attn_rope_table(cs, stream=st),
        "attn_qk_norm_rope": lambda st=None: cp.attn_qk_norm_rope(q, k, None, None, out, k2, stream=st),
        "attn_append_paged": lambda st=None: cp.attn_append_paged(k, k, pages, vpages, table, ctx, starts, stream=st),
        "attn_tree_paged": lambda st=None: cp.attn_tree_paged(*tree, num_splits=1, stream=st),
        "attn_tree_paged, merged through memory": lambda st=None: cp.attn_tree_paged(*tree, num_splits=20, workspace=ws,
                                                                                     stream=st),
        "attn_compact_paged": lambda st=None: cp.attn_compact_paged(pages, vpages, table, ctx, keep, counts, 4, stream=st),
        "attn_prefill": lambda st=None: cp.attn_prefill(q, long_k, long_v, out, 4000, stream=st),
        "attn_prefill_bf16kv": lambda st=None: cp.attn_prefill_bf16kv(q, bk, bv, out, 4000, stream=st),
        "attn_prefill_paged": lambda st=None: cp.attn_prefill_paged(q, pages, vpages, ids, out, 4000, stream=st),
        "attn_decode_paged": lambda st=None: cp.attn_decode_paged(q[:1], pages, vpages, table, ctx, out[:1], 4000, 8, ws,
                                                                  stream=st),
    }


NAMES = ["attn_rope_table", "attn_qk_norm_rope", "attn_append_paged", "attn_tree_paged",
         "attn_tree_paged, merged through memory", "attn_compact_paged", "attn_prefill", "attn_prefill_bf16kv",
         "attn_prefill_paged", "attn_decode_paged"]


@pytest.mark.parametrize("name", NAMES)
def test_a_refused_launch_is_not_reported_by_the_next_call(cp, name):
    call = calls(cp)
    call[name]()  # every set-up of the entry point is done
    torch.cuda.synchronize()
    with RefusingStream() as stream:
        with pytest.raises(cp.AttnError) as e:
            call[name](stream)
        assert e.value.code == cp.ATTN_ELAUNCH
    call["attn_rope_table"]()  # returns the runtime's last error
    call[name]()
    torch.cuda.synchronize()
    assert cp.attn_get_device_error() == 0
