"""The calls on cache weights in the forms that need a workspace (two launches, the second of
which reads what it may before the first has ended): captured and replayed without the
host between, one after another on one workspace, and on two streams with one each."""
import pytest

torch = pytest.importorskip("torch")
import spec_ref as R  # noqa: E402
import weights_ref as W  # noqa: E402
from test_gpu_evict import evict  # noqa: E402
from test_gpu_weights import bits, decode, ints, weigh, workspace  # noqa: E402

pytestmark = pytest.mark.gpu
STEPS = 4


@pytest.fixture(scope="module")
def cp():
    from chunked_prefill_gqa_gb300 import build
    build.build()
    import chunked_prefill_gqa_gb300 as m
    return m


class Step:
    """A window of 70 rows, a decode step and an eviction of one sequence or two, each with a bound that
    makes it two launches; the lengths stay, so that a step can follow another."""

    def __init__(self, cp, lens, bf16, seed):
        self.cp = cp
        self.b = R.make_batch(lens, bf16=bf16, seed=seed, extra_blocks=1900)
        self.grown = dict(self.b, lens=[(c + t, 0) for c, t in lens], ctx=ints([c + t for c, t in lens]))
        self.keep = ints([(c + t) * 2 // 3 for c, t in lens])
        self.w = W.weight_pool(self.b)
        gen = torch.Generator("cuda").manual_seed(seed)
        self.q = torch.randn(self.b["n"], 32, 64, device="cuda", generator=gen)
        self.qd = torch.randn(len(lens), 32, 64, device="cuda", generator=gen)
        self.out = torch.full_like(self.qd, float("nan"))
        sizes = (cp.attn_weigh_workspace_bytes(len(lens), self.b["n"], 70, 30000),
                 cp.attn_decode_weigh_workspace_bytes(len(lens), 30000), cp.attn_evict_workspace_bytes(len(lens), 30000))
        assert min(sizes) > 0
        self.ws = workspace(max(sizes))  # one for all three, one after another

    def run(self, stream=None):
        weigh(self.cp, self.b, self.q, self.w, 0.9, bound=30000, rows=70, ws=self.ws, stream=stream)
        call = self.cp.attn_decode_weigh_paged_bf16kv if self.b["kp"].dtype == torch.bfloat16 else self.cp.attn_decode_weigh_paged
        call(self.qd, self.b["kp"], self.b["vp"], self.w, self.b["table"], self.grown["ctx"], self.out, 30000, decay=0.95,
             workspace=self.ws, stream=stream)
        call = self.cp.attn_evict_paged_bf16kv if self.b["kp"].dtype == torch.bfloat16 else self.cp.attn_evict_paged
        call(self.b["kp"], self.b["vp"], self.w, self.b["table"], self.grown["ctx"], self.keep, 30000, keep_first=4,
             keep_last=64, workspace=self.ws, stream=stream)

    def state(self):
        return [bits(x).clone() for x in (self.w, self.b["kp"], self.b["vp"], self.out)]


def one_by_one(step):
    """The steps with the host waiting after every call: what the others have to give, bit by bit."""
    outs = []
    for _ in range(STEPS):
        weigh(step.cp, step.b, step.q, step.w, 0.9, bound=30000, rows=70)
        torch.cuda.synchronize()
        step.out.copy_(decode(step.cp, step.grown, step.qd, step.w, 0.95, bound=30000))
        torch.cuda.synchronize()
        outs.append(step.out.clone())
        evict(step.cp, step.grown, step.w, step.keep, 4, 64, bound=30000)
        torch.cuda.synchronize()
    return step.state(), outs


LENS = [[(1500, 70)], [(700, 70), (6000, 33)], [(20000, 64)]]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens", LENS)
def test_a_step_replayed(cp, bf16, lens):
    want, outs = one_by_one(Step(cp, lens, bf16, 31))
    step = Step(cp, lens, bf16, 31)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step.run()
    got = []
    for _ in range(STEPS):  # no host wait: the copy of each output follows its replay in the stream
        graph.replay()
        got.append(step.out.clone())
    torch.cuda.synchronize()
    assert cp.attn_get_device_error() == 0
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(got, outs))
    assert all(torch.equal(x, y) for x, y in zip(step.state(), want))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens", LENS)
def test_steps_one_after_another(cp, bf16, lens):
    """Eager, on a stream that is given to the calls, all on one workspace."""
    want, outs = one_by_one(Step(cp, lens, bf16, 32))
    step, stream = Step(cp, lens, bf16, 32), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(STEPS):
        step.run(stream)
    torch.cuda.synchronize()
    assert cp.attn_get_device_error() == 0
    assert torch.equal(bits(step.out), bits(outs[-1]))
    assert all(torch.equal(x, y) for x, y in zip(step.state(), want))


@pytest.mark.parametrize("bf16", [False, True])
def test_two_streams_at_once(cp, bf16):
    """Each with its own sequences and workspace; on one of them the step is a graph."""
    want = [one_by_one(Step(cp, lens, bf16, 33 + i))[0] for i, lens in enumerate(LENS[:2])]
    steps, streams = [Step(cp, lens, bf16, 33 + i) for i, lens in enumerate(LENS[:2])], [torch.cuda.Stream() for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        steps[1].run()
    torch.cuda.synchronize()
    for _ in range(STEPS):
        with torch.cuda.stream(streams[0]):
            steps[0].run()
        with torch.cuda.stream(streams[1]):
            graph.replay()
    torch.cuda.synchronize()
    assert cp.attn_get_device_error() == 0
    for step, state in zip(steps, want):
        assert all(torch.equal(x, y) for x, y in zip(step.state(), state))
