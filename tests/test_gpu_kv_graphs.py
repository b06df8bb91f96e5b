"""Every decode-serving call captured into a graph and replayed on other inputs, and on a side stream: the results are those
of the same calls made one by one."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests.test_gpu_kv_pages import State, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def captured(call):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g


def test_fork_compaction_and_page_copies_in_graphs(dev):  # noqa: F811
    s = State(dev, 8, 5, 40, 8, e4m3=True, d=128)
    s.resize([0, 1, 2], [13, 30, 8])
    parents, children = s.ints([0, 0]), s.ints([3, 4])
    src, dst = s.ints([0, 1]), s.ints([38, 39])
    fork = captured(lambda: q.qgemm_kv_fork(s.kv, s.table, s.lens, s.refs, parents, children))
    compact = captured(lambda: q.qgemm_kv_compact(s.kv, s.table, s.lens, s.refs))
    copy = captured(lambda: q.qgemm_kv_copy_pages(s.kv, src, dst))
    for a, b, c in ((0, 0, [3, 4]), (1, 2, [5, 6]), (3, 1, [4, 5])):
        s.before()
        assert not s.host.fork([a, b], c)
        parents.copy_(s.ints([a, b]))
        children.copy_(s.ints(c))
        fork.replay()
        assert q.qgemm_poll_device_error() == 0
        s.same("fork")
        s.resize([c[0]], [s.host.lens[c[0]] // 2])
        s.resize([0 if a else 7], [0 if a else 19])
        s.before()
        s.host.compact()
        compact.replay()
        assert q.qgemm_poll_device_error() == 0
        s.same("compact")
        s.before()
        s.host.moves = [(a, 38, 8), (c[0], 39, 8)]
        src.copy_(s.ints([a, c[0]]))
        copy.replay()
        assert q.qgemm_poll_device_error() == 0
        s.same("copy")


class Decode:
    """A token for each of B sequences a step: rope of other rows, append, attention."""

    def __init__(self, dev, e4m3, dtype, B=5, hq=8, hkv=2, d=128, page=16, steps=40):
        g = torch.Generator(device=dev).manual_seed(7)
        per = -(-(steps + 20) // page)
        shape = (1, B * per, hkv, page)
        if e4m3:
            planes = [torch.zeros(*shape, n, dtype=torch.uint8, device=dev) for n in (d, d, 4, 4)]
        else:
            planes = [torch.zeros(*shape, d, dtype=dtype, device=dev) for _ in "kv"]
        self.planes, self.kv = planes, q.qgemm_create_kv_cache(*planes)
        self.table = torch.randperm(B * per, generator=g, device=dev).to(torch.int32).view(B, per)
        self.seqs = torch.arange(B, dtype=torch.int32, device=dev)
        self.pos = torch.tensor([0, 3, 15, 16, 17][:B], dtype=torch.int32, device=dev)
        self.lens = self.pos + 1
        self.rope = q.qgemm_create_rope(d, scaling="linear", factor=2.0)
        self.x = torch.randn(B, hq + 2 * hkv, d, generator=g, device=dev).to(dtype)
        self.q, self.k, self.v = self.x.split([hq, hkv, hkv], 1)
        self.qo, self.o, self.y = (torch.zeros(B, hq, d, dtype=dtype, device=dev) for _ in "qoy")
        self.workspace = q.qgemm_paged_attention_workspace(self.kv, B, hq)

    def step(self, stream=None):
        q.qgemm_rope(self.q, self.pos, self.rope, out=self.y, inverse=True, stream=stream)
        q.qgemm_kv_append(self.kv, 0, self.k, self.v, self.seqs, self.pos, self.table, rope=self.rope, Q=self.q, Q_out=self.qo,
                          stream=stream)
        q.qgemm_paged_attention(self.qo, self.kv, 0, self.table, self.lens, self.o, seqs=self.seqs, workspace=self.workspace,
                                stream=stream)

    def advance(self, i):
        self.x.mul_(-1.0).add_(0.03125 * (i % 5))
        self.pos.add_(1)
        self.lens.add_(1)

    def outputs(self):
        return [t.clone() for t in (self.y, self.qo, self.o, *self.planes)]


@pytest.mark.parametrize("e4m3,dtype", [(False, torch.float16), (True, torch.bfloat16)])
def test_a_decode_step_in_a_graph_and_on_a_side_stream(dev, e4m3, dtype):  # noqa: F811
    serial, graph, side = (Decode(dev, e4m3, dtype) for _ in range(3))
    g = captured(graph.step)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for i in range(40):
        serial.step()
        g.replay()
        side.step(stream)
        with torch.cuda.stream(stream):
            side.advance(i)
        serial.advance(i)
        graph.advance(i)
    torch.cuda.synchronize()
    assert q.qgemm_poll_device_error() == 0
    for a, b, c in zip(serial.outputs(), graph.outputs(), side.outputs()):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert bool(serial.o.isfinite().all()) and float(serial.o.float().abs().max()) > 0
