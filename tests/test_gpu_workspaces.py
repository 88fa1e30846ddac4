"""The binding's workspaces on the GPU: graphs captured before a larger call took a
larger one, first calls inside a capture, streams given by the caller, and
decode calls that overlap on two streams or in two graphs."""
import numpy as np
import pytest
import torch

from mixed_precision_paged_thinkv_b200.binding import ThinKVCache, ThinkvError

import turnover_model as M
from test_gpu_shared import _ids

pytestmark = pytest.mark.gpu


def _cache(lens, max_seqs, pages=2000):
    """Sequence i with lens[i] tokens, room for max_seqs."""
    c = ThinKVCache(8, 2, 64, 32, (8, 4, 2), max_seqs, max([200, *(n // 16 + 4 for n in lens)]), (pages,) * 3)
    for s, n in enumerate(lens):
        if n:
            _append(c, [s] * n, range(n), s)
    assert c.status() == 0
    return c


def _append(c, seq, pos, seed):
    rng = np.random.default_rng(seed)
    n = len(seq)
    kv = torch.from_numpy(rng.standard_normal((2, n, c.H, c.d)).astype(np.float32)).half().cuda()
    c.append(_ids(seq), _ids(pos), torch.from_numpy(rng.integers(0, 3, n).astype(np.uint8)).cuda(), kv[0], kv[1])


def _use_freed_memory():
    """Other tensors take, and overwrite, whatever the allocator has free."""
    return [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
            for size in (256, 512, 1024, 4096, 16384, 1 << 18, 1 << 20, 1 << 22) for _ in range(16)]


def test_turnover_graph_outlives_a_larger_call():
    c = _cache([300, 40], 64)
    c.fork(_ids([0]), _ids([2]))
    c.release(_ids([2]))
    src, dst = _ids([0, 1]), _ids([2, 3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.fork(src, dst)
        c.release(dst)
        c.fork(src, dst)
    c.fork(_ids([0] * 50), _ids(range(10, 60)))        # needs more than the captured calls do
    c.release(_ids(range(10, 60)))
    taken = _use_freed_memory()
    torch.cuda.synchronize()
    want = M.host_buffers(c)
    graph.replay()
    M.fork(want, [0, 1], [2, 3], c.pool_pages)
    M.release(want, [2, 3], c.pool_pages)
    M.fork(want, [0, 1], [2, 3], c.pool_pages)
    torch.cuda.synchronize()
    assert c.status() == 0
    M.assert_same(M.host_buffers(c), want)
    assert all((t == 0x5A).all() for t in taken)


def test_append_graph_outlives_a_larger_call():
    a, b = _cache([20] * 8, 8), _cache([20] * 8, 8)
    seq, pos, tag = _ids(range(8)), _ids([100] * 8), torch.zeros(8, dtype=torch.uint8, device="cuda")
    kv = torch.randn(2, 8, a.H, a.d, device="cuda").half()
    _append(a, [0], [50], 1)
    _append(b, [0], [50], 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.append(seq, pos, tag, kv[0], kv[1])
    torch.cuda.synchronize()
    for c in (a, b):
        _append(c, [1] * 1500, range(60, 1560), 2)
    taken = _use_freed_memory()
    graph.replay()
    b.append(seq, pos, tag, kv[0], kv[1])
    torch.cuda.synchronize()
    assert a.status() == 0 and b.status() == 0
    x, y = a.snapshot(), b.snapshot()
    for name in ("num_blocks", "free_top", "fifo_head", "fifo_tail", "live_count", "num_live", "page_bump"):
        assert np.array_equal(x[name], y[name]), name
    for s, nb in enumerate(x["num_blocks"]):
        assert np.array_equal(x["table"][s, :nb], y["table"][s, :nb])
    q = torch.randn(8, a.Hq, a.d, device="cuda").half()
    assert torch.equal(a.decode(seq, q)[0], b.decode(seq, q)[0])
    assert all((t == 0x5A).all() for t in taken)


def test_first_turnover_in_a_capture_of_the_given_stream_is_refused():
    c = _cache([300, 40], 8)
    dst, side, graph = _ids([2, 3]), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.capture_begin()
    try:
        with pytest.raises(ThinkvError):               # the stream given captures, the current one does not
            c.release(dst, stream=side)
    finally:
        with torch.cuda.stream(side):
            graph.capture_end()
    c.release(dst, stream=side)
    side.synchronize()
    assert c.status() == 0


def test_first_append_in_a_capture():
    """The graph zeroes a workspace of its own; calls outside it have theirs."""
    a, b = _cache([], 8), _cache([], 8)
    seq, pos, tag = _ids(range(8)), _ids([100] * 8), torch.zeros(8, dtype=torch.uint8, device="cuda")
    kv = torch.randn(2, 8, a.H, a.d, device="cuda").half()
    graph = torch.cuda.CUDAGraph()
    taken = _use_freed_memory()
    del taken
    with torch.cuda.graph(graph):
        a.append(seq, pos, tag, kv[0], kv[1])
    _append(a, [3] * 20, range(20), 1)                 # before the graph ever ran
    graph.replay()
    _append(b, [3] * 20, range(20), 1)
    b.append(seq, pos, tag, kv[0], kv[1])
    q = torch.randn(8, a.Hq, a.d, device="cuda").half()
    assert torch.equal(a.decode(seq, q)[0], b.decode(seq, q)[0])
    assert a.status() == 0 and b.status() == 0
    assert a.snapshot()["live_count"].tolist() == [1, 1, 1, 21, 1, 1, 1, 1]


def test_first_append_on_a_side_stream():
    """The zero fill of a new workspace is in the order of the stream that uses it."""
    a, b = _cache([], 8), _cache([], 8)
    seq, pos, tag = _ids(range(8)), _ids([100] * 8), torch.zeros(8, dtype=torch.uint8, device="cuda")
    kv = torch.randn(2, 8, a.H, a.d, device="cuda").half()
    side = torch.cuda.Stream()
    b.append(seq, pos, tag, kv[0], kv[1])
    taken = _use_freed_memory()
    torch.cuda.synchronize()
    del taken
    torch.cuda._sleep(20_000_000)                      # the current stream is busy for some 10 ms
    a.append(seq, pos, tag, kv[0], kv[1], stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    q = torch.randn(8, a.Hq, a.d, device="cuda").half()
    assert torch.equal(a.decode(seq, q)[0], b.decode(seq, q)[0])
    assert a.status() == 0


def _decodes(c, shared, topk=None):
    """Two calls over different rows, and what each answers alone."""
    calls = []
    for part in (range(2, 34), range(34, 64)):
        seq, prefix = _ids(part), _ids([s % 2 for s in sorted(part, key=lambda s: s % 2)])
        q = torch.randn(len(part), c.Hq, c.d, device="cuda").half()

        def call(out=None, stream=None, seq=seq, prefix=prefix, q=q):
            if shared:
                return c.decode_shared(seq, prefix, q, topk=topk, out=out, stream=stream)[0]
            return c.decode(seq, q, topk=topk, out=out, stream=stream)[0]

        calls.append(call)
    want = [call().clone() for call in calls]
    torch.cuda.synchronize()
    return calls, want


@pytest.mark.parametrize("shared,topk", [(True, None), (True, 8), (False, None), (False, 8)])
def test_overlapping_decodes(shared, topk):
    c = _cache([12000, 9000] + [400] * 62, 64, pages=4000)
    calls, want = _decodes(c, shared, topk)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty_like(w) for _ in range(40)] for w in want]
    torch.cuda.synchronize()
    for i in range(40):
        for j in (0, 1):
            calls[j](out=outs[j][i], stream=streams[j])
    torch.cuda.synchronize()
    assert c.status() == 0
    for j in (0, 1):
        assert all(torch.equal(o, want[j]) for o in outs[j])


@pytest.mark.parametrize("shared", [True, False])
def test_overlapping_graphs(shared):
    """Two graphs of the same cache, replayed at the same time on two streams."""
    c = _cache([12000, 9000] + [400] * 62, 64, pages=4000)
    calls, want = _decodes(c, shared)
    graphs, outs = [], []
    for j in (0, 1):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[j]):
            outs.append([calls[j]() for _ in range(6)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for j in (0, 1):
            with torch.cuda.stream(streams[j]):
                graphs[j].replay()
    torch.cuda.synchronize()
    assert c.status() == 0
    for j in (0, 1):
        assert all(torch.equal(o, want[j]) for o in outs[j])
