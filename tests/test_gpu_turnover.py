"""Release and fork on the GPU: every buffer bit for bit against the host model
of the calls, forked sequences against the oracle replaying their history,
refused calls, reuse of released pages by append and compaction, streams and
graphs."""
import numpy as np
import pytest
import torch

from oracle import oracle as O
from mixed_precision_paged_thinkv_b200 import binding
from mixed_precision_paged_thinkv_b200.binding import ThinKVCache

import harness as Hn
import turnover_model as M

pytestmark = pytest.mark.gpu

LAYOUTS = {                      # q heads, kv heads, head dim, group, bits, fmt
    "d64": (4, 2, 64, 32, (8, 4, 2), (0, 0, 0)),
    "d128": (16, 8, 128, 64, (8, 4, 2), (0, 0, 0)),
    "raw": (6, 3, 128, 32, (16, 8, 4), (0, 0, 0)),
    "float": (8, 8, 64, 64, (8, 4, 2), (1, 1, 1)),
    "one-head": (1, 1, 64, 64, (2, 16, 2), (0, 0, 0)),
}


def _ids(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _append(cache, seq, start, count, rng, tags=None):
    """`count` random tokens of one sequence from position `start` on."""
    pos = np.arange(start, start + count, dtype=np.int32)
    tag = rng.integers(0, 3, count).astype(np.uint8) if tags is None else tags
    kv = rng.standard_normal((2, count, cache.H, cache.d)).astype(np.float16)
    k, v = torch.from_numpy(kv[0]), torch.from_numpy(kv[1])
    cache.append(torch.full((count,), seq, dtype=torch.int32, device="cuda"), torch.from_numpy(pos).cuda(),
                 torch.from_numpy(tag).cuda(), k.cuda(), v.cuda())
    return pos, tag, k, v


def _filled(layout, lens, extra_seqs, seed, tbe=False, pool=None, nb=None):
    """A cache whose first sequences hold lens[i] tokens, partly evicted; pool bytes random."""
    hq, h, d, g, bits, fmt = LAYOUTS[layout]
    rng = np.random.default_rng(seed)
    nb = nb or max(4, max(lens) // 16 + 4)
    ns = len(lens) + extra_seqs
    pool = pool or (2 * (sum(lens) // 16 + 3 * ns),) * 3
    c = ThinKVCache(hq, h, d, g, bits, ns, nb, pool, fmt=fmt, tbe=tbe)
    for s, n in enumerate(lens):
        at = 0
        while at < n:
            m = min(n - at, int(rng.integers(1, 700)))
            pos, tag, _, _ = _append(c, s, at, m, rng)
            if tbe:
                c.evict_tbe(torch.full((m,), s, dtype=torch.int32, device="cuda"), torch.from_numpy(pos).cuda(),
                            torch.from_numpy(tag).cuda(), t_min=2, schedule=[8, 4, 2])
            at += m
        if n > 40:
            c.evict(_ids(s), _ids(int(n * 0.7)))
    torch.cuda.synchronize()
    assert c.status() == 0
    return c


def _check(c, want):
    torch.cuda.synchronize()
    M.assert_same(M.host_buffers(c), want)


@pytest.mark.parametrize("tbe", [False, True])
@pytest.mark.parametrize("layout", sorted(LAYOUTS))
def test_calls_match_the_host_model(layout, tbe):
    """Ragged sequences (none, one token, one page, long), repeated sources, all of
    the released pages and fresh ones behind them."""
    lens = [333, 1, 0, 16, 17, 900, 150]
    c = _filled(layout, lens, 6, seed=5, tbe=tbe)
    want = M.host_buffers(c)
    for op, a, b in (("fork", [5, 0, 5, 2], [12, 7, 9, 8]), ("release", [0, 3, 2, 11], None),
                     ("fork", [9, 6], [3, 0]), ("release", [12, 5], None), ("fork", [0, 0, 0], [5, 12, 2]),
                     ("release", [5], None), ("release", [12, 2, 0, 1, 4, 3, 6, 7, 8, 9, 10, 11, 5], None)):
        if op == "fork":
            c.fork(_ids(*a), _ids(*b))
            M.fork(want, a, b, c.pool_pages)
        else:
            c.release(_ids(*a))
            M.release(want, a, c.pool_pages)
        _check(c, want)
    assert c.status() == 0
    # everything is empty: every page ever handed out waits on its stack, once
    snap = c.snapshot()
    for cl in range(3):
        assert sorted(snap["released"][cl].tolist()) == list(range(snap["page_bump"][cl]))


def test_tables_longer_than_one_pass():
    """More than 1,024 table entries a sequence: several passes of the counting."""
    hq, h, d, g, bits, fmt = LAYOUTS["d64"]
    rng = np.random.default_rng(3)
    nb, n = 2600, 2500 * 16
    c = ThinKVCache(hq, h, d, g, bits, 4, nb, (9000, 9000, 9000))
    for s, total in ((0, n), (1, 1024 * 16)):
        for at in range(0, total, 4096):
            m = min(4096, total - at)
            _append(c, s, at, m, rng, tags=np.repeat(rng.integers(0, 3, (m + 15) // 16), 16)[:m].astype(np.uint8))
    c.evict(_ids(0), _ids(n // 2))
    torch.cuda.synchronize()
    want = M.host_buffers(c)
    assert want["num_blocks"][0] > 2048
    c.fork(_ids(0, 1), _ids(3, 2))
    M.fork(want, [0, 1], [3, 2], c.pool_pages)
    c.release(_ids(1, 0))
    M.release(want, [1, 0], c.pool_pages)
    c.fork(_ids(2, 3), _ids(0, 1))
    M.fork(want, [2, 3], [0, 1], c.pool_pages)
    _check(c, want)


def test_many_sequences_in_a_call():
    """More sequences than threads of the scan, most of them of a page or none."""
    hq, h, d, g, bits, fmt = LAYOUTS["one-head"]
    rng = np.random.default_rng(9)
    ns = 1400
    c = ThinKVCache(hq, h, d, g, bits, ns, 4, (2000, 2000, 2000), fmt=fmt)
    seq = np.repeat(np.arange(700, dtype=np.int32), rng.integers(0, 3, 700))
    pos = np.array([i - np.flatnonzero(seq == s)[0] for i, s in enumerate(seq)], np.int32)
    kv = torch.randn(2, len(seq), 1, 64).half().cuda()
    c.append(torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda(),
             torch.from_numpy(rng.integers(0, 3, len(seq)).astype(np.uint8)).cuda(), kv[0], kv[1])
    torch.cuda.synchronize()
    want = M.host_buffers(c)
    src, dst = rng.integers(0, 700, 600).tolist(), (700 + rng.permutation(700)[:600]).tolist()
    gone = rng.permutation(ns)[:1000].tolist()
    c.fork(_ids(*src), _ids(*dst))
    M.fork(want, src, dst, c.pool_pages)
    c.release(_ids(*gone))
    M.release(want, gone, c.pool_pages)
    _check(c, want)


@pytest.mark.parametrize("per_call", [60, 700])       # one-launch appends, and the general path
def test_forks_go_on_as_if_they_had_their_history(per_call):
    """A fork appends, is annealed, evicts and decodes like a sequence that was
    given the source's whole history: state, codes and attention against the
    oracle, which replays it, while other sequences come and go."""
    hq, h, d, g, bits, fmt = LAYOUTS["d128"]
    rng = np.random.default_rng(per_call)
    args = (hq, h, d, g, bits, 6, 260, (400, 400, 400))
    c = ThinKVCache(*args, tbe=True)
    o = O.Oracle(*args)                                # oracle ids: 0 the source, 1 and 2 its forks

    def step(gpu_seqs, oracle_seqs, start, n, seed):
        r = np.random.default_rng(seed)
        tag = np.repeat(r.integers(0, 3, n // 6 + 1), 6)[:n].astype(np.uint8)
        kv = r.standard_normal((2, n, h, d)).astype(np.float16)
        k, v = torch.from_numpy(kv[0]), torch.from_numpy(kv[1])
        pos = np.arange(start, start + n, dtype=np.int32)
        for s in gpu_seqs:
            ids = torch.full((n,), s, dtype=torch.int32, device="cuda")
            p, t = torch.from_numpy(pos).cuda(), torch.from_numpy(tag).cuda()
            c.append(ids, p, t, k.cuda(), v.cuda())
            c.evict_tbe(ids, p, t, t_min=3, schedule=[20, 10, 5])
            c.evict(_ids(s), _ids((start + n) * 2 // 3))
        for s in oracle_seqs:
            ids = np.full(n, s, np.int32)
            assert o.append(ids, pos, tag, k, v) == O.OK
            assert o.tbe(ids, pos, tag, t_min=3, schedule=[20, 10, 5]) == O.OK
            assert o.evict(np.array([s], np.int32), np.array([(start + n) * 2 // 3], np.int32)) == O.OK

    _append(c, 4, 0, 500, rng)                         # a passer-by, released before the fork
    step([0], [0, 1, 2], 0, per_call, 1)
    c.release(_ids(4))
    step([0], [0, 1, 2], per_call, per_call, 2)
    c.fork(_ids(0, 0), _ids(3, 1))
    step([3], [1], 2 * per_call, per_call, 3)          # the forks go different ways
    _append(c, 5, 0, 90, rng)
    step([1], [2], 2 * per_call, per_call, 4)
    c.release(_ids(5))
    step([0], [0], 2 * per_call, per_call, 5)
    torch.cuda.synchronize()
    assert c.status() == 0
    gs, os_ = c.snapshot(), o.state()
    q = rng.standard_normal((3, hq, d)).astype(np.float16)
    out, _ = c.decode(_ids(0, 3, 1), torch.from_numpy(q).cuda())
    ref, _ = o.decode(np.arange(3, dtype=np.int32), torch.from_numpy(q))
    for j, s in enumerate((0, 3, 1)):
        Hn.compare_seq_structure(gs, s, os_, j)
        assert gs["nseg"][s] == os_["nseg"][j]
    Hn.check_slot_invariants(gs, 6)
    assert Hn.attn_error(out.cpu().numpy(), ref) <= Hn.TOL
    held = [set(), set(), set()]                       # no page belongs to two sequences, or to one and a stack
    for s in range(6):
        for e in gs["table"][s, :gs["num_blocks"][s]]:
            cl, page = int(O.entry_class(e)), int(O.entry_page(e))
            assert page not in held[cl]
            held[cl].add(page)
    for cl in range(3):
        free = gs["released"][cl].tolist()
        assert len(set(free)) == len(free) and not held[cl] & set(free)
        assert len(held[cl]) + len(free) == gs["page_bump"][cl]


def test_compaction_takes_released_pages():
    c = _filled("d64", [600, 300], 1, seed=11, nb=60)
    dst = _filled("d64", [100, 700, 50], 0, seed=12, nb=c.max_blocks, pool=c.pool_pages)
    dst.release(_ids(1, 0))
    c.compact_into(dst, _ids(1, 0), max_tokens=2000)
    torch.cuda.synchronize()
    assert dst.status() == 0 and c.status() == 0
    snap = dst.snapshot()
    Hn.check_slot_invariants(snap, 3)
    for s in (0, 1):
        assert sorted(Hn.gpu_live_by_pos(snap, s)) == sorted(Hn.gpu_live_by_pos(c.snapshot(), s))
    q = torch.randn(2, c.Hq, c.d, device="cuda").half()
    a, b = c.decode(_ids(0, 1), q)[0], dst.decode(_ids(0, 1), q)[0]
    # the same tokens in another order of pages: both within the decode's bound of the exact rows
    assert Hn.attn_error(a.cpu().numpy(), b.double().cpu().numpy()) <= 2 * Hn.TOL


def test_refused_calls_change_nothing():
    c = _filled("d64", [200, 40, 0, 90], 3, seed=21, pool=(20, 20, 20), nb=40)
    want = M.host_buffers(c)
    bad = [("release", [0, 0]), ("release", [1, 7]), ("release", [-1]), ("release", [0, 1 << 20]),
           ("fork", [0, 1], [4, 4]), ("fork", [0], [1]), ("fork", [0], [7]), ("fork", [-1], [4]),
           ("fork", [7], [4]), ("fork", [0, 4], [4, 5]), ("fork", [4], [4])]
    for op, *ids in bad:
        getattr(c, op)(*[_ids(*x) for x in ids])
        torch.cuda.synchronize()
        assert c.status() == binding.ERR_INVALID, (op, ids)
        c.release(_ids(0))                             # while the status is set, nothing happens
        c.fork(_ids(0), _ids(4))
        c.clear_status()
        _check(c, want)
    c.fork(_ids(0), _ids(4))
    M.fork(want, [0], [4], c.pool_pages)
    _check(c, want)
    _append(c, 4, 300, 200, np.random.default_rng(1))
    torch.cuda.synchronize()
    assert c.status() == 0
    want = M.host_buffers(c)
    c.fork(_ids(0, 0, 4), _ids(2, 5, 6))               # more pages than the pools have left
    torch.cuda.synchronize()
    assert c.status() == binding.ERR_OUT_OF_PAGES
    c.clear_status()
    _check(c, want)
    c.release(_ids(4, 0))
    M.release(want, [4, 0], c.pool_pages)
    _check(c, want)


def test_arguments_of_the_binding():
    c = _filled("d64", [40], 1, seed=2)
    c.release(_ids())
    c.fork(_ids(), _ids())
    for bad in (lambda: c.release(torch.zeros(1, dtype=torch.int64, device="cuda")),
                lambda: c.release(torch.zeros(1, dtype=torch.int32)),
                lambda: c.fork(_ids(0), _ids(1, 1)),
                lambda: c.fork(_ids(0, 0, 0)[::2], _ids(1, 1, 1)[::2])):
        with pytest.raises(AssertionError):
            bad()
    with pytest.raises(binding.ThinkvError):
        c.release(_ids(0, 1, 0))                       # more ids than the cache has sequences
    buffers = dict(c.buf)
    again = ThinKVCache(4, 2, 64, 32, (8, 4, 2), c.max_seqs, c.max_blocks, c.pool_pages, buffers=buffers)
    M.assert_same(M.host_buffers(again), M.host_buffers(c))
    for bad in (dict(buffers, fifo=None), dict(buffers, fifo=buffers["fifo"][:-1]),
                dict(buffers, fifo=buffers["fifo"].cpu())):
        with pytest.raises(binding.ThinkvError):
            ThinKVCache(4, 2, 64, 32, (8, 4, 2), c.max_seqs, c.max_blocks, c.pool_pages, buffers=bad)


def test_pool_lives_on_released_pages():
    """Rounds of finished and new sequences in pools that hold one round only."""
    hq, h, d, g, bits, fmt = LAYOUTS["d64"]
    rng = np.random.default_rng(4)
    c = ThinKVCache(hq, h, d, g, bits, 8, 40, (48, 48, 48))
    for turn in range(6):
        n = int(rng.integers(60, 120))
        seq = np.repeat(np.arange(8, dtype=np.int32), n)
        kv = torch.randn(2, len(seq), h, d).half().cuda()
        c.append(torch.from_numpy(seq).cuda(), torch.from_numpy(np.tile(np.arange(n, dtype=np.int32), 8)).cuda(),
                 torch.from_numpy(rng.integers(0, 3, len(seq)).astype(np.uint8)).cuda(), kv[0], kv[1])
        torch.cuda.synchronize()
        assert c.status() == 0, turn
        Hn.check_slot_invariants(c.snapshot(), 8)
        c.release(_ids(*rng.permutation(8).tolist()))
    assert (c.snapshot()["page_bump"] <= 48).all()


def test_side_stream_and_graph():
    """A turnover on a side stream, then captured and replayed: each replay ends the
    copies and starts them again from the source as it then is."""
    c = _filled("d128", [500, 64], 3, seed=31)
    want = M.host_buffers(c)
    src, dst = _ids(0, 1, 0), _ids(4, 2, 3)
    with pytest.raises(binding.ThinkvError):           # no workspace yet: refused while capturing
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            c.release(dst)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.release(dst, stream=side)
    c.fork(src, dst, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    M.release(want, dst.tolist(), c.pool_pages)
    M.fork(want, src.tolist(), dst.tolist(), c.pool_pages)
    _check(c, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.release(dst)
        c.fork(src, dst)
    _check(c, want)
    for _ in range(2):
        _append(c, 0, 1000, 40, np.random.default_rng(1))
        torch.cuda.synchronize()
        want = M.host_buffers(c)
        graph.replay()
        M.release(want, dst.tolist(), c.pool_pages)
        M.fork(want, src.tolist(), dst.tolist(), c.pool_pages)
        _check(c, want)
        c.evict(_ids(0), _ids(300))
    assert c.status() == 0
