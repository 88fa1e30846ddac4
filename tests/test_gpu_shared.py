"""Shared-prefix decode on the GPU against softmax attention in 64 bits over the
cache's dequantised pages, on both of its paths (the prefix kernel for runs
that are worth it, the split kernel otherwise), with holes, ragged and empty
sequences, one token to long prefixes, every code format and head layout, bad
ids, the top-k mass, streams and graphs."""
import numpy as np
import pytest
import torch

from mixed_precision_paged_thinkv_b200 import binding
from mixed_precision_paged_thinkv_b200.binding import ThinKVCache

import harness as Hn
from layout_decode import decode_blocks

pytestmark = pytest.mark.gpu

# q heads, kv heads, head dim, group
HEADS = {"tiny": (4, 2, 64, 32), "gqa4": (32, 8, 128, 64), "gqa5": (40, 8, 128, 64), "gqa8": (64, 8, 64, 32),
         "mha": (8, 8, 128, 32), "gqa3": (9, 3, 64, 64), "gqa7": (14, 2, 128, 64), "gqa6": (6, 1, 128, 32)}
BITS = {"842": ((8, 4, 2), (0, 0, 0)), "float": ((8, 4, 2), (1, 1, 1)), "raw": ((16, 8, 4), (0, 0, 0)),
        "fp4": ((4, 2, 8), (1, 0, 1)), "two": ((2, 2, 2), (0, 1, 0))}

# Bound of an output element, from the roundings that the kernels make.  Keys,
# values and weights enter the products as fp16, each off by at most e = 2^-11
# of itself and, being roundings of unrelated numbers, by e / sqrt(3) at most in
# the mean square and independently of one another.  A key's error moves its
# token's logit by a mean square of sx^2 = scale^2 e^2 / 3 sum_c (q_c k_c)^2; a
# logit's shift dx moves the output by w dx (v - o), a weight's or a value's error
# by w v times it.  So the element's error has the mean square
#   s^2 = sum_t w_t^2 [ (v_t - o)^2 sx_t^2 + (v_t^2 + a_t^2) e^2 / 3 ],
# where a_t is what the weight's rounding multiplies: the value, or, as the split
# kernel rounds weight times scale and multiplies the centred code by it, up to
# scale * 2^(b-1) where that is larger than the value (integer codes).  The error is taken to stay below 8 s (one in 10^15 for a normal sum; a call has up to
# 10^6 elements), plus the output's own rounding e |o| and 2^-20 of sum w |v| for the
# fp32 sums (one weight of several thousand products: 2^-24 sqrt(10^4) < 2^-17 of a
# random sum's size, which is itself below 1/8 of that) and 2^-24 for fp16's smallest
# outputs.
E = 2.0 ** -11


def _ids(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _e4m3(c):
    return torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()


_FP4 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])


class Exact:
    """K and V of a cache's live tokens in 64 bits, and attention over them."""

    def __init__(self, cache):
        self.c, self.snap, self.kept = cache, cache.snapshot(), {}
        self.pools = [cache.pool_bytes(c) for c in range(3)]

    def tokens(self, s):
        if s < 0:
            return [np.zeros((0, self.c.H, self.c.d))] * 3
        if s not in self.kept:
            c, got = self.c, [[], [], []]               # K, V, what a weight's rounding multiplies
            t = self.snap["table"][s, :self.snap["num_blocks"][s]]
            for cl in range(3):
                mine = t[((t >> np.uint64(32)) & np.uint64(0xFF)) == cl]
                if not len(mine):
                    continue
                blocks = self.pools[cl][(mine & np.uint64(0xFFFFFFFF)).astype(np.int64)]
                live = ((mine >> np.uint64(48))[:, None] >> np.arange(16, dtype=np.uint64)) & np.uint64(1) == 1
                codes = decode_blocks(blocks, c.d, c.G, c.bits[cl])
                for kv in range(2):
                    x, par = codes[kv], codes[2 + kv]            # [p, H, 16, d], [p, H, 16, ng, 2]
                    if par is None:
                        v = x.view(np.float16).astype(np.float64)
                    else:
                        s_z = np.repeat(np.ascontiguousarray(par).view(np.float16).astype(np.float64), c.G, axis=3)
                        if c.fmt[cl] and c.bits[cl] == 8:
                            x = _e4m3(x)
                        elif c.fmt[cl] and c.bits[cl] == 4:
                            x = _FP4[x]
                        with np.errstate(invalid="ignore", over="ignore"):     # dead slots hold noise
                            v = x * s_z[..., 0] + s_z[..., 1]
                    got[kv].append(v.transpose(0, 2, 1, 3)[live])
                    if kv == 1:
                        amp = np.abs(v)
                        if par is not None and not (c.fmt[cl] and c.bits[cl] > 2):
                            with np.errstate(invalid="ignore", over="ignore"):
                                amp = np.maximum(amp, s_z[..., 0] * 2.0 ** (c.bits[cl] - 1))
                        got[2].append(amp.transpose(0, 2, 1, 3)[live])
            self.kept[s] = [np.concatenate(x) if x else np.zeros((0, c.H, c.d)) for x in got]
        return self.kept[s]

    def rows(self, seq, prefix, q, scale=None, topk=None):
        c = self.c
        dev = {s: [torch.from_numpy(x).cuda() for x in self.tokens(s)] for s in {*seq, *prefix}}
        out = torch.zeros(len(seq), c.Hq, c.d, dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(out)
        mass = torch.zeros(len(seq), c.Hq, dtype=torch.float64, device="cuda")
        scale = scale or 1 / np.sqrt(c.d)
        qd = torch.from_numpy(q).cuda().double().view(len(seq), c.H, c.Hq // c.H, c.d)
        for i, (s, p) in enumerate(zip(seq, prefix)):
            k, v, amp = (torch.cat(x) for x in zip(dev[p], dev[s]))
            if not len(k):
                continue
            w = torch.softmax(torch.einsum("thd,hgd->hgt", k, qd[i]) * scale, -1)
            o = torch.einsum("hgt,thd->hgd", w, v)
            out[i] = o.reshape(c.Hq, c.d)
            sx = scale ** 2 * E ** 2 / 3 * torch.einsum("thd,hgd->hgt", k * k, qd[i] ** 2)
            a, b = w * w * sx, w * w * (E ** 2 / 3)
            var = (torch.einsum("hgt,thd->hgd", a + b, v * v) + torch.einsum("hgt,thd->hgd", b, amp * amp) - 2 * o * torch.einsum("hgt,thd->hgd", a, v) +
                   o * o * a.sum(-1, keepdim=True))
            bound[i] = (8 * var.clamp(min=0).sqrt() + E * o.abs() + 2.0 ** -24 +
                        2.0 ** -20 * torch.einsum("hgt,thd->hgd", w, v.abs())).reshape(c.Hq, c.d)
            if topk:
                mass[i] = w.topk(min(topk, len(k)), -1).values.sum(-1).reshape(-1)
        return out.cpu().numpy(), mass.cpu().numpy(), bound.cpu().numpy()


def _fill(heads, bits, lens, seed, holes=0.0, dirt=True, spread=1.0):
    """A cache with lens[i] tokens in sequence i, of which a share is evicted out
    of order; the pools' bytes start as noise (NaN patterns among it)."""
    hq, h, d, g = HEADS[heads]
    b, fmt = BITS[bits]
    rng = np.random.default_rng(seed)
    nb = max(4, max(lens) // 16 + 4)
    pool = (sum(lens) // 16 + 3 * len(lens) + 3,) * 3
    c = ThinKVCache(hq, h, d, g, b, len(lens), nb, pool, fmt=fmt)
    if dirt:
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for n in "RET":
            c.buf["pool_" + n].random_(0, 256, generator=gen)
            c.buf["pool_" + n][::7] = 0xFF
    for s, n in enumerate(lens):
        for at in range(0, n, 4096):
            m = min(4096, n - at)
            kv = torch.from_numpy(rng.standard_normal((2, m, h, d)).astype(np.float32)) * spread
            kv[..., :: 37] *= 6
            kv = kv.half().cuda()
            tag = np.repeat(rng.integers(0, 3, m // 5 + 1), 5)[:m].astype(np.uint8)
            c.append(torch.full((m,), s, dtype=torch.int32, device="cuda"),
                     torch.arange(at, at + m, dtype=torch.int32, device="cuda"), torch.from_numpy(tag).cuda(),
                     kv[0], kv[1])
        if holes and n:
            head, tail = c.snapshot()["fifo_head"][s], c.snapshot()["fifo_tail"][s]
            for cl in range(3):
                gone = np.flatnonzero(rng.random(tail[cl] - head[cl]) < holes) + head[cl]
                if len(gone):
                    c.evict_slots(_ids([s] * len(gone)), torch.full((len(gone),), cl, dtype=torch.uint8, device="cuda"),
                                  _ids(gone.tolist()))
    torch.cuda.synchronize()
    assert c.status() == 0
    return c


def _within(out, ref, bound):
    """Every element within its bound; prints the worst share of it."""
    err = np.abs(out.double().cpu().numpy() - ref)
    print(f"worst element at {(err / np.maximum(bound, 1e-30)).max():.2f} of its bound, "
          f"row-normalised {Hn.attn_error(out.cpu().numpy(), ref):.2e}")
    worst = np.argwhere(err > bound)
    assert len(worst) == 0, f"{len(worst)} elements, first at (row, head, channel) {worst[0]}"


def _compare(c, seq, prefix, seed=0, topk=None, scale=None):
    rng = np.random.default_rng(seed + 100)
    q = rng.standard_normal((len(seq), c.Hq, c.d)).astype(np.float16)
    out, mass = c.decode_shared(_ids(seq), _ids(prefix), torch.from_numpy(q).cuda(), topk=topk,
                                softmax_scale=scale or 0.0)
    torch.cuda.synchronize()
    assert c.status() == 0
    ref, rmass, bound = Exact(c).rows(seq, prefix, q, scale, topk)
    _within(out, ref, bound)
    if topk:
        assert np.abs(mass.cpu().numpy() - rmass).max() <= Hn.MASS_TOL
    return out


@pytest.mark.parametrize("heads", sorted(HEADS))
@pytest.mark.parametrize("bits", sorted(BITS))
def test_small_calls(heads, bits):
    """Prefixes and sequences of a few tokens and pages, none, and no prefix: the
    split kernel reads every page."""
    lens = [40, 1, 0, 17, 3, 0, 250, 16]
    c = _fill(heads, bits, lens, seed=1, holes=0.2)
    _compare(c, [3, 4, 5, 6, 7, 3], [0, 0, 0, 1, 2, -1])
    _compare(c, [5], [0])                              # all tokens in the prefix
    _compare(c, [5, 2], [2, -1])                       # no tokens at all: zeros
    _compare(c, [6, 6, 6], [6, 0, 6])                  # a sequence with itself, and twice in a call


@pytest.mark.parametrize("heads", sorted(HEADS))
@pytest.mark.parametrize("bits", sorted(BITS))
def test_prefix_kernel_formats(heads, bits):
    """A run large enough for the prefix kernel, in every layout and format, with
    holes and a last page tile that is not full."""
    members = 24 if heads != "tiny" else 70
    lens = [5003] + [int(x) for x in np.random.default_rng(7).integers(0, 70, members)]
    c = _fill(heads, bits, lens, seed=2, holes=0.15)
    assert (members - 1) * c.snapshot()["num_live"][0] * c.H >= 5000
    _compare(c, range(1, members + 1), [0] * members)


@pytest.mark.parametrize("members,prefix,own", [
    (2, 20000, 5), (3, 9000, 0), (16, 1500, 300), (31, 4000, 1), (32, 4001, 40), (33, 4100, 17), (63, 3000, 64),
    (64, 2048, 5), (65, 2047, 5), (66, 2049, 5), (129, 1024, 20), (200, 700, 3), (300, 1, 9), (257, 130, 0)])
def test_run_sizes(members, prefix, own):
    """Row blocks of one group, of two, several blocks; key tiles from one up."""
    lens = [prefix] + [(i * 7) % (own + 1) for i in range(members)]
    c = _fill("gqa4", "842", lens, seed=members)
    _compare(c, range(1, members + 1), [0] * members, seed=members)


def test_many_runs_and_rows_without_prefix():
    """Runs of every size next to each other, a run that comes back, rows without a
    prefix between them, and an empty prefix."""
    lens = [4000, 2500, 900, 0, 1] + [(i * 13) % 90 for i in range(120)]
    c = _fill("gqa4", "float", lens, seed=5, holes=0.3)
    prefix = [0] * 30 + [1] * 20 + [-1] * 5 + [2] * 9 + [0] * 25 + [3] * 7 + [1] + [4] * 20 + [-1, 0, -1]
    _compare(c, range(5, 5 + len(prefix)), prefix)


def test_long_prefix_many_splits():
    """A prefix that every SM takes a part of, wide logits (the reference exponent
    moves), and a caller's scale."""
    c = _fill("gqa8", "842", [30000] + [50] * 40, seed=6, spread=2.5)
    _compare(c, range(1, 41), [0] * 40, scale=0.25)
    _compare(c, range(1, 41), [0] * 40)


def test_rising_logits_move_the_reference():
    """Keys that grow along the prefix: the running maximum rises all the time."""
    hq, h, d, g = HEADS["mha"]
    c = ThinKVCache(hq, h, d, g, (16, 16, 16), 101, 400, (500, 500, 500))
    n = 6000
    k = torch.ones(n, h, d) * torch.linspace(0, 8, n)[:, None, None]
    v = torch.randn(n, h, d, generator=torch.Generator().manual_seed(3))
    c.append(torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda"),
             torch.zeros(n, dtype=torch.uint8, device="cuda"), k.half().cuda(), v.half().cuda())
    q = torch.full((100, hq, d), 1.0, dtype=torch.float16)
    q[::2] = -1.0
    q[::3] = 0.0
    seq, prefix = list(range(1, 101)), [0] * 100
    out, _ = c.decode_shared(_ids(seq), _ids(prefix), q.cuda())
    torch.cuda.synchronize()
    ref, _, bound = Exact(c).rows(seq, prefix, q.numpy())
    _within(out, ref, bound)


def test_extreme_values_stay_finite():
    """Values at fp16's largest and smallest, zero keys, and zero queries."""
    hq, h, d, g = HEADS["gqa4"]
    for bits, fmt in (((8, 4, 2), (0, 0, 0)), ((8, 4, 2), (1, 1, 1))):
        c = ThinKVCache(hq, h, d, g, bits, 41, 300, (300, 300, 300), fmt=fmt)
        n = 3500
        gen = torch.Generator().manual_seed(1)
        v = (torch.rand(n, h, d, generator=gen) * 2 - 1) * 65504
        v[:, :, ::5] = 65504.0
        v[:, :, 1::5] = -65504.0
        v[:, :, 2::5] = 6e-8
        k = torch.zeros(n, h, d)
        k[:, :, 0] = 1e-7
        tag = torch.arange(n) % 3
        c.append(torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda"),
                 tag.to(torch.uint8).cuda(), k.half().cuda(), v.half().cuda())
        q = torch.zeros(40, hq, d, dtype=torch.float16)
        out, _ = c.decode_shared(_ids(range(1, 41)), _ids([0] * 40), q.cuda())
        got = out.cpu().numpy()
        ref, _, bound = Exact(c).rows(list(range(1, 41)), [0] * 40, q.numpy())
        assert np.isfinite(got.astype(np.float64)).all()
        # a group whose top code lies past fp16's range: its scale is lowered to fit, by up to one step
        # (it was rounded up by one) and rounded down (another), 2 * 2^-10 of the range of 2 * 65504
        over = np.abs(got - np.clip(ref, -65504, 65504)).max(axis=(0, 1)) - bound.max(axis=(0, 1)) - 2 * 2.0 ** -10 * 131008
        assert over.max() <= 0, f"channel {over.argmax()}: {over.max()}"


@pytest.mark.parametrize("topk", [1, 5, 32, 33, 64])
def test_topk_mass(topk):
    c = _fill("gqa4", "842", [3000, 700, 0] + [(i * 11) % 60 for i in range(20)], seed=8, holes=0.1)
    prefix = [0] * 12 + [1] * 4 + [2, -1, 2, 0]
    _compare(c, range(3, 23), prefix, topk=topk)


def test_same_as_one_sequence():
    """A sequence alone, a sequence with its history as a prefix, and decode()."""
    c = _fill("gqa4", "842", [3000, 0, 500], seed=9)
    q = torch.randn(2, c.Hq, c.d, device="cuda").half()
    a = c.decode(_ids([0, 2]), q)[0]
    b = c.decode_shared(_ids([0, 2]), _ids([-1, -1]), q)[0]
    e = c.decode_shared(_ids([1, 1]), _ids([0, 2]), q)[0]
    ref, _, bound = Exact(c).rows([0, 2], [-1, -1], q.cpu().numpy())
    for out in (a, b, e):                              # the calls split the work differently
        _within(out, ref, bound)
    assert torch.equal(b, e)


def test_bad_ids_decode_as_empty():
    c = _fill("gqa4", "842", [4000] + [30] * 60, seed=10)
    n = 60
    seq, prefix = list(range(1, n + 1)), [0] * n
    q = np.random.default_rng(0).standard_normal((n, c.Hq, c.d)).astype(np.float16)
    good = c.decode_shared(_ids(seq), _ids(prefix), torch.from_numpy(q).cuda())[0].cpu()
    bound = Exact(c).rows(seq, prefix, q)[2]
    for at, s, p in ((3, 61, 0), (10, -1, 0), (20, 5, 61), (30, 5, -2), (40, 1 << 30, -1), (59, 7, 1 << 30)):
        bs, bp = list(seq), list(prefix)
        bs[at], bp[at] = s, p
        out = c.decode_shared(_ids(bs), _ids(bp), torch.from_numpy(q).cuda())[0].cpu()
        torch.cuda.synchronize()
        assert c.status() == binding.ERR_INVALID
        c.clear_status()
        assert not out[at].any()
        keep = [i for i in range(n) if i != at]
        _within(out[keep], good[keep].double().numpy(), 2 * bound[keep])


def test_arguments_of_the_binding():
    c = _fill("tiny", "842", [40, 40], seed=2)
    q = torch.zeros(2, c.Hq, c.d, dtype=torch.float16, device="cuda")
    good = (_ids([0, 1]), _ids([-1, 0]), q)
    c.decode_shared(*good)
    for i, bad in ((0, _ids([0])), (1, _ids([0])), (1, _ids([0, 1]).long()), (1, _ids([0, 1]).cpu()), (2, q.float()),
                   (2, q[:1]), (2, q.transpose(0, 1)), (0, _ids([0, 1, 0, 1])[::2])):
        args = list(good)
        args[i] = bad
        with pytest.raises(AssertionError):
            c.decode_shared(*args)
    with pytest.raises(binding.ThinkvError):
        c.decode_shared(*good, topk=65)
    with pytest.raises(binding.ThinkvError):
        c.decode_shared(_ids([]), _ids([]), q[:0])


def test_life_of_samples():
    """Samples of two prompts as a serving loop runs them: prompts appended once,
    samples append and decode against their prompt, finished ones are released,
    one forks its prompt and is evicted on its own."""
    hq, h, d, g = HEADS["gqa4"]
    c = ThinKVCache(hq, h, d, g, (8, 4, 2), 40, 400, (700, 700, 700))
    rng = np.random.default_rng(12)

    def append(seqs, pos, tags):
        n = len(seqs)
        kv = torch.from_numpy(rng.standard_normal((2, n, h, d)).astype(np.float32)).half().cuda()
        c.append(_ids(seqs), _ids(pos), torch.tensor(tags, dtype=torch.uint8, device="cuda"), kv[0], kv[1])

    for s, n in ((0, 4500), (1, 2300)):
        append([s] * n, list(range(n)), np.repeat(rng.integers(0, 3, n // 4 + 1), 4)[:n].tolist())
    seq, prefix = list(range(2, 30)), [0] * 18 + [1] * 10
    start = {0: 4500, 1: 2300}
    for step in range(12):
        append(seq, [start[p] + step if p >= 0 else 9000 + step for p in prefix], rng.integers(0, 3, len(seq)).tolist())
        if step % 4 == 1:                              # two samples end; their ids start again
            gone = [seq[3], seq[-1]]
            c.release(_ids(gone))
            if step == 5:                              # one goes on alone, from a copy of its prompt
                c.fork(_ids([0]), _ids([gone[0]]))
                prefix[3] = -1
                c.evict(_ids([gone[0]]), _ids([3000]))
        _compare(c, seq, prefix, seed=step)
    Hn.check_slot_invariants(c.snapshot(), 40)
    c.release(_ids(range(40)))
    torch.cuda.synchronize()
    snap = c.snapshot()
    assert all(len(snap["released"][x]) == snap["page_bump"][x] for x in range(3))


def test_stream_and_graph():
    """On a side stream; captured once and replayed over a cache that has grown."""
    c = _fill("gqa4", "842", [5000] + [20] * 40, seed=14)
    seq, prefix = _ids(range(1, 41)), _ids([0] * 40)
    q = torch.randn(40, c.Hq, c.d, device="cuda").half()
    want = c.decode_shared(seq, prefix, q)[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = c.decode_shared(seq, prefix, q, stream=side)[0]
    side.synchronize()
    assert torch.equal(out, want)                      # fixed shares and order of sums: the same bits
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = c.decode_shared(seq, prefix, q)
    kv = torch.randn(2, 40, c.H, c.d, device="cuda").half()
    for step in range(3):
        c.append(seq, torch.full((40,), 6000 + step, dtype=torch.int32, device="cuda"),
                 torch.full((40,), step, dtype=torch.uint8, device="cuda"), kv[0], kv[1])
        graph.replay()
        again = c.decode_shared(seq, prefix, q)[0]
        torch.cuda.synchronize()
        assert torch.equal(out, again)
    ref, _, bound = Exact(c).rows(seq.tolist(), prefix.tolist(), q.cpu().numpy())
    _within(out, ref, bound)


def test_back_to_back_calls():
    """Calls queued without a wait in between, of different sizes over one workspace."""
    c = _fill("gqa4", "842", [6000, 300] + [25] * 50, seed=15)
    calls = [(list(range(2, 2 + n)), [p] * n) for n, p in ((50, 0), (2, 1), (33, 0), (1, 0), (50, 1), (50, 0))] * 3
    qs = [torch.randn(len(s), c.Hq, c.d, device="cuda").half() for s, _ in calls]
    outs = [c.decode_shared(_ids(s), _ids(p), q)[0] for (s, p), q in zip(calls, qs)]
    torch.cuda.synchronize()
    exact = Exact(c)
    for (s, p), q, out in zip(calls, qs, outs):
        ref, _, bound = exact.rows(s, p, q.cpu().numpy())
        _within(out, ref, bound)


@pytest.mark.parametrize("n,heads", [(1500, "tiny"), (3000, "gqa8"), (16384, "tiny")])
def test_large_calls(n, heads):
    """More rows than the plan has threads, up to the largest call: runs of every length,
    rows that share a sequence, rows without a prefix; a sample of the rows is compared."""
    rng = np.random.default_rng(n)
    lens = [700, 260, 90, 1] + [int(x) for x in rng.integers(0, 50, 60)]
    c = _fill(heads, "842", lens, seed=16, holes=0.1)
    prefix = np.repeat(rng.integers(-1, 4, n), rng.integers(1, 300, n))[:n]
    seq = rng.integers(4, 64, n)
    q = rng.standard_normal((n, c.Hq, c.d)).astype(np.float16)
    out, _ = c.decode_shared(_ids(seq.tolist()), _ids(prefix.tolist()), torch.from_numpy(q).cuda())
    torch.cuda.synchronize()
    assert c.status() == 0
    pick = np.unique(np.concatenate([rng.integers(0, n, 400), [0, 1023, 1024, n - 1]]))
    ref, _, bound = Exact(c).rows(seq[pick].tolist(), prefix[pick].tolist(), q[pick])
    _within(out[torch.from_numpy(pick).cuda()], ref, bound)


def test_many_rows_with_topk():
    c = _fill("tiny", "float", [300, 40] + [20] * 10, seed=17)
    rng = np.random.default_rng(3)
    n = 1300
    prefix, seq = np.repeat(rng.integers(-1, 2, 13), 100), rng.integers(2, 12, n)
    q = rng.standard_normal((n, c.Hq, c.d)).astype(np.float16)
    out, mass = c.decode_shared(_ids(seq.tolist()), _ids(prefix.tolist()), torch.from_numpy(q).cuda(), topk=8)
    torch.cuda.synchronize()
    pick = rng.integers(0, n, 200)
    ref, rmass, bound = Exact(c).rows(seq[pick].tolist(), prefix[pick].tolist(), q[pick], topk=8)
    _within(out[torch.from_numpy(pick).cuda()], ref, bound)
    assert np.abs(mass.cpu().numpy()[pick] - rmass).max() <= Hn.MASS_TOL
