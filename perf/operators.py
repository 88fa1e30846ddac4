"""The operators for requests that share a prompt, as measured cases.

- shared-prefix decode attention: each sequence attends over the live tokens of
  a prefix sequence that several of them share, and over its own live tokens
  (``ThinKVCache.decode_shared``);
- release and fork: finished sequences give their pages back to the pools, and
  new ones start as copies of a source sequence (``ThinKVCache.release``,
  ``ThinKVCache.fork``).

With ``own`` false, ``run`` computes them in elementary torch operations on the
cache's buffers (layout: include/thinkv.h); with ``own`` true it makes the
calls of the package.  Inputs are synthetic: K and V are approximately N(0, 1)
with a few outlier channels, quantised into pages of mixed precision, evicted
slots left as holes.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
OUTLIERS = 0.01            # share of (kv-head, channel) pairs with 8x values
MIX = (0.3, 0.5, 0.2)      # share of R, E, T tokens

# head layouts of this repository's workloads: query heads, kv-heads, head dim, group
HEADS = {
    "tiny": (4, 2, 64, 32),
    "llama": (32, 8, 128, 64),
    "qwen": (40, 8, 128, 64),
    "gptoss": (64, 8, 64, 32),
    "mha": (8, 8, 128, 32),          # no sharing of kv-heads
}
BITS = {
    "842": ((8, 4, 2), (0, 0, 0)),               # the default integer codes
    "float": ((8, 4, 2), (1, 1, 1)),             # FP8, FP4, ternary
    "raw": ((16, 8, 4), (0, 0, 0)),              # R tokens kept in fp16
}


def _decode(name, heads, bits, runs, n, prefix, own_lo, own_hi, holes, shape):
    return {"name": name, "op": "decode", "heads": heads, "bits": bits, "runs": runs, "n": n, "prefix": prefix,
            "own_lo": own_lo, "own_hi": own_hi, "holes": holes, "shape": shape}


def _turnover(name, heads, bits, sources, n, tokens, ragged, holes, shape):
    return {"name": name, "op": "turnover", "heads": heads, "bits": bits, "sources": sources, "n": n, "tokens": tokens,
            "ragged": ragged, "holes": holes, "shape": shape}


def listed():
    return [
        # two samples of a short prompt, in the smallest layout: latency counts
        _decode("decode tiny", "tiny", "842", 1, 2, 512, 1, 64, 0.0, 1),
        # two samples of one prompt: hardly anything to share
        _decode("decode pair", "llama", "842", 1, 2, 2048, 1, 128, 0.0, 2),
        # best-of-16 on a long prompt
        _decode("decode sixteen", "llama", "842", 1, 16, 16384, 200, 1024, 0.0, 3),
        # five query heads a kv-head, an evicted prompt with holes, ragged samples
        _decode("decode holes", "qwen", "842", 1, 32, 8191, 0, 2000, 0.3, 4),
        # head dim 64, eight query heads a kv-head, sixty-four samples
        _decode("decode d64", "gptoss", "842", 1, 64, 32768, 100, 1500, 0.05, 5),
        # several prompts in one batch, some requests without one; the float formats
        _decode("decode runs", "llama", "float", 7, 96, 5000, 16, 1200, 0.1, 6),
        # no sharing of kv-heads, raw fp16 R tokens
        _decode("decode mha", "mha", "raw", 2, 200, 3001, 1, 300, 0.02, 7),
        # a large batch on a very long shared context
        _decode("decode largest", "llama", "842", 1, 128, 65536, 512, 2048, 0.0, 8),
        # one finished sample replaced by a new one of a short prompt
        _turnover("turnover one", "tiny", "842", 1, 1, 512, False, 0.0, 9),
        # sixteen samples of one long prompt retire and start again
        _turnover("turnover sixteen", "llama", "842", 1, 16, 16384, False, 0.1, 10),
        # many prompts of ragged lengths, a few samples each
        _turnover("turnover ragged", "qwen", "float", 48, 110, 3000, True, 0.3, 11),
        # a wide restart with raw fp16 R tokens
        _turnover("turnover largest", "gptoss", "raw", 2, 64, 20000, True, 0.05, 12),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    heads, bits = rng.choice(sorted(HEADS)), rng.choice(sorted(BITS))
    holes, shape = rng.choice([0.0, round(rng.uniform(0.0, 0.6), 3)]), rng.randrange(1 << 30)
    if rng.random() < 0.6:
        n, prefix = log(1, 256), log(1, 65536)
        hq, _, d, _ = HEADS[heads]
        prefix = max(1, min(prefix, 128 * 65536 * 32 * 128 // (n * hq * d)))   # the largest listed case's products
        hi = max(1, min(log(1, 4096), 100000 // n))
        c = _decode("", heads, bits, min(n, rng.choice([1, 1, 2, log(1, 24)])), n, prefix, rng.randrange(0, hi + 1), hi, holes, shape)
    else:
        n, tokens = log(1, 128), log(1, 20000)
        sources = rng.randrange(1, max(2, min(n, 40)))
        tokens = max(1, min(tokens, 300000 // (n + sources)))
        c = _turnover("", heads, bits, sources, n, tokens, rng.random() < 0.5, holes, shape)
    del c["name"]
    return c


# ----------------------------------------------------------------------------
# the cache's shape: which sequences hold which pages (from the case alone)
# ----------------------------------------------------------------------------
def _phb(d, g, b):
    return 64 * d if b == 16 else 4 * d * b + 128 * (d // g)


def _shape(case):
    """Table entries, live masks and lengths of every sequence (numpy, from case["shape"])."""
    rng = np.random.default_rng(case["shape"])
    if case["op"] == "decode":
        runs, n = case["runs"], case["n"]
        # prefixes first, then the members; with several runs every fifth has no prefix
        plen = [max(1, int(case["prefix"] * (1.0 if r == 0 else rng.uniform(0.05, 1.0)))) for r in range(runs)]
        cuts = np.sort(rng.choice(np.arange(1, n), size=runs - 1, replace=False)) if runs > 1 else np.zeros(0, np.int64)
        run_of = np.searchsorted(cuts, np.arange(n), side="right")
        prefix = np.array([-1 if runs > 1 and r % 5 == 4 else r for r in range(runs)])[run_of]
        seq = runs + np.arange(n)
        lens = plen + [int(x) for x in rng.integers(case["own_lo"], case["own_hi"] + 1, n)]
        more = {"prefix": prefix.astype(np.int32), "seq": seq.astype(np.int32), "run_of": run_of.astype(np.int64)}
    else:
        m, n = case["sources"], case["n"]
        lens = [max(1, int(case["tokens"] * (rng.uniform(0.05, 1.0) if case["ragged"] and i else 1.0))) for i in range(m)]
        src = np.sort(rng.integers(0, m, n))
        more = {"src": src.astype(np.int32), "dst": (m + rng.permutation(n)).astype(np.int32)}
    seqs = []                                       # per sequence: class, used slots, live mask of each entry
    for length in lens:
        cnt = rng.multinomial(length, MIX)
        pages = (cnt + PAGE - 1) // PAGE
        cls = rng.permutation(np.repeat(np.arange(3), pages))
        rank = np.zeros(len(cls), np.int64)
        for c in range(3):
            rank[cls == c] = np.arange(pages[c])
        used = np.minimum(PAGE, cnt[cls] - rank * PAGE)
        slot_used = np.arange(PAGE)[None, :] < used[:, None]
        live = slot_used & (rng.random((len(cls), PAGE)) >= case["holes"])
        seqs.append({"cls": cls, "used": slot_used, "live": live})
    if case["op"] == "turnover":                    # the children: as many pages as their source, other contents
        kids = [None] * n
        for s, t in zip(more["src"], more["dst"]):
            p = seqs[s]
            kids[t - m] = {"cls": rng.permutation(p["cls"]), "used": p["used"], "live": p["live"] & (rng.random(p["live"].shape) < 0.5)}
        seqs = seqs + kids
    return {"seqs": seqs, **more}


def _tokens(seqs, i):
    return int(seqs[i]["live"].sum())


def _phbs(case):
    (_, _, d, g), (bits, _) = HEADS[case["heads"]], BITS[case["bits"]]
    return [_phb(d, g, b) for b in bits]


def work(case):
    hq, h, d, g = HEADS[case["heads"]]
    bits, _ = BITS[case["bits"]]
    sh = _shape(case)
    seqs = sh["seqs"]
    if case["op"] == "decode":
        tok = [2 * d * b / 8 + (0 if b == 16 else 8 * (d // g)) for b in bits]     # K and V bytes of a token and head

        def read(i):
            p = seqs[i]
            per = p["live"].sum(1)
            return sum(h * tok[c] * int(per[p["cls"] == c].sum()) + 16 * int(((p["cls"] == c) & (per > 0)).sum()) for c in range(3))

        prefixes = sorted({int(x) for x in sh["prefix"] if x >= 0})
        nbytes = sum(read(i) for i in prefixes) + sum(read(int(i)) for i in sh["seq"])
        nbytes += case["n"] * (2 * hq * d * 2 + 8)
        pairs = sum(_tokens(seqs, int(s)) + (_tokens(seqs, int(p)) if p >= 0 else 0) for s, p in zip(sh["seq"], sh["prefix"]))
        return {"bytes": float(nbytes), "flops": 4.0 * hq * d * pairs}
    phb = _phbs(case)

    def held(i, what):                               # bytes of a sequence's pages, or of its bookkeeping
        p = seqs[i]
        pages = np.bincount(p["cls"], minlength=3)
        if what == "pages":
            return float(sum(pages[c] * (h * phb[c] + 64) for c in range(3)))
        return float(16 * p["used"].sum() + 20 * len(p["cls"]) + 64)               # FIFO, free slots, table, live list

    nbytes = sum(held(int(i), "pages") + held(int(i), "book") for i in np.unique(sh["src"]))
    nbytes += sum(held(int(i), "pages") + held(int(i), "book") + 76.0 * len(seqs[int(i)]["cls"]) for i in sh["dst"])
    return {"bytes": nbytes, "flops": 0.0}


# ----------------------------------------------------------------------------
# packed codes: where each code of a page-head block sits
# ----------------------------------------------------------------------------
_ORDER = {}


def _order(d, g, b, kv, device):
    """For one K or V region: the field (b-bit, in memory order) of each (slot, channel)."""
    key = (d, g, b, kv, str(device))
    if key not in _ORDER:
        slot, ch = np.meshgrid(np.arange(PAGE), np.arange(d), indexing="ij")
        if kv == 0:
            gid, r, gr, t, e = slot % 8, slot // 8, ch // g, (ch % g) // (g // 4), ch % (g // 4)
            word = min(32, g * b // 4)               # bits of a word of the piece
            m = max(1, word // b)
            p = e if b == 16 else np.where(e % 2 == 0, e % m // 2, m // 2 + e % m // 2)
            bit = (gr * 2 + r) * (g * b // 4) + (e * 16 if b == 16 else e // m * word + p * b)
            lane = 4 * gid + t
        else:
            half, t, pp = slot % 2, slot % 8 // 2, slot // 8
            e, gid = ch // 16 * 2 + ch % 16 // 8, ch % 8
            q = d // 8 if b == 16 else d * b // 128
            per = 1 if b == 16 else 16 // b
            bit = (pp * q + e // per) * 32 + half * 16 + e % per * b
            lane = 4 * gid + t
        lb = d * b // 16
        u = min(16, lb)
        o = bit // 8
        at = (o // u) * 32 * u + lane * u + o % u    # byte of the region
        field = (at * 8 + bit % 8) // b
        _ORDER[key] = torch.from_numpy(field.astype(np.int64)).to(device)
    return _ORDER[key]


_FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _codes(x, b, f, g):
    """x fp32 [..., d] -> codes (uint8, or fp16 values for b = 16), scale and zero (fp16 [..., d/g])."""
    if b == 16:
        return x.half(), None, None
    y = x.unflatten(-1, (-1, g))
    if f == 0:
        z = (y.amin(-1) - 1e-3).half()
        s = ((y.amax(-1) - z.float()) / (2 ** b - 1) * 1.001).half()
        c = torch.round((y - z.float()[..., None]) / s.float()[..., None]).clamp(0, 2 ** b - 1).to(torch.uint8)
        return c.flatten(-2), s, z
    s = (y.abs().amax(-1) / (448.0 if b == 8 else 6.0 if b == 4 else 1.0) * 1.001).half()
    r = y / s.float()[..., None]
    z = torch.zeros_like(s) if b != 2 else -s
    if b == 8:
        c = r.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    elif b == 4:
        grid = torch.tensor(_FP4, device=x.device)
        k = torch.bucketize(r.abs(), (grid[1:] + grid[:-1]) / 2)
        c = (k + 8 * (r < 0)).to(torch.uint8)
    else:
        c = (torch.round(r).clamp(-1, 1) + 1).to(torch.uint8)
    return c.flatten(-2), s, z


def _pack(codes, b, order):
    """codes [..., 16, d] -> bytes of the region [..., 2*d*b]."""
    flat = codes.flatten(-2)
    mem = torch.empty_like(flat)
    mem[..., order.reshape(-1)] = flat
    if b == 16:
        return mem.view(torch.uint8)
    per = 8 // b
    parts = mem.unflatten(-1, (-1, per)).int()
    return (parts << torch.arange(0, 8, b, device=mem.device, dtype=torch.int32)).sum(-1).to(torch.uint8)


def _values(pool, region, b, f, d, g, order):
    """Values (fp32 [pages, H, 16, d]) of the K (region 0) or V (region 1) codes of a pool."""
    size = 2 * d * b
    raw = pool[..., region * size:(region + 1) * size].contiguous()
    if b == 16:
        return raw.view(torch.float16)[..., order].float()
    mem = (raw[..., None] >> torch.arange(0, 8, b, device=raw.device, dtype=torch.uint8)) & (2 ** b - 1)
    code = mem.flatten(-2)[..., order]               # [pages, H, 16, d]
    ng = d // g
    at = 2 * size + region * 64 * ng
    par = pool[..., at:at + 64 * ng].contiguous().view(torch.float16).float().unflatten(-1, (ng, PAGE, 2))
    par = par.transpose(-3, -2).repeat_interleave(g, dim=-2)     # [pages, H, 16, d, (scale, zero)]
    if f == 1 and b == 8:
        val = code.view(torch.float8_e4m3fn).float()
    elif f == 1 and b == 4:
        grid = torch.tensor(_FP4 + tuple(-x for x in _FP4), device=raw.device)
        val = grid[code.long()]
    else:
        val = code.float()
    return val * par[..., 0] + par[..., 1]


# ----------------------------------------------------------------------------
# prepare: the cache's buffers and the call's inputs
# ----------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    hq, h, d, g = HEADS[case["heads"]]
    bits, fmt = BITS[case["bits"]]
    sh = _shape(case)
    seqs = sh["seqs"]
    ns, nb = len(seqs), max(1, max(len(p["cls"]) for p in seqs))
    cap = nb * PAGE
    rng = np.random.default_rng([seed, case["shape"]])
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    first = np.concatenate([[0], np.cumsum([len(p["cls"]) for p in seqs])])
    cls = np.concatenate([p["cls"] for p in seqs])
    live = np.concatenate([p["live"] for p in seqs])
    used = np.concatenate([p["used"] for p in seqs])
    owner = np.repeat(np.arange(ns), np.diff(first))
    entry = np.arange(len(cls)) - first[owner]
    page = np.zeros(len(cls), np.int64)
    total = [int((cls == c).sum()) for c in range(3)]
    pool_pages = [t + 4 for t in total]
    for c in range(3):
        page[cls == c] = rng.permutation(total[c])
    mask = (live << np.arange(PAGE)).sum(1).astype(np.int64)

    table = np.zeros((ns, nb), np.uint64)
    table[owner, entry] = (page.astype(np.uint64) | (cls.astype(np.uint64) << np.uint64(32)) | (mask.astype(np.uint64) << np.uint64(48)))
    llist, lindex = np.zeros((ns, nb), np.uint64), np.full((ns, nb), -1, np.int32)
    num_live = np.zeros(ns, np.int32)
    fifo, head, tail = np.zeros((ns, 3, cap), np.int32), np.zeros((ns, 3), np.int32), np.zeros((ns, 3), np.int32)
    free, top = np.zeros((ns, 3, cap), np.int32), np.zeros((ns, 3), np.int32)
    for s, p in enumerate(seqs):
        at = rng.permutation(np.flatnonzero(p["live"].any(1)))
        num_live[s] = len(at)
        f = first[s]
        llist[s, :len(at)] = page[f + at].astype(np.uint64) | (p["cls"][at].astype(np.uint64) << np.uint64(32)) | (at.astype(np.uint64) << np.uint64(40))
        lindex[s, at] = np.arange(len(at))
        for c in range(3):
            of = np.flatnonzero(p["cls"] == c)
            ids = (of[:, None] * PAGE + np.arange(PAGE)).reshape(-1)
            u, lv = p["used"][of].reshape(-1), p["live"][of].reshape(-1)
            order = np.where(lv, ids, -1)[u]                     # arrival order; evicted tokens left tombstones
            head[s, c] = rng.integers(0, 2 * cap)
            tail[s, c] = head[s, c] + len(order)
            fifo[s, c, (head[s, c] + np.arange(len(order))) % cap] = order
            gone = rng.permutation(ids[~lv])
            free[s, c, :len(gone)] = gone
            top[s, c] = len(gone)

    buf, vals = {}, {}
    for c, name in enumerate("RET"):
        b, f = bits[c], fmt[c]
        spots = torch.rand(h, d, device=dev, generator=gen) < OUTLIERS
        parts, prm = [], []
        for kv in range(2):
            x = torch.randn(pool_pages[c], h, PAGE, d, device=dev, generator=gen)
            x = torch.where(spots[None, :, None, :], x * 8, x).half().float()
            code, s, z = _codes(x, b, f, g)
            parts.append(_pack(code, b, _order(d, g, b, kv, dev)))
            if b != 16:
                prm.append(torch.stack([s, z], -1).transpose(-3, -2).contiguous().flatten(-3).view(torch.uint8))
        buf["pool_" + name] = torch.cat(parts + prm, -1).contiguous()
        pos = np.full((pool_pages[c], PAGE), -1, np.int32)
        own_c = cls == c
        pos[page[own_c]] = np.where(live[own_c], (entry[own_c] * PAGE)[:, None] + np.arange(PAGE), -1)
        vals["slot_pos_" + name] = pos
    bump = np.zeros(6 + sum(pool_pages), np.int32)
    bump[:3] = total
    vals.update(block_table=table.view(np.int64), num_blocks=np.diff(first).astype(np.int32), free_slots=free, free_top=top,
                fifo=fifo, fifo_head=head, fifo_tail=tail,
                live_count=np.array([int(p["live"].sum()) for p in seqs], np.int32), live_list=llist.view(np.int64),
                live_index=lindex, num_live=num_live, page_bump=bump, status=np.zeros(1, np.int32))
    buf.update({k: torch.from_numpy(v).to(dev) for k, v in vals.items()})
    state = {"case": case, "geo": (hq, h, d, g, bits, fmt, ns, nb, tuple(pool_pages)), "buf": buf}
    if case["op"] == "decode":
        n = case["n"]
        state["q"] = torch.randn(n, hq, d, device=dev, generator=gen).half()
        state["seq"], state["prefix"] = (torch.from_numpy(sh[k]).to(dev) for k in ("seq", "prefix"))
        # the plain form's plan: which run and which place of it each sequence has
        run_of = sh["run_of"]
        place = np.arange(n) - np.searchsorted(run_of, run_of)
        state["place"] = torch.from_numpy(run_of * (place.max() + 1) + place).to(dev)
        state["rows"] = (case["runs"], int(place.max()) + 1)
        state["run_prefix"] = torch.from_numpy(sh["prefix"][np.searchsorted(run_of, np.arange(case["runs"]))].astype(np.int64)).to(dev)
        state["most"] = (int(num_live[:case["runs"]].max()), max(1, int(num_live[case["runs"]:].max())))
    else:
        state["src"], state["dst"] = (torch.from_numpy(sh[k]).to(dev) for k in ("src", "dst"))
    return state


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------
def _all_values(state):
    """K and V of every page of the three pools, fp32 [pages, H, 16, d]."""
    hq, h, d, g, bits, fmt, ns, nb, pool_pages = state["geo"]
    buf, dev = state["buf"], state["q"].device
    return [torch.cat([_values(buf["pool_" + n], x, bits[c], fmt[c], d, g, _order(d, g, bits[c], x, dev)) for c, n in enumerate("RET")]) for x in range(2)]


def _pages(state, values, ids, most):
    """K and V (fp32 [x, H, most*16, d]) and the live tokens of the sequences ids (-1: none)."""
    pool_pages, buf = state["geo"][-1], state["buf"]
    have = ids >= 0
    row = buf["live_list"][ids.clamp(min=0), :most]
    ok = (torch.arange(most, device=row.device) < buf["num_live"][ids.clamp(min=0)][:, None]) & have[:, None]
    row = torch.where(ok, row, 0)
    page, cls, ent = row & 0xFFFFFFFF, (row >> 32) & 0xFF, row >> 40
    start = torch.tensor([0, pool_pages[0], pool_pages[0] + pool_pages[1]], device=row.device)
    at = page + start[cls]
    mask = (torch.gather(buf["block_table"][ids.clamp(min=0)], 1, ent) >> 48) & 0xFFFF
    live = (((mask[..., None] >> torch.arange(PAGE, device=row.device)) & 1) == 1) & ok[..., None]
    k, v = (x[at].transpose(1, 2).flatten(2, 3) for x in values)
    return k, v, live.flatten(1)


def _attend(q, k, v, live, scale):
    """Row maxima, sums and unnormalised rows of softmax attention: q [x, H, r, d]."""
    s = (q @ k.transpose(-1, -2)) * scale
    s = torch.where(live[:, None, None, :], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    v = torch.where(live[:, None, :, None], v, 0.0)
    return m, p.sum(-1, keepdim=True), p @ v


def _plain_decode(state):
    hq, h, d, g, bits, fmt, ns, nb, pool_pages = state["geo"]
    q, n = state["q"].float(), state["case"]["n"]
    gq, scale = hq // h, 1.0 / math.sqrt(d)
    runs, most = state["rows"]
    # the prefix, once a run: the rows of all its members together
    qr = torch.zeros(runs * most, hq, d, device=q.device).index_copy(0, state["place"], q)
    qr = qr.view(runs, most, h, gq, d).transpose(1, 2).reshape(runs, h, most * gq, d)
    values = _all_values(state)
    k, v, live = _pages(state, values, state["run_prefix"], state["most"][0])
    part = _attend(qr, k, v, live, scale)
    m1, l1, o1 = (x.view(runs, h, most, gq, -1).transpose(1, 2).reshape(runs * most, h, gq, -1)[state["place"]] for x in part)
    # each sequence's own tokens
    k, v, live = _pages(state, values, state["seq"].long(), state["most"][1])
    m2, l2, o2 = _attend(q.view(n, h, gq, d), k, v, live, scale)
    m = torch.maximum(m1, m2)
    m = torch.where(m == -math.inf, 0.0, m)
    w1, w2 = torch.exp(m1 - m), torch.exp(m2 - m)
    l = l1 * w1 + l2 * w2
    o = torch.where(l > 0, (o1 * w1 + o2 * w2) / torch.where(l > 0, l, 1.0), 0.0)
    return o.reshape(n, hq, d).half()


def _entries(buf, ids):
    """Table entries of the sequences ids: (row, entry, page, class) of each, in call order."""
    t, nb = buf["block_table"][ids], buf["num_blocks"][ids]
    row, ent = torch.nonzero(torch.arange(t.shape[1], device=t.device) < nb[:, None], as_tuple=True)
    x = t[row, ent]
    return row, ent, x & 0xFFFFFFFF, (x >> 32) & 0xFF


def _plain_release(state, ids):
    pool_pages, buf = state["geo"][-1], state["buf"]
    ids = ids.long()
    row, ent, page, cls = _entries(buf, ids)
    bump = buf["page_bump"]
    for c, name in enumerate("RET"):
        mine = page[cls == c]
        at = 6 + sum(pool_pages[:c]) + bump[3 + c] + torch.arange(len(mine), device=mine.device)
        bump[at] = mine.flip(0).int()                # the first page released is the first granted again
        bump[3 + c] += len(mine)
        buf["slot_pos_" + name][mine] = -1
    buf["block_table"][ids[row], ent] = 0
    buf["live_index"][ids[row], ent] = -1
    for name in ("num_blocks", "free_top", "fifo_head", "fifo_tail", "live_count", "num_live"):
        buf[name][ids] = 0


def _plain_fork(state, src, dst):
    pool_pages, buf = state["geo"][-1], state["buf"]
    src, dst = src.long(), dst.long()
    row, ent, page, cls = _entries(buf, src)
    bump, new = buf["page_bump"], torch.empty_like(page)
    for c, name in enumerate("RET"):
        mine = cls == c
        k = torch.arange(int(mine.sum()), device=page.device)
        freed = bump[3 + c].long()
        at = 6 + sum(pool_pages[:c]) + (freed - 1 - k).clamp(min=0)
        new[mine] = torch.where(k < freed, bump[at].long(), bump[c] + k - freed)
        took = torch.minimum(freed, torch.tensor(len(k), device=page.device))
        bump[3 + c] -= took.int()
        bump[c] += (len(k) - took).int()
        for pool in ("pool_", "slot_pos_"):
            buf[pool + name][new[mine]] = buf[pool + name][page[mine]]
    old = buf["block_table"][src[row], ent]
    buf["block_table"][dst[row], ent] = (old & ~0xFFFFFFFF) | new
    index = buf["live_index"][src[row], ent]
    buf["live_index"][dst[row], ent] = index
    on = index >= 0
    buf["live_list"][dst[row[on]], index[on].long()] = new[on] | (cls[on] << 32) | (ent[on] << 40)
    cap = buf["fifo"].shape[2]
    at = torch.arange(cap, device=page.device)
    h, t = buf["fifo_head"][src].long()[..., None], buf["fifo_tail"][src].long()[..., None]
    inside = (at - h) % cap < t - h                  # the ring's window
    buf["fifo"][dst] = torch.where(inside, buf["fifo"][src], buf["fifo"][dst])
    buf["free_slots"][dst] = torch.where(at < buf["free_top"][src][..., None], buf["free_slots"][src], buf["free_slots"][dst])
    for name in ("num_blocks", "free_top", "fifo_head", "fifo_tail", "live_count", "num_live"):
        buf[name][dst] = buf[name][src]


def _cache(state):
    """The package's cache over the state's buffers, opened at the first pass and kept."""
    if "cache" not in state:
        from mixed_precision_paged_thinkv_b200 import ThinKVCache
        hq, h, d, g, bits, fmt, ns, nb, pool_pages = state["geo"]
        state["cache"] = ThinKVCache(hq, h, d, g, bits, ns, nb, pool_pages, fmt=fmt, buffers=state["buf"])
    return state["cache"]


def run(state):
    if state["case"]["op"] == "decode":
        if own:
            return _cache(state).decode_shared(state["seq"], state["prefix"], state["q"])[0]
        return _plain_decode(state)
    if own:
        _cache(state).release(state["dst"])
        _cache(state).fork(state["src"], state["dst"])
    else:
        _plain_release(state, state["dst"])
        _plain_fork(state, state["src"], state["dst"])
    return state["buf"]


# ----------------------------------------------------------------------------
# exact: 64 bits, one sequence and one kv-head's rows after the other
# ----------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] != "decode":
        return None                                  # copies: no computed numbers
    state = prepare(case, seed)
    hq, h, d, g, bits, fmt, ns, nb, pool_pages = state["geo"]
    dev = state["q"].device
    gq = hq // h
    seq, prefix = state["seq"].tolist(), state["prefix"].tolist()
    if sum(_tokens(_shape(case)["seqs"], max(p, 0)) for p in prefix) * hq * d > 1 << 38:
        return None
    tables = state["buf"]["block_table"].cpu().numpy().view(np.uint64)
    blocks = state["buf"]["num_blocks"].tolist()

    def codes(pages, c, region):
        """Field by field from the documented places of each lane's bytes."""
        b = bits[c]
        raw = state["buf"]["pool_" + "RET"[c]][pages]              # [p, H, phb]
        lb, ng = d * b // 16, d // g
        u = min(16, lb)
        out = torch.zeros(raw.shape[0], h, PAGE, d, dtype=torch.int32, device=dev)
        lane = np.arange(32)
        gid, tid = lane // 4, lane % 4
        base = region * 2 * d * b

        def byte(o):                                               # byte o of every lane's portion
            return raw[:, :, torch.from_numpy(base + o // u * 32 * u + lane * u + o % u).to(dev)].int()

        if region == 0:
            for gr in range(ng):
                for r in range(2):
                    for e in range(g // 4):
                        first = (gr * 2 + r) * g * b // 32
                        if b == 16:
                            v = byte(first + 2 * e) | (byte(first + 2 * e + 1) << 8)
                        else:
                            word = min(4, g * b // 32)             # bytes of a word
                            per = word * 8 // b
                            w, x = e // per, e % per
                            bit = (x // 2 + (per // 2 if x % 2 else 0)) * b
                            v = (byte(first + w * word + bit // 8) >> (bit % 8)) & (2 ** b - 1)
                        out[:, :, torch.from_numpy(gid + 8 * r).to(dev), torch.from_numpy(gr * g + tid * (g // 4) + e).to(dev)] = v
        else:
            q = d // 8 if b == 16 else d * b // 128
            per = 1 if b == 16 else 16 // b
            for half_page in range(2):
                for w in range(q):
                    for half in range(2):
                        for x in range(per):
                            e = w * per + x
                            o = (half_page * q + w) * 4 + half * 2
                            v = (byte(o) | (byte(o + 1) << 8)) if b == 16 else (byte(o + x * b // 8) >> (x * b % 8)) & (2 ** b - 1)
                            out[:, :, torch.from_numpy(2 * tid + 8 * half_page + half).to(dev),
                                torch.from_numpy(16 * (e // 2) + gid + 8 * (e % 2)).to(dev)] = v
        if b == 16:
            return out.to(torch.int16).view(torch.float16).double()
        at = 4 * d * b + region * 64 * ng
        par = raw[:, :, at:at + 64 * ng].contiguous().view(torch.float16).double().view(-1, h, ng, PAGE, 2)
        s, z = (par[..., x].transpose(2, 3)[..., None] for x in range(2))
        if fmt[c] == 1 and b == 8:
            sign, exp, man = out >> 7, (out >> 3) & 15, (out & 7).double()
            mag = torch.where(exp == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * torch.pow(2.0, (exp - 7).double()))
            val = torch.where(sign == 1, -mag, mag)
        elif fmt[c] == 1 and b == 4:
            sign, exp, man = out >> 3, (out >> 1) & 3, (out & 1).double()
            mag = torch.where(exp == 0, man / 2, (1 + man / 2) * torch.pow(2.0, (exp - 1).double()))
            val = torch.where(sign == 1, -mag, mag)
        else:
            val = out.double()
        return (val.unflatten(-1, (ng, g)) * s + z).flatten(-2)

    def tokens(s):
        """K and V of a sequence's live tokens, fp64 [H, tokens, d]."""
        t = tables[s, :blocks[s]]
        got = [[], []]
        for c in range(3):
            mine = t[((t >> np.uint64(32)) & np.uint64(0xFF)) == c]
            if not len(mine):
                continue
            pages = torch.from_numpy((mine & np.uint64(0xFFFFFFFF)).astype(np.int64)).to(dev)
            live = torch.from_numpy(((mine >> np.uint64(48))[:, None] >> np.arange(PAGE, dtype=np.uint64)) & np.uint64(1) == 1).to(dev)
            for region in range(2):
                got[region].append(codes(pages, c, region).transpose(1, 2)[live])
        return [torch.cat(x).transpose(0, 1) if x else torch.zeros(h, 0, d, dtype=torch.float64, device=dev) for x in got]

    out = torch.zeros(case["n"], hq, d, dtype=torch.float64, device=dev)
    kept = (None, None)
    for i, (s, p) in enumerate(zip(seq, prefix)):
        k, v = tokens(s)
        if p >= 0:
            if kept[0] != p:
                kept = (p, tokens(p))
            k, v = torch.cat([kept[1][0], k], 1), torch.cat([kept[1][1], v], 1)
        if k.shape[1]:
            logit = state["q"][i].double().view(h, gq, d) @ k.transpose(1, 2) / math.sqrt(d)
            out[i] = (torch.softmax(logit, -1) @ v).reshape(hq, d)
    return out
