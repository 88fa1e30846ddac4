"""Release and fork on host copies of a cache's buffers (plain numpy): what the
calls do to every array, sequence by sequence and page by page."""
import numpy as np

PAGE = 16


def host_buffers(cache) -> dict:
    """Every buffer of the cache as a numpy array in its documented shape."""
    ns, nb = cache.max_seqs, cache.max_blocks
    cap = nb * PAGE
    shapes = {"block_table": (np.uint64, (ns, nb)), "num_blocks": (np.int32, (ns,)),
              "free_slots": (np.int32, (ns, 3, cap)), "free_top": (np.int32, (ns, 3)),
              "fifo": (np.int32, (ns, 3, cap)), "fifo_head": (np.int32, (ns, 3)),
              "fifo_tail": (np.int32, (ns, 3)), "live_count": (np.int32, (ns,)),
              "live_list": (np.uint64, (ns, nb)), "live_index": (np.int32, (ns, nb)),
              "num_live": (np.int32, (ns,)), "status": (np.int32, (1,)),
              "page_bump": (np.int32, (6 + sum(cache.pool_pages),))}
    for c, n in enumerate("RET"):
        shapes["pool_" + n] = (np.uint8, (cache.pool_pages[c], cache.H * cache.page_head_bytes(c)))
        shapes["slot_pos_" + n] = (np.int32, (cache.pool_pages[c], PAGE))
    out = {k: cache._host(k, *v) for k, v in shapes.items()}
    if cache.tbe is not None:
        for k, shape in (("seg", (ns, cap, 4)), ("nseg", (ns,)), ("settled", (ns,))):
            out[k] = cache.tbe_buf[k].cpu().numpy().view(np.int32).reshape(shape).copy()
    return out


def _stacks(b, pool_pages):
    first = 6
    for c in range(3):
        yield c, first
        first += pool_pages[c]


def release(b: dict, seqs, pool_pages):
    first = dict(_stacks(b, pool_pages))
    pages = [[], [], []]
    for s in seqs:
        for e in range(b["num_blocks"][s]):
            x = int(b["block_table"][s, e])
            page, c = x & 0xFFFFFFFF, (x >> 32) & 0xFF
            pages[c].append(page)
            b["slot_pos_" + "RET"[c]][page] = -1
            b["block_table"][s, e] = 0
            b["live_index"][s, e] = -1
        for k in ("num_blocks", "live_count", "num_live", "free_top", "fifo_head", "fifo_tail"):
            b[k][s] = 0
        for k in ("nseg", "settled"):
            if k in b:
                b[k][s] = 0
    for c in range(3):
        for page in reversed(pages[c]):
            b["page_bump"][first[c] + b["page_bump"][3 + c]] = page
            b["page_bump"][3 + c] += 1


def fork(b: dict, src, dst, pool_pages):
    first = dict(_stacks(b, pool_pages))
    cap = b["fifo"].shape[2]
    for s, t in zip(src, dst):
        for e in range(b["num_blocks"][s]):
            x = int(b["block_table"][s, e])
            page, c = x & 0xFFFFFFFF, (x >> 32) & 0xFF
            if b["page_bump"][3 + c]:
                b["page_bump"][3 + c] -= 1
                new = int(b["page_bump"][first[c] + b["page_bump"][3 + c]])
            else:
                new = int(b["page_bump"][c])
                b["page_bump"][c] += 1
            for k in ("pool_", "slot_pos_"):
                b[k + "RET"[c]][new] = b[k + "RET"[c]][page]
            b["block_table"][t, e] = (x & ~0xFFFFFFFF) | new
            at = int(b["live_index"][s, e])
            b["live_index"][t, e] = at
            if at >= 0:
                b["live_list"][t, at] = new | (c << 32) | (e << 40)
        for c in range(3):
            top = b["free_top"][s, c]
            b["free_slots"][t, c, :top] = b["free_slots"][s, c, :top]
            idx = np.arange(b["fifo_head"][s, c], b["fifo_tail"][s, c]) % cap
            b["fifo"][t, c, idx] = b["fifo"][s, c, idx]
        for k in ("num_blocks", "live_count", "num_live", "free_top", "fifo_head", "fifo_tail"):
            b[k][t] = b[k][s]
        if "nseg" in b:
            b["seg"][t, :b["nseg"][s]] = b["seg"][s, :b["nseg"][s]]
            b["nseg"][t], b["settled"][t] = b["nseg"][s], b["settled"][s]


def assert_same(got: dict, want: dict, skip=()):
    for k in want:
        if k not in skip:
            assert np.array_equal(got[k], want[k]), k
