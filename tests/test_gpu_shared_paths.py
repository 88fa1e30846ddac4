"""Shared-prefix decode through the prefix kernel where the other tests' sizes stay
below its threshold: few kv-heads in every format, few rows, prefixes of one page,
and short runs beside a long one."""
import os
import re

import numpy as np
import pytest
import torch

from test_gpu_shared import BITS, HEADS, Exact, _compare, _fill, _ids, _within

pytestmark = pytest.mark.gpu

_HEADER = os.path.join(os.path.dirname(__file__), "..", "mixed_precision_paged_thinkv_b200", "csrc", "thinkv_shared.h")
TILE_COST, WORTH = (int(re.search(name + r" = (\d+)", open(_HEADER).read()).group(1))
                    for name in ("kTileCost", "kWorthPageSteps"))


def _runs_taken(c, prefix):
    """The rows that the prefix kernel takes, by the rules of the plan and the launch."""
    pages = c.snapshot()["num_live"]
    runs, gained, at = [], 0, 0
    while at < len(prefix):
        end = at
        while end < len(prefix) and prefix[end] == prefix[at]:
            end += 1
        if prefix[at] >= 0 and end - at > 1:
            n, p = end - at, int(pages[prefix[at]])
            blocks = -(-n // (256 // (c.Hq // c.H)))
            gain = ((n - 1) * p - TILE_COST * blocks * -(-p // 8)) * c.H
            if gain > 0:
                runs.append((at, n))
                gained += gain
        at = end
    return runs if gained >= WORTH and (len(prefix) - 1) * c.max_blocks * c.H >= WORTH else []


@pytest.mark.parametrize("bits", sorted(BITS))
@pytest.mark.parametrize("heads,members,prefix", [("gqa6", 40, 16003), ("gqa6", 43, 16003), ("gqa6", 100, 8003),
                                                  ("gqa3", 50, 8003), ("gqa3", 90, 8003), ("gqa7", 60, 8003),
                                                  ("tiny", 80, 8003)])
def test_few_kv_heads(heads, bits, members, prefix):
    """One to three kv-heads; six query heads with 240 rows in one block, 258 in two
    and 600 in three."""
    lens = [prefix] + [int(x) for x in np.random.default_rng(7).integers(0, 70, members)]
    c = _fill(heads, bits, lens, seed=members, holes=0.15)
    assert _runs_taken(c, [0] * members) == [(0, members)]
    _compare(c, range(1, members + 1), [0] * members)


@pytest.mark.parametrize("members,prefix,own", [(3, 70000, 5), (5, 20000, 0), (9, 9000, 30), (16, 4000, 300), (17, 4001, 1)])
def test_few_rows(members, prefix, own):
    lens = [prefix] + [(i * 7) % (own + 1) for i in range(members)]
    c = _fill("gqa4", "842", lens, seed=members)
    assert _runs_taken(c, [0] * members) == [(0, members)]
    _compare(c, range(1, members + 1), [0] * members, seed=members)


@pytest.mark.parametrize("heads,members,tokens", [("gqa4", 4000, 1), ("gqa4", 3000, 15), ("mha", 3500, 1), ("gqa8", 2500, 17),
                                                  ("gqa5", 3000, 16), ("gqa3", 4000, 33)])
def test_prefixes_of_a_few_tokens(heads, members, tokens):
    """One key tile with one to four pages."""
    c = _fill(heads, "842", [tokens] + [(i * 7) % 10 for i in range(50)], seed=tokens)
    prefix = [0] * members
    seq = [1 + i % 50 for i in range(members)]
    assert _runs_taken(c, prefix) == [(0, members)]
    _compare(c, seq, prefix, seed=tokens)


def test_short_runs_beside_a_long_one():
    """Runs of three and five rows, on one token and on long prefixes, that go through
    the prefix kernel because of what the call gains as a whole; runs of two do not."""
    lens = [6000, 1, 17, 2600, 128, 129] + [(i * 13) % 40 for i in range(90)]
    c = _fill("gqa4", "842", lens, seed=21, holes=0.1)
    prefix = [3] * 3 + [0] * 50 + [2] * 5 + [-1] + [3] * 2 + [4] * 4 + [5] * 3 + [1] * 14 + [0] * 2 + [3]
    taken = _runs_taken(c, prefix)
    assert (0, 3) in taken and (3, 50) in taken and len(taken) >= 4 and all(n > 2 for _, n in taken)
    _compare(c, range(6, 6 + len(prefix)), prefix)


@pytest.mark.parametrize("heads,n", [("tiny", 16384), ("gqa8", 4096)])
def test_one_run_of_many_rows(heads, n):
    """The largest call as one run, and many blocks of rows; a sample is compared."""
    rng = np.random.default_rng(n)
    c = _fill(heads, "float", [900] + [int(x) for x in rng.integers(0, 40, 60)], seed=22, holes=0.1)
    seq, prefix = rng.integers(1, 61, n), np.zeros(n, dtype=np.int64)
    assert _runs_taken(c, prefix.tolist()) == [(0, n)]
    q = rng.standard_normal((n, c.Hq, c.d)).astype(np.float16)
    out, _ = c.decode_shared(_ids(seq.tolist()), _ids(prefix.tolist()), torch.from_numpy(q).cuda())
    torch.cuda.synchronize()
    assert c.status() == 0
    pick = np.unique(np.concatenate([rng.integers(0, n, 300), [0, 127, 128, n - 1]]))
    ref, _, bound = Exact(c).rows(seq[pick].tolist(), [0] * len(pick), q[pick])
    _within(out[torch.from_numpy(pick).cuda()], ref, bound)
