"""Shared-prefix decode through the prefix kernel where the other tests' sizes stay
below its threshold: six query heads a kv-head in every format, prefixes of one
page, and short runs beside a long one."""
import os
import re

import numpy as np
import pytest
import torch

from test_gpu_shared import BITS, HEADS, Exact, _compare, _fill, _ids, _within

pytestmark = pytest.mark.gpu

_HEADER = os.path.join(os.path.dirname(__file__), "..", "mixed_precision_paged_thinkv_b200", "csrc", "thinkv_shared.h")
WORTH = int(re.search(r"kWorthPageSteps = (\d+)", open(_HEADER).read()).group(1))


def _takes_prefix_kernel(c, prefix):
    """Both of the rules that send a call's runs to the prefix kernel."""
    pages = c.snapshot()["num_live"]
    runs, at = [], 0
    while at < len(prefix):
        end = at
        while end < len(prefix) and prefix[end] == prefix[at]:
            end += 1
        if prefix[at] >= 0 and end - at > 1:
            runs.append((end - at - 1) * int(pages[prefix[at]]) * c.H)
        at = end
    return sum(runs) >= WORTH and (len(prefix) - 1) * c.max_blocks * c.H >= WORTH


@pytest.mark.parametrize("bits", sorted(BITS))
@pytest.mark.parametrize("members", [40, 43, 100])
def test_six_query_heads(bits, members):
    """240 rows in one block, 258 in two, 600 in three."""
    lens = [5003] + [int(x) for x in np.random.default_rng(7).integers(0, 70, members)]
    c = _fill("gqa6", bits, lens, seed=members, holes=0.15)
    assert _takes_prefix_kernel(c, [0] * members)
    _compare(c, range(1, members + 1), [0] * members)


@pytest.mark.parametrize("heads,members,tokens", [("gqa4", 1200, 1), ("gqa4", 1100, 15), ("mha", 1101, 1), ("gqa8", 1100, 17),
                                                  ("gqa5", 1100, 16), ("gqa3", 1500, 33)])
def test_prefixes_of_a_few_tokens(heads, members, tokens):
    """One key tile with one to three pages."""
    c = _fill(heads, "842", [tokens] + [(i * 7) % 10 for i in range(50)], seed=tokens)
    prefix = [0] * (members * (8 // HEADS[heads][1] + 1) if HEADS[heads][1] < 8 else members)
    seq = [1 + i % 50 for i in range(len(prefix))]
    assert _takes_prefix_kernel(c, prefix)
    _compare(c, seq, prefix, seed=tokens)


def test_short_runs_beside_a_long_one():
    """Runs of two and three rows, on one token and on long prefixes, that go through the
    prefix kernel because of what the call spares as a whole."""
    lens = [6000, 1, 17, 2600, 128, 129] + [(i * 13) % 40 for i in range(90)]
    c = _fill("gqa4", "842", lens, seed=21, holes=0.1)
    prefix = [1] * 2 + [0] * 50 + [2] * 3 + [-1] + [3] * 2 + [4] * 2 + [5] * 3 + [1] * 2 + [0] * 2 + [3] + [4] * 5
    assert _takes_prefix_kernel(c, prefix)
    _compare(c, range(6, 6 + len(prefix)), prefix)


@pytest.mark.parametrize("heads,n", [("tiny", 16384), ("gqa8", 4096)])
def test_one_run_of_many_rows(heads, n):
    """The largest call as one run, and many blocks of rows; a sample is compared."""
    rng = np.random.default_rng(n)
    c = _fill(heads, "float", [900] + [int(x) for x in rng.integers(0, 40, 60)], seed=22, holes=0.1)
    seq, prefix = rng.integers(1, 61, n), np.zeros(n, dtype=np.int64)
    assert _takes_prefix_kernel(c, prefix.tolist())
    q = rng.standard_normal((n, c.Hq, c.d)).astype(np.float16)
    out, _ = c.decode_shared(_ids(seq.tolist()), _ids(prefix.tolist()), torch.from_numpy(q).cuda())
    torch.cuda.synchronize()
    assert c.status() == 0
    pick = np.unique(np.concatenate([rng.integers(0, n, 300), [0, 127, 128, n - 1]]))
    ref, _, bound = Exact(c).rows(seq[pick].tolist(), [0] * len(pick), q[pick])
    _within(out[torch.from_numpy(pick).cuda()], ref, bound)
