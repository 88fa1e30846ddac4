"""Decode where a raw fp16 page raises the running maximum after pages with zero
terms: the zero terms summed so far move with the maximum like the rest."""
import numpy as np
import pytest
import torch

from oracle import oracle as O
from mixed_precision_paged_thinkv_b200.binding import ThinKVCache

import harness as Hn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,G", [(64, 32), (64, 64), (128, 32), (128, 64)])
def test_raw_page_that_raises_the_maximum(d, G):
    # 7,500 pages a head of the two long sequences: every split warp steps through several of them;
    # pages alternate between 4-bit (values around 5: large zero terms) and raw fp16, and
    # the raw keys grow along the sequence
    args = (2, 2, d, G, (16, 4, 2), 8, 3800, (15100, 15100, 10))
    c, o = ThinKVCache(*args), O.Oracle(*args)
    rng = np.random.default_rng(d + G)
    n = 60000
    tag = np.repeat(np.arange(n // 16) % 2, 16).astype(np.uint8)
    k = rng.standard_normal((n, 2, d)).astype(np.float32) * 0.1
    k += (tag == 0)[:, None, None] * np.linspace(0, 0.5, n)[:, None, None]
    v = rng.standard_normal((n, 2, d)).astype(np.float32) * 0.1 + 5 * (tag == 1)[:, None, None]
    k, v = torch.from_numpy(k).half(), torch.from_numpy(v).half()
    for s in range(8):
        m = n if s < 2 else 200 * s
        seq, pos = np.full(m, s, np.int32), np.arange(m, dtype=np.int32)
        c.append(*[torch.from_numpy(x).cuda() for x in (seq, pos, tag[:m])], k[:m].cuda(), v[:m].cuda())
        assert o.append(seq, pos, tag[:m], k[:m], v[:m]) == O.OK
    q = torch.ones(8, 2, d, dtype=torch.float16)
    out, _ = c.decode(torch.arange(8, dtype=torch.int32, device="cuda"), q.cuda())
    torch.cuda.synchronize()
    assert c.status() == 0
    ref, _ = o.decode(np.arange(8, dtype=np.int32), q)
    assert Hn.attn_error(out.cpu().numpy(), ref) <= Hn.TOL
