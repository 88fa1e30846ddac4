"""Shared-prefix decode where the running maximum jumps inside a tile of 128
keys: the prefix kernel then rescales weights and sums that it stored a moment
before.  Raw fp16 pages, so that keys and values are exact."""
import numpy as np
import pytest
import torch

from mixed_precision_paged_thinkv_b200.binding import ThinKVCache

from test_gpu_shared import HEADS, _ids

pytestmark = pytest.mark.gpu

# Bound of an output element.  Keys and values are exact, products of fp16 numbers are
# summed in fp32, and a weight is rounded to fp16 twice at most where it is rescaled
# (2^-11 of itself each time; below fp16's normal numbers 2^-25 for a factor down to
# 2^-14, and for a smaller one, taken in two factors of which the second is 1/2 at most,
# 2^-25 / 2 + 2^-25, beside a largest weight of at least 2^6: 1.5 * 2^-31 a key).  The fp32 exponent (scores of up to 4,096, the
# scale is ln 2, so that a score counts powers of two: tokens that carry weight are
# within 40 of the maximum, 40 * 2^-24 of a weight), exp2's own error (2^-22) and the
# fp32 sums stay below 2^-17.  The output is rounded to fp16 once.
LN2 = float(np.log(2.0))
TILE = 128


def _raw_cache(heads, k, v, members):
    """A prompt of raw fp16 tokens in sequence 0 and `members` empty sequences."""
    hq, h, d, g = HEADS[heads]
    n = len(k)
    nb = n // 16 + 2
    c = ThinKVCache(hq, h, d, g, (16, 16, 16), members + 1, nb, (nb, 1, 1))
    for at in range(0, n, 4096):
        m = min(4096, n - at)
        c.append(_ids([0] * m), _ids(range(at, at + m)), torch.zeros(m, dtype=torch.uint8, device="cuda"),
                 k[at:at + m].half().cuda().contiguous(), v[at:at + m].half().cuda().contiguous())
    torch.cuda.synchronize()
    assert c.status() == 0
    # rows enough that the run goes through the prefix kernel, and tiles enough that
    # every CTA of it sums over several
    assert (members - 1) * (n // 16) * h >= 8192
    return c


def _check(c, k, v, q, members, rel=2 * 2.0 ** -11, floor=2.0 ** -24):
    out, _ = c.decode_shared(_ids(range(1, members + 1)), _ids([0] * members), q, softmax_scale=LN2)
    torch.cuda.synchronize()
    assert c.status() == 0
    kd, vd = k.half().cuda().double(), v.half().cuda().double()
    qd = q.double().view(members, c.H, c.Hq // c.H, c.d)
    worst = 0.0
    for i in range(members):
        w = torch.softmax(torch.einsum("thd,hgd->hgt", kd, qd[i]) * LN2, -1)
        o = torch.einsum("hgt,thd->hgd", w, vd)
        wv = torch.einsum("hgt,thd->hgd", w, vd.abs())
        lost = 1.5 * 2.0 ** -31 * torch.einsum("hgt,thd->hgd", (w > 0).double(), vd.abs())
        bound = (rel + 2.0 ** -17) * wv + torch.minimum(lost, wv) + 2.0 ** -11 * o.abs() + floor
        err = (out[i].double().view_as(o) - o).abs()
        worst = max(worst, (err / bound).max().item())
        assert (err <= bound).all(), f"row {i}: {(err / bound).max().item():.2f} of the bound"
    print(f"worst element at {worst:.2f} of its bound")


def _queries(c_heads, members, seed):
    """Rows that follow the rising keys, fall along them, or are indifferent."""
    hq, h, d, g = HEADS[c_heads]
    gen = torch.Generator().manual_seed(seed)
    q = torch.zeros(members, hq, d)
    q[:, :, 0] = torch.tensor([1.0, 1.0, -1.0, 0.0])[torch.randint(0, 4, (members, hq), generator=gen)]
    q[:, :, 1] = torch.rand(members, hq, generator=gen)
    return q.half().cuda()


@pytest.mark.parametrize("heads,members", [("gqa4", 64), ("gqa4", 30), ("gqa8", 32), ("gqa8", 15)])
def test_maximum_jumps_in_every_quarter_of_a_tile(heads, members):
    """32 keys after 32 keys the scores rise by ten powers of two, over 100 tiles:
    several moves in one tile, with products of earlier tiles already summed."""
    hq, h, d, g = HEADS[heads]
    n = 100 * TILE + 5
    gen = torch.Generator().manual_seed(members)
    k = torch.zeros(n, h, d)
    k[:, :, 0] = (10.0 * (torch.arange(n) // 32))[:, None]
    k[:, :, 1] = torch.randint(-2, 3, (n, h), generator=gen).float()
    v = torch.randn(n, h, d, generator=gen)
    c = _raw_cache(heads, k, v, members)
    _check(c, k, v, _queries(heads, members, 1), members)


@pytest.mark.parametrize("quarter", [0, 1, 2, 3])
@pytest.mark.parametrize("heads,members", [("gqa4", 64), ("gqa8", 15)])
def test_maximum_jumps_once_a_tile(heads, members, quarter):
    """One move a tile, in each of its quarters: the weights stored before it, up to
    96 keys a few powers of two below the new maximum, still carry a share of the row."""
    hq, h, d, g = HEADS[heads]
    n = 100 * TILE + 37
    gen = torch.Generator().manual_seed(quarter)
    k = torch.zeros(n, h, d)
    at = torch.arange(n) + (4 - quarter) * 32             # the score rises where this reaches the next tile
    k[:, :, 0] = (10.0 * (at // TILE))[:, None]
    k[:, :, 1] = torch.randint(-1, 2, (n, h), generator=gen).float()
    v = torch.randn(n, h, d, generator=gen)
    # what lies before a move is large, so that it is seen under what follows
    v[at % TILE >= 64] *= 64
    c = _raw_cache(heads, k, v, members)
    _check(c, k, v, _queries(heads, members, 2), members)


@pytest.mark.parametrize("jump", [12.0, 17.5, 20.0])
@pytest.mark.parametrize("heads,members", [("gqa4", 64), ("gqa8", 15)])
def test_weights_before_a_large_jump_count(heads, members, jump):
    """64 keys eight powers of two above the first ones (they stay under the same
    reference), then keys far above them in the same tile, whose values are zero: the
    output is what is left of the 64 keys' weights, to fp16's relative precision."""
    hq, h, d, g = HEADS[heads]
    n = 100 * TILE
    gen = torch.Generator().manual_seed(3)
    k = torch.zeros(n, h, d)
    k[:, :, 0] = -100.0
    k[:32, :, 0], k[32:96, :, 0], k[96:128, :, 0] = 0.0, 8.0, 8.0 + jump
    v = torch.zeros(n, h, d)
    v[32:96] = 500 + 500 * torch.rand(64, h, d, generator=gen)
    c = _raw_cache(heads, k, v, members)
    q = torch.zeros(members, hq, d)
    q[:, :, 0] = 1.0
    _check(c, k, v, q.half().cuda(), members)
