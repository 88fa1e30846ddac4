"""Shared-prefix decode over live tokens that hold an infinity or a NaN: the
prefix kernel and the split kernel answer what the definition says (zero + code *
scale, softmax over all tokens), not-a-numbers and infinities included, and the
heads without such a token stay as exact as ever."""
import numpy as np
import pytest
import torch

from mixed_precision_paged_thinkv_b200.binding import ThinKVCache

from test_gpu_shared import BITS, HEADS, Exact, _ids

pytestmark = pytest.mark.gpu

MEMBERS, TOKENS, BAD = 40, 3000, 1234
ALL = {**BITS, "raws": ((16, 16, 16), (0, 0, 0))}


def _cache(heads, bits, tag, kv, value, channel=5):
    """A prompt whose token BAD, of class `tag`, has `value` in one channel of the
    keys (kv 0) or the values (kv 1) of the last kv-head."""
    hq, h, d, g = HEADS[heads]
    b, fmt = ALL[bits]
    c = ThinKVCache(hq, h, d, g, b, MEMBERS + 1, 200, (300, 300, 300), fmt=fmt)
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(2, TOKENS, h, d, generator=gen).half()
    x[kv, BAD, h - 1, channel] = value
    tags = (torch.arange(TOKENS) // 5 % 3).to(torch.uint8)
    tags[BAD] = tag
    x = x.cuda()
    c.append(_ids([0] * TOKENS), _ids(range(TOKENS)), tags.cuda(), x[0], x[1])
    seq = list(range(1, MEMBERS + 1))
    y = torch.randn(2, MEMBERS, h, d, generator=gen).half().cuda()
    c.append(_ids(seq), _ids([TOKENS] * MEMBERS), torch.zeros(MEMBERS, dtype=torch.uint8, device="cuda"), y[0], y[1])
    torch.cuda.synchronize()
    assert c.status() == 0
    return c, seq


def _same(out, ref, bound, what):
    got = out.double().cpu().numpy()
    odd = ~np.isfinite(ref)
    assert np.array_equal(np.isfinite(got), ~odd), \
        f"{what}: {(np.isfinite(got) & odd).sum()} of {odd.sum()} not-finite elements came out finite, " \
        f"{(~np.isfinite(got) & ~odd).sum()} the other way round"
    assert np.array_equal(got[odd], ref[odd], equal_nan=True), what
    err = np.abs(got - ref)[~odd]
    assert (err <= bound[~odd]).all(), what


def _reference(c, seq, q):
    """Definition, and the bound of its finite elements.  A key whose score is -inf has
    weight 0 where the output is finite: its head's bound is that of the other tokens."""
    exact = Exact(c)
    with np.errstate(invalid="ignore"):
        ref, _, bound = exact.rows(seq, [0] * len(seq), q)
        keep = np.isfinite(exact.kept[0][0]).all(axis=(1, 2))
        if not keep.all():
            exact.kept[0] = [x[keep] for x in exact.kept[0]]
            own = c.Hq - c.Hq // c.H
            bound[:, own:] = exact.rows(seq, [0] * len(seq), q)[2][:, own:]
    assert np.isfinite(ref[:, :c.Hq - c.Hq // c.H]).all()
    return ref, bound


WHERE = pytest.mark.parametrize("heads,bits,tag", [
    ("gqa4", "842", 0), ("gqa4", "842", 1), ("gqa4", "842", 2), ("gqa8", "842", 1), ("gqa4", "float", 0),
    ("gqa4", "float", 1), ("gqa4", "float", 2), ("mha", "two", 1), ("gqa8", "fp4", 0), ("gqa4", "raws", 0),
    ("gqa8", "raws", 2)])


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("kv", [0, 1])
@WHERE
def test_rows_alone(heads, bits, tag, kv, value):
    """The split kernel: rows with the prefix to themselves, and decode() of a copy."""
    c, seq = _cache(heads, bits, tag, kv, value)
    seq = seq[:3]
    q = np.random.default_rng(3).standard_normal((3, c.Hq, c.d)).astype(np.float16)
    qd = torch.from_numpy(q).cuda()
    ref, bound = _reference(c, seq, q)
    out = torch.cat([c.decode_shared(_ids([s]), _ids([0]), qd[i:i + 1])[0] for i, s in enumerate(seq)])
    torch.cuda.synchronize()
    _same(out, ref, bound, "rows alone")
    c.release(_ids(range(1, MEMBERS + 1)))
    c.fork(_ids([0]), _ids([1]))
    ref, bound = _reference(c, [2] * 3, q)
    out = torch.cat([c.decode(_ids([1]), qd[i:i + 1])[0] for i in range(3)])
    torch.cuda.synchronize()
    assert c.status() == 0
    _same(out, ref, bound, "decode")


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("kv", [0, 1])
@WHERE
def test_rows_of_a_run(heads, bits, tag, kv, value):
    """The prefix kernel: rows that read the prefix together."""
    c, seq = _cache(heads, bits, tag, kv, value)
    assert (MEMBERS - 1) * c.snapshot()["num_live"][0] * c.H >= 8192
    q = np.random.default_rng(4).standard_normal((MEMBERS, c.Hq, c.d)).astype(np.float16)
    ref, bound = _reference(c, seq, q)
    out = c.decode_shared(_ids(seq), _ids([0] * MEMBERS), torch.from_numpy(q).cuda())[0]
    torch.cuda.synchronize()
    assert c.status() == 0
    _same(out, ref, bound, "rows of a run")


@pytest.mark.parametrize("heads", ["gqa4", "gqa8"])
@pytest.mark.parametrize("bad", [16, 700])
def test_keys_without_weight(heads, bad):
    """Whole pages and tiles of raw keys whose scores are -inf, first in the list: a
    row's maximum is -inf until its first finite score, and their weight is 0."""
    hq, h, d, g = HEADS[heads]
    c = ThinKVCache(hq, h, d, g, (16, 16, 16), MEMBERS + 1, 200, (300, 1, 1))
    gen = torch.Generator().manual_seed(bad)
    x = torch.randn(2, TOKENS, h, d, generator=gen).half()
    x[0, :bad, :, 5] = np.inf
    x = x.cuda()
    c.append(_ids([0] * TOKENS), _ids(range(TOKENS)), torch.zeros(TOKENS, dtype=torch.uint8, device="cuda"), x[0], x[1])
    seq = list(range(1, MEMBERS + 1))
    q = np.random.default_rng(bad).standard_normal((MEMBERS, hq, d)).astype(np.float16)
    q[:, :, 5] = -np.abs(q[:, :, 5]) - np.float16(0.1)
    qd = torch.from_numpy(q).cuda()
    exact = Exact(c)
    exact.kept[0] = [y[bad:] for y in exact.tokens(0)]
    ref, _, bound = exact.rows(seq, [0] * MEMBERS, q)
    run = c.decode_shared(_ids(seq), _ids([0] * MEMBERS), qd)[0]
    alone = torch.cat([c.decode_shared(_ids([1]), _ids([0]), qd[i:i + 1])[0] for i in range(6)])
    one = torch.cat([c.decode(_ids([0]), qd[i:i + 1])[0] for i in range(6)])
    many = c.decode(_ids([0] * MEMBERS), qd)[0]
    torch.cuda.synchronize()
    assert c.status() == 0
    _same(run, ref, bound, "rows of a run")
    _same(alone, ref[:6], bound[:6], "rows alone")
    _same(one, ref[:6], bound[:6], "decode")
    _same(many, ref, bound, "decode of many rows")
    with np.errstate(invalid="ignore"):
        odd, _, _ = Exact(c).rows([1], [0], -q[:1])      # scores of +inf
    out = c.decode_shared(_ids([1]), _ids([0]), -qd[:1])[0]
    assert np.isnan(odd).all() and torch.isnan(out).all()
