"""A cache taken over from existing buffers: what is not usable is refused when
the cache is made (no GPU needed)."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def binding():
    from mixed_precision_paged_thinkv_b200 import build, binding
    build.build()
    return binding


ARGS = dict(num_q_heads=4, num_kv_heads=2, head_dim=64, group_size=32, bits=(8, 4, 2), max_seqs=3,
            max_blocks_per_seq=5, pool_pages=(7, 0, 4))


def _buffers(binding, **kw):
    L = binding.make_layout(**{**ARGS, **kw}, fmt=(0, 0, 0))
    lib = binding.lib()
    out = {name: torch.zeros(lib.thinkv_buffer_bytes(C.byref(L), i), dtype=torch.uint8)
           for i, name in enumerate(binding.BUFFERS)}
    out.update({name: torch.zeros(lib.thinkv_tbe_buffer_bytes(C.byref(L), i), dtype=torch.uint8)
                for i, name in enumerate(binding.TBE_BUFFERS)})
    return out


def _make(binding, buffers, **kw):
    return binding.ThinKVCache(**ARGS, device="cpu", buffers=buffers, **kw)


def test_taken_over_as_it_stands(binding):
    b = _buffers(binding)
    b["block_table"].fill_(3)
    c = _make(binding, b, tbe=True)
    assert c.buf["block_table"].data_ptr() == b["block_table"].data_ptr() and (b["block_table"] == 3).all()
    assert c.cs.block_table == b["block_table"].data_ptr() and c.tbe.seg == b["seg"].data_ptr()


def test_missing_short_and_strided_buffers(binding):
    for name in ("pool_R", "slot_pos_T", "free_slots", "page_bump", "status", "nseg"):
        for bad in (None, torch.zeros(3, dtype=torch.uint8), _buffers(binding)[name].repeat_interleave(2)[::2]):
            b = _buffers(binding)
            b[name] = bad
            with pytest.raises(binding.ThinkvError):
                _make(binding, b, tbe=True)


@pytest.mark.parametrize("name,align", [("pool_R", 16), ("seg", 16), ("block_table", 8), ("live_list", 8),
                                        ("slot_pos_T", 4), ("free_top", 4), ("status", 4), ("settled", 4)])
def test_alignment(binding, name, align):
    for off, good in ((align // 2, False), (align, True)):
        b = _buffers(binding)
        n = b[name].numel()
        room = torch.zeros(n + 64, dtype=torch.uint8)
        at = -room.data_ptr() % 32 + off
        b[name] = room[at:at + n]
        if good:
            assert _make(binding, b, tbe=True).cs.L.max_seqs == 3
        else:
            with pytest.raises(binding.ThinkvError):
                _make(binding, b, tbe=True)


def test_device(binding):
    b = _buffers(binding)
    b["fifo"] = torch.empty(b["fifo"].numel(), dtype=torch.uint8, device="meta")
    with pytest.raises(binding.ThinkvError):
        _make(binding, b)
    with pytest.raises(binding.ThinkvError):             # all elsewhere
        binding.ThinKVCache(**ARGS, device="cuda", buffers=_buffers(binding))


class _On:
    """A tensor that says it is on another device (one GPU here, or none)."""

    def __init__(self, t, device):
        self.t, self.device = t, torch.device(device)

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_buffers_of_two_devices(binding):
    for odd in ("block_table", "status", "settled"):
        b = {name: _On(t, "cuda:1" if name == odd else "cuda:0") for name, t in _buffers(binding).items()}
        with pytest.raises(binding.ThinkvError):
            binding.ThinKVCache(**ARGS, device="cuda", buffers=b, tbe=True)


def test_a_class_without_pages(binding):
    """Whatever is given for its pool is not taken."""
    b = _buffers(binding)
    b["pool_E"] = torch.zeros(33, dtype=torch.uint8)[1:]
    c = _make(binding, b)
    assert c.buf["pool_E"] is None and not c.cs.pool[1] and not c.cs.slot_pos[1]
