"""Host-side checks of release and fork (no GPU): arguments are refused before
any CUDA call, and the host model of the calls keeps the slot invariants."""
import ctypes as C

import numpy as np
import pytest

import turnover_model as M


@pytest.fixture(scope="module")
def lib():
    from mixed_precision_paged_thinkv_b200 import build, binding
    build.build()
    return binding.lib()


def _cache(**kw):
    from mixed_precision_paged_thinkv_b200 import binding
    a = dict(num_q_heads=32, num_kv_heads=8, head_dim=128, group_size=64, bits=(8, 4, 2),
             max_seqs=16, max_blocks_per_seq=100, pool_pages=(10, 20, 30))
    a.update(kw)
    cs = binding.CacheStruct()
    cs.L = binding.make_layout(**a)
    for name, _ in binding.CacheStruct._fields_[1:]:
        v = getattr(cs, name)
        if isinstance(v, C.Array):
            for i in range(3):
                v[i] = 4096
        else:
            setattr(cs, name, 4096)
    return cs


def test_released_stacks_are_part_of_page_bump(lib):
    cs = _cache()
    assert lib.thinkv_buffer_bytes(C.byref(cs.L), 17) == 4 * (6 + 10 + 20 + 30)


def test_workspace_sizes(lib):
    cs = _cache()
    f = lib.thinkv_turnover_workspace_bytes
    assert f(C.byref(cs.L), -1) == 0 and f(C.byref(cs.L), 17) == 0      # more than max_seqs
    assert f(C.byref(cs.L), 1) >= 256 and f(C.byref(cs.L), 16) >= 16 * 4 * 12
    # the widest layout's size does not overflow 32 bits
    wide = _cache(max_seqs=65536, max_blocks_per_seq=1 << 21)
    assert f(C.byref(wide.L), 65536) > 65536 * 65536 * 12


def test_arguments_are_refused_before_any_launch(lib):
    from mixed_precision_paged_thinkv_b200 import binding
    cs = _cache()
    ok, odd, word = C.c_void_p(4096), C.c_void_p(4098), C.c_void_p(4100)
    need = lib.thinkv_turnover_workspace_bytes(C.byref(cs.L), 4)
    rel, fork = lib.thinkv_release, lib.thinkv_fork
    c = C.byref(cs)
    assert rel(c, None, -1, ok, ok, need, None) == 1
    assert rel(c, None, 17, ok, ok, 1 << 40, None) == 1
    assert rel(c, None, 4, None, ok, need, None) == 1
    assert rel(c, None, 4, odd, ok, need, None) == 1
    assert rel(c, None, 4, ok, word, need, None) == 1
    assert rel(c, None, 4, ok, ok, need - 1, None) == binding.ERR_WORKSPACE
    assert rel(c, None, 4, ok, None, need, None) == binding.ERR_WORKSPACE
    assert rel(c, None, 0, None, None, 0, None) == 0
    assert fork(c, None, -1, ok, ok, ok, need, None) == 1
    assert fork(c, None, 4, None, ok, ok, need, None) == 1
    assert fork(c, None, 4, ok, None, ok, need, None) == 1
    assert fork(c, None, 4, odd, ok, ok, need, None) == 1
    assert fork(c, None, 4, ok, odd, ok, need, None) == 1
    assert fork(c, None, 4, ok, ok, word, need, None) == 1
    assert fork(c, None, 4, ok, ok, ok, need - 1, None) == binding.ERR_WORKSPACE
    assert fork(c, None, 0, None, None, None, 0, None) == 0
    half = binding.TbeStruct(4096, 4096, None)                     # TBE state without `settled`
    assert rel(c, C.byref(half), 4, ok, ok, need, None) == 1
    assert fork(c, C.byref(half), 4, ok, ok, ok, need, None) == 1
    cs.page_bump = 4098
    assert rel(c, None, 4, ok, ok, need, None) == 1


def test_model_round_trip():
    """The host model itself: a fork after a release takes the released pages in
    call order, and releasing the copies gives them back."""
    pool = (4, 4, 4)
    b = {"block_table": np.zeros((3, 4), np.uint64), "num_blocks": np.array([3, 2, 0], np.int32),
         "free_slots": np.zeros((3, 3, 64), np.int32), "free_top": np.zeros((3, 3), np.int32),
         "fifo": np.zeros((3, 3, 64), np.int32), "fifo_head": np.zeros((3, 3), np.int32),
         "fifo_tail": np.zeros((3, 3), np.int32), "live_count": np.zeros(3, np.int32),
         "live_list": np.zeros((3, 4), np.uint64), "live_index": np.full((3, 4), -1, np.int32),
         "num_live": np.zeros(3, np.int32), "page_bump": np.zeros(18, np.int32)}
    for n in "RET":
        b["pool_" + n] = np.arange(4, dtype=np.uint8)[:, None].repeat(8, 1)
        b["slot_pos_" + n] = np.arange(64, dtype=np.int32).reshape(4, 16)
    for s, ents in enumerate([[(0, 0), (1, 0), (0, 1)], [(0, 2), (0, 3)]]):     # (class, page)
        for e, (c, page) in enumerate(ents):
            b["block_table"][s, e] = page | (c << 32) | (1 << 48)
    b["page_bump"][:3] = (4, 1, 0)
    M.release(b, [1], pool)
    assert b["page_bump"][3:6].tolist() == [2, 0, 0] and b["page_bump"][6:8].tolist() == [3, 2]
    M.fork(b, [0], [2], pool)
    assert [int(x) & 0xFFFFFFFF for x in b["block_table"][2, :3]] == [2, 1, 3]
    assert b["page_bump"][:6].tolist() == [4, 2, 0, 0, 0, 0]
    assert b["pool_R"][2].tolist() == [0] * 8 and b["slot_pos_R"][3].tolist() == b["slot_pos_R"][1].tolist()
    M.release(b, [2], pool)
    assert b["page_bump"][3:6].tolist() == [2, 1, 0] and b["page_bump"][6:8].tolist() == [3, 2]


def test_decode_shared_arguments_are_refused_before_any_launch(lib):
    cs = _cache()
    ok, odd, word = C.c_void_p(4096), C.c_void_p(4098), C.c_void_p(4100)
    f, c, big = lib.thinkv_decode_shared, None, 10 ** 9
    c = C.byref(cs)
    for n in (0, -1, 16385):
        assert f(c, n, ok, ok, ok, ok, None, 0, 0.0, ok, big, None) == 1
    for hole in range(4):                              # seq, prefix, q, out
        args = [ok] * 4
        args[hole] = None
        assert f(c, 4, *args, None, 0, 0.0, ok, big, None) == 1
    assert f(c, 4, odd, ok, ok, ok, None, 0, 0.0, ok, big, None) == 1
    assert f(c, 4, ok, odd, ok, ok, None, 0, 0.0, ok, big, None) == 1
    assert f(c, 4, ok, ok, word, ok, None, 0, 0.0, ok, big, None) == 1
    assert f(c, 4, ok, ok, ok, word, None, 0, 0.0, ok, big, None) == 1
    assert f(c, 4, ok, ok, ok, ok, odd, 4, 0.0, ok, big, None) == 1
    assert f(c, 4, ok, ok, ok, ok, None, 0, 0.0, word, big, None) == 1
    for topk in (0, 65):
        assert f(c, 4, ok, ok, ok, ok, ok, topk, 0.0, ok, big, None) == 1
    w = lib.thinkv_decode_shared_workspace_bytes
    assert w(C.byref(cs.L), 0, 0) == 0 and w(C.byref(cs.L), 16385, 0) == 0 and w(C.byref(cs.L), 4, 65) == 0
