"""Argument checks of the cache operators beside decode, without a GPU: every
refusal is a status, given before anything is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.build import build
    build()
    return _lib


def _desc(lib, **kw):
    d = dict(num_kv_heads=8, head_dim=128, block_size=16, num_blocks=4, k_bits=8, v_bits=8,
             k_codes=0x1000, v_codes=0x2000, meta=0x3000)
    d.update(kw)
    return lib.CacheDesc(**d)


WINDOW = dict(window=16, window_batch=1, k_window=0xD000, v_window=0xE000)


@pytest.mark.parametrize("cache,rope,kw,status", [
    (dict(head_dim=64), {}, {}, 2),
    ({}, dict(rotary_dim=0), {}, 2), ({}, dict(rotary_dim=12), {}, 2), ({}, dict(rotary_dim=136), {}, 2),
    ({}, dict(interleaved=2), {}, 1), ({}, dict(max_pos=0), {}, 1), ({}, dict(table=None), {}, 1),
    ({}, dict(table=0x4008), {}, 3),
    ({}, {}, dict(n=-1), 1), ({}, {}, dict(q_heads=-1), 1), ({}, {}, dict(mode=3), 1),
    # queries need an output and heads; keys need values; something has to be given
    ({}, {}, dict(q_out=None), 1), ({}, {}, dict(q_heads=0), 1), ({}, {}, dict(v_new=None), 1),
    ({}, {}, dict(q=None, q_out=None, q_heads=0, k_new=None, v_new=None), 1),
    # row strides: a multiple of 4, not shorter than a row; in place only for contiguous rows
    ({}, {}, dict(q_stride=32 * 128 - 4), 1), ({}, {}, dict(q_stride=32 * 128 + 2), 3),
    ({}, {}, dict(k_stride=8 * 128 - 4), 1), ({}, {}, dict(v_stride=8 * 128 + 1), 3),
    ({}, {}, dict(q_out=0x5000, q_stride=48 * 128), 1),
    ({}, {}, dict(q=0x5004), 3), ({}, {}, dict(k_new=0x7004), 3), ({}, {}, dict(q_out=0x6002), 3),
    # the write's own arguments, as kvq_append has them
    ({}, {}, dict(seq_idx=None), 1), ({}, {}, dict(pos=None), 1), ({}, {}, dict(block_table=None), 1),
    ({}, {}, dict(batch=0), 1), ({}, {}, dict(mbps=0), 1), ({}, {}, dict(mode=1), 1), ({}, {}, dict(mode=2), 1),
    (dict(k_bits=2, v_bits=2, **WINDOW), {}, dict(mode=2), 2),
    # queries only still need positions
    ({}, {}, dict(k_new=None, v_new=None, rope_pos=None, pos=None), 1),
    # more vectors than a grid holds
    ({}, {}, dict(n=2 ** 30), 2),
    # no rows: nothing to do, nothing read
    ({}, dict(table=None), dict(n=0, q=None, k_new=None), 0),
])
def test_rope_append_refusals(lib, cache, rope, kw, status):
    r = dict(rotary_dim=128, interleaved=0, max_pos=64, table=0x4000)
    r.update(rope)
    a = dict(q=0x5000, q_heads=32, q_stride=0, q_out=0x6000, k_new=0x7000, k_stride=0, v_new=0x8000, v_stride=0, n=1,
             rope_pos=0x9000, seq_idx=0xA000, pos=0xB000, mode=0, block_table=0xC000, batch=1, mbps=1)
    a.update(kw)
    st = lib.load().kvq_rope_append(ctypes.byref(_desc(lib, **cache)), ctypes.byref(lib.RopeDesc(**r)), a["q"],
                                    a["q_heads"], a["q_stride"], a["q_out"], a["k_new"], a["k_stride"], a["v_new"],
                                    a["v_stride"], a["n"], a["rope_pos"], a["seq_idx"], a["pos"], a["mode"],
                                    a["block_table"], a["batch"], a["mbps"], None, None)
    assert st == status


@pytest.mark.parametrize("freqs,rotary,max_pos,table,status", [
    (dict(base=1.0), 128, 8, 0x4000, 1), (dict(base=float("nan")), 128, 8, 0x4000, 1),
    (dict(base=float("inf")), 128, 8, 0x4000, 1), (dict(scaling=4), 128, 8, 0x4000, 1),
    (dict(scaling=1, factor=0.5), 128, 8, 0x4000, 1), (dict(scaling=2, factor=float("nan")), 128, 8, 0x4000, 1),
    (dict(scaling=3, factor=8.0), 128, 8, 0x4000, 1),
    (dict(scaling=3, factor=8.0, original_len=8192, low_turns=4, high_turns=4), 128, 8, 0x4000, 1),
    (dict(amplitude=-1.0), 128, 8, 0x4000, 1), ({}, 10, 8, 0x4000, 2), ({}, 128, 0, 0x4000, 1),
    ({}, 128, 8, None, 1), ({}, 128, 8, 0x4004, 3),
])
def test_rope_table_refusals(lib, freqs, rotary, max_pos, table, status):
    f = dict(base=10000.0, scaling=0, factor=1.0, amplitude=1.0)
    f.update(freqs)
    assert lib.load().kvq_rope_table(ctypes.byref(lib.RopeFreqs(**f)), rotary, max_pos, table, None) == status


def test_null_descriptors_are_refused(lib):
    so = lib.load()
    assert so.kvq_rope_table(None, 128, 8, 0x4000, None) == lib.KVQ_ERR_INVALID_ARG
    assert so.kvq_rope_append(ctypes.byref(_desc(lib)), None, 0x5000, 32, 0, 0x6000, 0x7000, 0, 0x8000, 0, 1, 0x9000,
                              0xA000, 0xB000, 0, 0xC000, 1, 1, None, None) == lib.KVQ_ERR_INVALID_ARG


@pytest.mark.parametrize("cache,kw,status", [
    (dict(block_size=32), {}, 2), ({}, dict(batch=-1), 1), ({}, dict(batch=5000), 2), ({}, dict(q_heads=12), 1),
    ({}, dict(q_heads=128), 2), ({}, dict(q=None), 1), ({}, dict(lse=None), 1), ({}, dict(lens=None), 1),
    ({}, dict(table=None), 1), ({}, dict(mass=None), 1), ({}, dict(mbps=0), 1), ({}, dict(stride=0), 1),
    ({}, dict(stride=18), 3), ({}, dict(mass=0x9004), 3), ({}, dict(q=0x5008), 3), ({}, dict(decay=float("nan")), 1),
    ({}, dict(decay=float("inf")), 1), ({}, dict(batch=0, q=None), 0),
    (dict(window=16, window_batch=1, k_window=0xD000, v_window=0xE000), dict(batch=2), 1),
])
def test_attn_mass_refusals(lib, cache, kw, status):
    a = dict(q=0x5000, batch=1, q_heads=8, lse=0x6000, lens=0x7000, table=0x8000, mbps=1, mass=0x9000, stride=16,
             decay=1.0)
    a.update(kw)
    st = lib.load().kvq_attn_mass(ctypes.byref(_desc(lib, **cache)), a["q"], a["batch"], a["q_heads"], a["lse"],
                                  a["lens"], a["table"], a["mbps"], a["mass"], a["stride"], a["decay"], None, None)
    assert st == status


@pytest.mark.parametrize("cache,kw,status", [
    # a token cannot leave a 2-bit block's scale
    (dict(k_bits=2, v_bits=2), {}, 2), (dict(k_codes=None), {}, 1),
    ({}, dict(batch=-1), 1), ({}, dict(batch=5000), 2), ({}, dict(mass=None), 1), ({}, dict(lens=None), 1),
    ({}, dict(keep=None), 1), ({}, dict(table=None), 1), ({}, dict(new_lens=None), 1), ({}, dict(source=None), 1),
    ({}, dict(stride=0), 1), ({}, dict(mbps=0), 1), ({}, dict(first=-1), 1), ({}, dict(recent=-1), 1),
    # the lengths are read by both launches
    ({}, dict(new_lens=0x6000), 1), ({}, dict(new_lens=0x7000), 1),
    # positions in need positions out and the next position
    ({}, dict(new_lens=0xB000, next=0xB000), 1), ({}, dict(source=0xA000, pos=0xA000, pos_out=0xB000, next=0xE000), 1),
    ({}, dict(source=0xB000, pos=0xA000, pos_out=0xB000, next=0xE000), 1), ({}, dict(stride=(1 << 30) + 1), 1),
    ({}, dict(pos=0xA000), 1), ({}, dict(pos=0xA000, pos_out=0xA000), 1), ({}, dict(pos=0xA000, next=0xB000), 1),
    ({}, dict(batch=0, mass=None), 0),
])
def test_evict_refusals(lib, cache, kw, status):
    a = dict(mass=0x5000, mass_out=None, stride=16, lens=0x6000, keep=0x7000, first=0, recent=0, pos=None,
             pos_out=None, next=None, table=0x8000, batch=1, mbps=1, new_lens=0x9000, source=0xC000)
    a.update(kw)
    st = lib.load().kvq_evict(ctypes.byref(_desc(lib, **cache)), a["mass"], a["mass_out"], a["stride"], a["lens"],
                              a["keep"], a["first"], a["recent"], a["pos"], a["pos_out"], a["next"], a["table"],
                              a["batch"], a["mbps"], a["new_lens"], a["source"], None, None)
    assert st == status


@pytest.mark.parametrize("cache,kw,status", [
    (dict(head_dim=64), {}, 2), ({}, dict(batch=-1), 1), ({}, dict(batch=5000), 2), ({}, dict(q_heads=12), 1),
    ({}, dict(q_heads=128), 2), ({}, dict(groups=0), 1), ({}, dict(groups=257), 2), ({}, dict(q=None), 1),
    ({}, dict(lens=None), 1), ({}, dict(table=None), 1), ({}, dict(mbps=0), 1), ({}, dict(start=None), 1),
    ({}, dict(blocks=None), 1), ({}, dict(out=None), 1), ({}, dict(q=0x5008), 3), ({}, dict(out=0xA008), 3),
    ({}, dict(ws=None), 4), ({}, dict(ws=0xB008), 3), ({}, dict(batch=0, q=None, ws=None), 0),
])
def test_decode_shared_refusals(lib, cache, kw, status):
    a = dict(q=0x5000, batch=2, q_heads=8, lens=0x6000, table=0x7000, mbps=4, groups=1, start=0x8000, blocks=0x9000,
             out=0xA000, ws=0xB000, nbytes=1 << 30)
    a.update(kw)
    st = lib.load().kvq_decode_shared(ctypes.byref(_desc(lib, **cache)), a["q"], a["batch"], a["q_heads"], a["lens"],
                                      a["table"], a["mbps"], a["groups"], a["start"], a["blocks"], a["out"], 0, None,
                                      a["ws"], a["nbytes"], None, None)
    assert st == status
    import ctypes as c
    size = c.c_size_t(0)
    if "groups" in kw or "batch" in kw and kw["batch"] != 0:
        assert lib.load().kvq_decode_shared_workspace_size(ctypes.byref(_desc(lib)), a["batch"], a["q_heads"],
                                                           a["groups"], c.byref(size)) == status
