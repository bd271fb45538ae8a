"""Argument checks of sliding-window serving without a GPU: normed rotary write, attention with sinks, pages.  The
library's refusals are statuses given before any launch; the binding's are seen with a recorder in the library's place."""
import ctypes

import pytest

from test_binding_host import Recorder, _i, refused
from test_ops_host import WINDOW, _desc, lib as built  # noqa: F401  (a fixture)

torch = pytest.importorskip("torch")


@pytest.fixture
def rec(monkeypatch):
    from quantized_kv_cache_07_gb300 import _lib
    _lib._need_torch()
    so = Recorder()
    monkeypatch.setattr(_lib, "_current_device", lambda: -1)
    monkeypatch.setattr(_lib, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(_lib, "load", lambda: so)
    monkeypatch.setattr(_lib, "status_string", str)
    monkeypatch.setattr(_lib, "recorder", so, raising=False)
    return _lib


# ------------------------------------------------------------------ the library

@pytest.mark.parametrize("norm,kw,status", [
    (None, {}, 1), (dict(eps=0.0), {}, 1), (dict(eps=-1e-6), {}, 1), (dict(eps=float("nan")), {}, 1),
    (dict(eps=float("inf")), {}, 1), (dict(eps=1e-13), {}, 1), (dict(eps=2.0), {}, 1), (dict(per_head=2), {}, 1),
    (dict(per_head=-1), {}, 1), (dict(q_weight=0x4008), {}, 3), (dict(k_weight=0x4004), {}, 3),
    # what kvq_rope_append refuses
    ({}, dict(q_out=None), 1), ({}, dict(k_stride=8 * 128 - 4), 1), ({}, dict(mode=1), 1), ({}, dict(rope_pos=None, pos=None), 1),
    ({}, dict(n=0), 0), (dict(q_weight=None, k_weight=None), dict(n=0), 0),
])
def test_norm_rope_append_refusals(built, norm, kw, status):
    a = dict(q=0x5000, q_heads=32, q_stride=0, q_out=0x6000, k_new=0x7000, k_stride=0, v_new=0x8000, v_stride=0, n=1,
             rope_pos=0x9000, seq_idx=0xA000, pos=0xB000, mode=0, block_table=0xC000, batch=1, mbps=1)
    a.update(kw)
    d = None
    if norm is not None:
        d = ctypes.byref(built.NormDesc(**dict(dict(eps=1e-6, per_head=0, q_weight=0x4000, k_weight=0x4100), **norm)))
    rope = built.RopeDesc(rotary_dim=128, interleaved=0, max_pos=64, table=0x4000)
    assert built.load().kvq_norm_rope_append(ctypes.byref(_desc(built)), ctypes.byref(rope), d, *a.values(), None,
                                             None) == status


@pytest.mark.parametrize("cache,kw,status", [
    ({}, dict(sinks=-1), 1), ({}, dict(span=0), 1), ({}, dict(span=-5), 1), (WINDOW, dict(span=15), 2),
    (dict(head_dim=64), {}, 2), ({}, dict(q_heads=12), 1), ({}, dict(q_heads=128), 2), ({}, dict(q=None), 1),
    ({}, dict(table=None), 1), ({}, dict(out=0xA008), 3), ({}, dict(ctas=-1), 1), ({}, dict(ws=None), 4),
    ({}, dict(nbytes=64), 4), ({}, dict(batch=0, q=None), 0),
])
def test_decode_sinks_refusals(built, cache, kw, status):
    a = dict(q=0x5000, batch=1, q_heads=8, lens=0x6000, table=0x7000, mbps=4, sinks=4, span=64, out=0xA000, fp32=0, lse=None,
             ws=0xB000, nbytes=1 << 30, ctas=5)
    a.update(kw)
    assert built.load().kvq_decode_sinks(ctypes.byref(_desc(built, **cache)), *a.values(), None, None) == status


@pytest.mark.parametrize("cache,kw,status", [
    ({}, dict(sinks=-1), 1), ({}, dict(span=0), 1), (WINDOW, {}, 2), ({}, dict(n=5000), 2), ({}, dict(v_new=0x9000), 1),
    ({}, dict(ctas=-3), 1), (dict(q_bits=32), dict(ctas=-2), 2),
    (dict(k_bits=16, v_bits=16, meta=None), dict(ctas=-2), 2), (dict(k_bits=16, v_bits=16, meta=None), dict(ctas=-1), 2),
    ({}, dict(q=0x5004, ctas=-2), 3), ({}, dict(batch=0), 1), ({}, dict(n=0, q=None), 0),
])
def test_prefill_sinks_refusals(built, cache, kw, status):
    a = dict(q=0x5000, n=4, q_heads=8, seq=0x6000, pos=0x6100, k_new=None, v_new=None, table=0x7000, batch=1, mbps=4, sinks=4,
             span=64, out=0xA000, fp32=0, lse=None, ws=None, nbytes=0, ctas=-1)
    a.update(kw)
    assert built.load().kvq_prefill_sinks(ctypes.byref(_desc(built, **cache)), *a.values(), None, None) == status


def test_units_are_of_prefill_sinks_alone(built):
    so, d, size = built.load(), ctypes.byref(_desc(built)), ctypes.c_size_t(7)
    assert so.kvq_prefill(d, 0x5000, 4, 8, 0x6000, 0x6100, None, None, 0x7000, 1, 4, 0xA000, 0, None, None, 0, -2, None,
                          None) == built.KVQ_ERR_INVALID_ARG
    assert so.kvq_prefill_workspace_size(d, 4, 8, -2, ctypes.byref(size)) == 0 and size.value == 0
    q32 = ctypes.byref(_desc(built, q_bits=32))
    assert so.kvq_prefill_workspace_size(q32, 4, 8, -2, ctypes.byref(size)) == built.KVQ_ERR_UNSUPPORTED


PAGES = dict(refs=0x1000, num_blocks=64, table=0x2000, lens=0x3000, parent=None, batch=2, mbps=8, window=0, room=1,
             rooms=None, sinks=0, span=0, refs_out=0x1000, table_out=0x4000, lens_out=0x5000, parent_out=None,
             copies=0x6000, num=0x7000, ws=0x8000, nbytes=1 << 20)


@pytest.mark.parametrize("kw,status", [
    (dict(num_blocks=0), 1), (dict(num_blocks=(1 << 30) + 1), 2), (dict(batch=0), 1), (dict(batch=4097), 2), (dict(mbps=0), 1),
    (dict(window=-16), 1), (dict(window=24), 2), (dict(window=144), 2), (dict(room=-1), 1), (dict(sinks=-1), 1),
    (dict(span=-1), 1), (dict(window=64, span=63), 2), (dict(batch=4096, mbps=1 << 20), 2),
    (dict(refs=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(refs_out=None), 1), (dict(table_out=None), 1),
    (dict(lens_out=None), 1), (dict(copies=None), 1), (dict(num=None), 1), (dict(copies=0x6004), 3),
    # rows read one another's entries: not in place
    (dict(table_out=0x2000), 1), (dict(lens_out=0x3000), 1), (dict(parent=0x9000, parent_out=0x9000), 1),
    (dict(ws=None), 4), (dict(nbytes=100), 4), (dict(ws=0x8008), 3),
])
def test_pages_update_refusals(built, kw, status):
    assert built.load().kvq_pages_update(*dict(PAGES, **kw).values(), None, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(num_blocks=0), 1), (dict(num_blocks=(1 << 30) + 1), 2), (dict(batch=-1), 1), (dict(mbps=0), 1), (dict(refs=None), 1),
    (dict(refs_out=None), 1), (dict(table=None), 1), (dict(table_out=None), 1), (dict(moves=None), 1), (dict(counts=None), 1),
    (dict(moves=0x6004), 3), (dict(ws=None), 4), (dict(nbytes=100), 4), (dict(ws=0x8008), 3),
])
def test_pages_compact_refusals(built, kw, status):
    a = dict(refs=0x1000, num_blocks=64, table=0x2000, batch=2, mbps=8, refs_out=0x1000, table_out=0x2000, moves=0x6000,
             counts=0x7000, ws=0x8000, nbytes=1 << 20)
    a.update(kw)
    assert built.load().kvq_pages_compact(*a.values(), None, None) == status


def test_copies_and_rings_refusals(built):
    so = built.load()

    def arr(*kws):
        return (built.CacheDesc * len(kws))(*[_desc(built, **kw) for kw in kws])
    one = arr({})
    copy = lambda c, n, copies=0x1000, num=0x2000, most=4: so.kvq_copy_blocks(c, n, copies, num, most, None, None)
    assert copy(one, -1) == 1 and copy(None, 1) == 1 and copy(one, 1, copies=None) == 1 and copy(one, 1, num=None) == 1
    assert copy(one, 1, most=-1) == 1 and copy(one, 1, copies=0x1004) == 3
    assert copy(arr({}, dict(head_dim=64)), 2) == 2 and copy(arr({}, dict(meta=None)), 2) == 1
    assert copy(one, 0) == 0 and copy(one, 1, copies=None, most=0) == 0
    assert copy(arr(dict(num_blocks=1 << 29)), 1) == 2                       # 8 heads: blocks of a pool beyond 32 bits
    fork = lambda c, n, parent=0x1000, batch=1: so.kvq_fork_windows(c, n, parent, batch, None, None)
    ring = arr(WINDOW)
    assert fork(ring, -1) == 1 and fork(None, 1) == 1 and fork(ring, 1, parent=None) == 1 and fork(ring, 1, batch=-1) == 1
    assert fork(ring, 1, batch=4097) == 2 and fork(one, 1) == 1 and fork(ring, 1, batch=2) == 1
    assert fork(arr(WINDOW, {}), 2) == 1 and fork(ring, 1, batch=0, parent=None) == 0 and fork(ring, 0) == 0
    size = ctypes.c_size_t(0)
    assert so.kvq_pages_workspace_size(0, ctypes.byref(size)) == 1 and so.kvq_pages_workspace_size(5, None) == 1
    assert so.kvq_pages_workspace_size(1000, ctypes.byref(size)) == 0 and size.value >= 4000


def test_constants_of_the_header(built):
    from test_abi_host import header_constants
    h = header_constants()
    assert built.PREFILL_UNITS == h["KVQ_PREFILL_UNITS"] and built.KVQ_DEVERR_NO_BLOCKS == h["KVQ_DEVERR_NO_BLOCKS"]


# ------------------------------------------------------------------ the binding

def sinks_call(rec, batch=2, **kw):
    a = dict(q=torch.zeros(batch, 4, 128, dtype=torch.bfloat16), batch=batch, q_heads=4, seq_lens=_i(*[3] * batch),
             block_table=torch.zeros(batch, 3, dtype=torch.int32), max_blocks_per_seq=3, sinks=4, span=20,
             out=torch.empty(batch, 4, 128, dtype=torch.bfloat16), workspace=torch.empty(512, dtype=torch.uint8),
             workspace_bytes=512)
    a.update(kw)
    rec.kvq_decode_sinks(rec.CacheDesc(), **a)
    return rec.recorder.calls[-1]


def chunk_call(rec, n=5, **kw):
    x = torch.zeros(n, 4, 128, dtype=torch.bfloat16)
    a = dict(q=x, q_heads=4, seq_idx=_i(*[0] * n), pos=_i(*range(n)), block_table=torch.zeros(2, 3, dtype=torch.int32),
             batch=2, max_blocks_per_seq=3, sinks=4, span=20, out=torch.empty_like(x))
    a.update(kw)
    rec.kvq_prefill_sinks(rec.CacheDesc(num_kv_heads=2), **a)
    return rec.recorder.calls[-1]


def update_call(rec, batch=2, width=3, blocks=9, **kw):
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)
    a = dict(refs=z(blocks), block_table=z(batch, width), seq_lens=z(batch), refs_out=z(blocks), table_out=z(batch, width),
             lens_out=z(batch), copies=z(batch, 2), num_copies=z(1), parent=z(batch), room=1,
             workspace=torch.zeros(64, dtype=torch.uint8))
    a.update(kw)
    rec.kvq_pages_update(**a)
    return rec.recorder.calls[-1]


def compact_call(rec, blocks=9, **kw):
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)
    a = dict(refs=z(blocks), block_table=z(2, 3), refs_out=z(blocks), table_out=z(2, 3), moves=z(blocks // 2, 2), counts=z(2),
             workspace=torch.zeros(64, dtype=torch.uint8))
    a.update(kw)
    rec.kvq_pages_compact(**a)
    return rec.recorder.calls[-1]


def copy_call(rec, **kw):
    a = dict(caches=rec.CacheList([rec.CacheDesc()]), copies=torch.zeros(4, 2, dtype=torch.int32), num_copies=_i(0))
    a.update(kw)
    rec.kvq_copy_blocks(**a)
    return rec.recorder.calls[-1]


def fork_call(rec, **kw):
    a = dict(caches=rec.CacheList([rec.CacheDesc()]), parent=_i(0, 1, 1), batch=3)
    a.update(kw)
    rec.kvq_fork_windows(**a)
    return rec.recorder.calls[-1]


Z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype)


@pytest.mark.parametrize("call,kw", [
    (sinks_call, dict(q=Z(2, 4, 128, dtype=torch.float16))), (sinks_call, dict(q=Z(1, 4, 128, dtype=torch.bfloat16))),
    (sinks_call, dict(seq_lens=Z(1))), (sinks_call, dict(block_table=Z(2, 2))), (sinks_call, dict(block_table=Z(3, 2).t())),
    (sinks_call, dict(workspace_bytes=513)), (sinks_call, dict(lse=Z(2, 4))), (sinks_call, dict(out=Z(2, 4, 64, dtype=torch.bfloat16))),
    (chunk_call, dict(seq_idx=_i(0, 0))), (chunk_call, dict(k_new=Z(5, 4, 128, dtype=torch.bfloat16))),
    (chunk_call, dict(block_table=Z(1, 3))), (chunk_call, dict(q=Z(5, 8, 128, dtype=torch.bfloat16)[:, ::2])),
    (chunk_call, dict(out=Z(4, 4, 128, dtype=torch.bfloat16))),
    (update_call, dict(refs_out=Z(8))), (update_call, dict(seq_lens=Z(3))), (update_call, dict(parent=Z(1))),
    (update_call, dict(table_out=Z(2, 4))), (update_call, dict(lens_out=Z(2, dtype=torch.int64))), (update_call, dict(copies=Z(1, 2))),
    (update_call, dict(num_copies=Z(0))), (update_call, dict(room=Z(3))), (update_call, dict(parent_out=Z(3))),
    (update_call, dict(block_table=Z(3, 2).t())), (update_call, dict(workspace=Z(64))),
    (compact_call, dict(moves=Z(3, 2))), (compact_call, dict(counts=Z(1))), (compact_call, dict(refs_out=Z(10))),
    (compact_call, dict(table_out=Z(3, 2))),
    (copy_call, dict(copies=Z(4, 2, dtype=torch.int64))), (copy_call, dict(num_copies=Z(0))), (copy_call, dict(copies=Z(2, 4).t())),
    (fork_call, dict(batch=4)), (fork_call, dict(parent=Z(3, dtype=torch.int64))),
])
def test_the_binding_refuses(rec, call, kw):
    call(rec)
    refused(rec, lambda **k: call(rec, **k), **kw)


@pytest.mark.parametrize("call", [sinks_call, chunk_call, update_call, compact_call, copy_call, fork_call])
def test_error_words_are_on_the_device(rec, call):
    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 1
    refused(rec, lambda **kw: call(rec, **kw), err_word=Z(1).as_subclass(Elsewhere))
    refused(rec, lambda **kw: call(rec, **kw), err_word=Z(1)[:0])
    call(rec, err_word=Z(1))


def test_what_the_binding_passes(rec):
    """Rooms of each row, a table's width, no table, the pairs that a list holds."""
    rooms = _i(5, 6)
    args = update_call(rec, room=rooms)[1]
    assert args[8] == 0 and args[9] == rooms.data_ptr()
    args = update_call(rec, room=7)[1]
    assert args[8] == 7 and args[9] is None and args[5:7] == (2, 3) and args[1] == 9
    assert compact_call(rec, block_table=None, table_out=None)[1][2:5] == (None, 0, 0)
    assert copy_call(rec)[1][4] == 4 and fork_call(rec)[1][1] == 1


def test_weights_of_too_few_heads(rec, monkeypatch):
    from quantized_kv_cache_07_gb300 import cache
    one, per = cache.HeadNorm(torch.ones(128), device="cpu"), cache.HeadNorm(torch.ones(4, 128), torch.ones(2, 128), device="cpu")
    i = _i(0, 1, 2)
    def call(norm, heads=4, kv=2):
        x, y = Z(3, heads, 128, dtype=torch.bfloat16), Z(3, kv, 128, dtype=torch.bfloat16)
        rec.kvq_norm_rope_append(rec.CacheDesc(num_kv_heads=kv), rec.RopeDesc(), norm.desc, x, heads, torch.empty_like(x), y, y,
                                 i, i * 0, i, rec.APPEND_QUANT, Z(1, 2), 1, 2)
    call(one, 64, 8)
    call(per)
    refused(rec, lambda: call(per, heads=5))
    refused(rec, lambda: call(per, kv=3))
    for q, k in ((torch.ones(64), None), (torch.ones(4, 128), torch.ones(128)), (torch.ones(1, 4, 128), None)):
        with pytest.raises(ValueError):
            cache.HeadNorm(q, k, device="cpu")


def test_pages_of_unlike_caches(monkeypatch):
    from types import SimpleNamespace

    from quantized_kv_cache_07_gb300 import cache
    like = dict(num_blocks=8, window=0, desc=None, device="cpu")
    with pytest.raises(ValueError):
        cache.Pages([SimpleNamespace(**like), SimpleNamespace(**dict(like, num_blocks=9))], 2, 4)
