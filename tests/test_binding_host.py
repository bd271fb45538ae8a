"""The binding's own checks, without a GPU: tensors on the CPU stand for the current device's, and a recorder for the
library, so that what would be read or written out of range is seen to be refused before any call."""
import pytest

torch = pytest.importorskip("torch")


class Recorder:
    """Takes the library's place: every entry point notes its arguments and succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, args))
            return 0
        return entry


@pytest.fixture
def lib(monkeypatch):
    from quantized_kv_cache_07_gb300 import _lib
    _lib._need_torch()
    so = Recorder()
    monkeypatch.setattr(_lib, "_current_device", lambda: -1)
    monkeypatch.setattr(_lib, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(_lib, "load", lambda: so)
    monkeypatch.setattr(_lib, "status_string", str)
    monkeypatch.setattr(_lib, "recorder", so, raising=False)
    return _lib


def refused(lib, call, **kw):
    """The call with these arguments is an invalid argument, and nothing reaches the library."""
    before = len(lib.recorder.calls)
    with pytest.raises(lib.KvqError) as e:
        call(**kw)
    assert e.value.status == lib.KVQ_ERR_INVALID_ARG
    assert len(lib.recorder.calls) == before


def _i(*x):
    return torch.tensor(x, dtype=torch.int32)


def rope_call(lib, n=3, heads=2, **kw):
    """kvq_rope_append of n rows into a cache of `heads` KV heads, with these arguments replaced."""
    x = torch.zeros(n, heads, 128, dtype=torch.bfloat16)
    i = torch.arange(n, dtype=torch.int32)
    a = dict(q=x, q_heads=heads, q_out=torch.empty_like(x), k_new=x, v_new=x, pos=i, seq_idx=i * 0, slot=i,
             mode=lib.APPEND_QUANT, block_table=_i(0, 1).view(1, 2), batch=1, max_blocks_per_seq=2)
    a.update(kw)
    lib.kvq_rope_append(lib.CacheDesc(num_kv_heads=heads), lib.RopeDesc(), **a)
    return lib.recorder.calls[-1]


def test_expanded_rows_are_refused(lib):
    """A row stride of 0 stands for contiguous rows in the library: rows behind the one that exists would be read."""
    name, args = rope_call(lib)
    assert name == "kvq_rope_append"
    one = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    flat = torch.zeros(1, 256, dtype=torch.bfloat16)
    for arg in ("q", "k_new", "v_new"):
        refused(lib, lambda **kw: rope_call(lib, **kw), **{arg: one.expand(3, 2, 128)})
        refused(lib, lambda **kw: rope_call(lib, **kw), **{arg: flat.expand(3, 256)})
    # rows that overlap in part
    refused(lib, lambda **kw: rope_call(lib, **kw), k_new=torch.zeros(600, dtype=torch.bfloat16).as_strided((3, 256), (128, 1)))
    # one row has no stride that matters; slices of a wider projection keep theirs
    rope_call(lib, n=1, k_new=one.expand(1, 2, 128))
    wide = torch.zeros(3, 700, dtype=torch.bfloat16)
    assert rope_call(lib, k_new=wide[:, 256:512])[1][7] == 700


def test_the_rotated_queries_fit_their_output(lib):
    """n rows of q_out are written: a smaller tensor is refused; more rows, or another shape, are not."""
    new = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16)
    for out in (new(1, 2, 128), new(3, 1, 128), new(2, 2, 128), new(0)):
        refused(lib, lambda **kw: rope_call(lib, **kw), q_out=out)
    for out in (new(3, 256), new(64, 2, 128)):
        rope_call(lib, q_out=out)
    rope_call(lib, q=None, q_heads=0, q_out=None)


def test_the_block_table_of_the_rotary_write_is_not_too_small(lib):
    """Entries behind the table would be read by a larger batch or max_blocks_per_seq."""
    table = torch.zeros(2, 4, dtype=torch.int32)
    for kw in (dict(batch=3, max_blocks_per_seq=4), dict(batch=2, max_blocks_per_seq=5), dict(batch=9, max_blocks_per_seq=1)):
        refused(lib, lambda **k: rope_call(lib, **k), block_table=table, **kw)
    for t in (table, table.flatten(), torch.zeros(50, 4, dtype=torch.int32)):
        rope_call(lib, block_table=t, batch=2, max_blocks_per_seq=4)
    # not read by the ring, nor for queries alone
    rope_call(lib, block_table=table, batch=3, max_blocks_per_seq=4, mode=lib.APPEND_RING)
    rope_call(lib, block_table=table, batch=3, max_blocks_per_seq=4, k_new=None, v_new=None, seq_idx=None)
    rope_call(lib, block_table=None, batch=0, max_blocks_per_seq=0, k_new=None, v_new=None, seq_idx=None, slot=None)


def shared_call(lib, batch=2, **kw):
    """kvq_decode_shared of a batch with 4 query heads, with these arguments replaced."""
    a = dict(q=torch.zeros(batch, 4, 128, dtype=torch.bfloat16), batch=batch, q_heads=4,
             seq_lens=torch.zeros(batch, dtype=torch.int32), block_table=torch.zeros(batch, 3, dtype=torch.int32),
             max_blocks_per_seq=3, num_groups=1, group_start=_i(0, batch), prefix_blocks=_i(1),
             out=torch.empty(batch, 4, 128, dtype=torch.bfloat16), workspace=torch.empty(512, dtype=torch.uint8),
             workspace_bytes=512)
    a.update(kw)
    lib.kvq_decode_shared(lib.CacheDesc(), **a)
    return lib.recorder.calls[-1]


def test_a_workspace_holds_the_bytes_that_are_named(lib):
    """The library goes by workspace_bytes: a smaller tensor would be written behind its end."""
    refused(lib, lambda **kw: shared_call(lib, **kw), workspace_bytes=513)
    refused(lib, lambda **kw: shared_call(lib, **kw), workspace=torch.empty(100, dtype=torch.uint8))
    assert shared_call(lib, workspace_bytes=500)[1][14] == 500


def test_a_rotary_table_holds_its_positions(lib):
    """max_pos rows of rotary_dim / 2 pairs are written."""
    call = lambda **kw: lib.kvq_rope_table(lib.RopeFreqs(), **kw)
    for shape in ((7, 64, 2), (8, 63, 2), (8, 64)):
        refused(lib, call, rotary_dim=128, max_pos=8, table=torch.empty(shape))
    call(rotary_dim=128, max_pos=8, table=torch.empty(8, 64, 2))
    call(rotary_dim=64, max_pos=8, table=torch.empty(600))


def mass_call(lib, **kw):
    """kvq_attn_mass of two sequences, with these arguments replaced."""
    i = torch.zeros(2, dtype=torch.int32)
    a = dict(q=torch.zeros(2, 4, 128, dtype=torch.bfloat16), batch=2, q_heads=4, lse=torch.zeros(2, 4), seq_lens=i,
             block_table=torch.zeros(2, 3, dtype=torch.int32), max_blocks_per_seq=3, mass=torch.zeros(2, 1, 48))
    a.update(kw)
    lib.kvq_attn_mass(lib.CacheDesc(num_kv_heads=1), **a)


def evict_call(lib, **kw):
    """kvq_evict of two sequences, with these arguments replaced."""
    i, rows = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 1, 48, dtype=torch.int32)
    a = dict(mass=torch.zeros(2, 1, 48), mass_out=None, seq_lens=i, keep=i, block_table=torch.zeros(2, 3, dtype=torch.int32),
             batch=2, max_blocks_per_seq=3, source=rows, new_lens=i.clone())
    a.update(kw)
    lib.kvq_evict(lib.CacheDesc(num_kv_heads=1), **a)


@pytest.mark.parametrize("call", [rope_call, shared_call, mass_call, evict_call])
def test_the_error_word_is_on_the_device(lib, call):
    """Kernels write it: a word of another device, or a tensor without one, is refused."""
    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 1

    word = torch.zeros(1, dtype=torch.int32)
    refused(lib, lambda **kw: call(lib, **kw), err_word=word.as_subclass(Elsewhere))
    refused(lib, lambda **kw: call(lib, **kw), err_word=word[:0])
    for w in (None, word, 0x1000, torch.zeros(4, dtype=torch.uint8), torch.zeros((), dtype=torch.int64)):
        call(lib, err_word=w)


def test_a_rotary_descriptor_keeps_its_table(lib, monkeypatch):
    """The descriptor holds a raw pointer: taken from a RopeTable that nothing else refers to, it must not dangle."""
    import gc
    import weakref

    from quantized_kv_cache_07_gb300 import cache
    monkeypatch.setattr(cache, "_require_cuda", lambda: None)
    turns = cache.RopeTable(16, device="cpu")
    desc, table = turns.desc, weakref.ref(turns.table)
    del turns
    gc.collect()
    assert table() is not None and table().data_ptr() == desc.table
