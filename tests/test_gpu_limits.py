"""Positions and block tables at the ends of 32 bits."""
import numpy as np
import pytest

from synth import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

FORMATS = {"int8": dict(k_bits=8, v_bits=8), "int4": dict(k_bits=4, v_bits=4), "int2": dict(k_bits=2, v_bits=2),
           "bf16": dict(k_bits=16, v_bits=16)}


def _bits(rng, *shape):
    bits = f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))
    return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)


def _i(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def _write(how, c, q, k, v, rope, seq, slot, table, B, mbps, err):
    from quantized_kv_cache_07_gb300 import _lib
    if how == "append":
        _lib.kvq_append(c.desc, k, v, seq, slot, _lib.APPEND_QUANT, table, B, mbps, err_word=err)
    else:
        n, Hq = q.shape[:2]
        out = torch.empty(n, Hq, 128, dtype=torch.bfloat16, device="cuda")
        _lib.kvq_rope_append(c.desc, rope.desc, q, Hq, out, k, v, seq * 0, seq, slot, _lib.APPEND_QUANT, table, B, mbps,
                             err_word=err)


def _pools(c):
    return [t.view(torch.uint8) for t in (c.k_codes, c.v_codes, c.meta) if t is not None]


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("how,n", [("append", 48), ("rope", 48), ("rope", 1000)])   # 1000 rows: windows of 16
def test_a_block_at_the_last_positions_is_behind_every_table(fmt, how, n):
    """Sixteen rows at 2^31 - 16 .. 2^31 - 1, a whole block: flagged and skipped, the other rows written as without them."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache, RopeTable
    rng = np.random.default_rng(1)
    H, Hq, mbps = 3, 26, 64
    assert n < 1000 or n * (Hq + 2 * H) >= 3 * 152 * 64
    q, k, v = _bits(rng, n, Hq, 128), _bits(rng, n, H, 128), _bits(rng, n, H, 128)
    rope, table = RopeTable(1), _i(rng.permutation(2 * mbps).reshape(2, mbps))
    seq = np.repeat([0, 1], [16, n - 16])
    far = np.concatenate([2 ** 31 - 16 + np.arange(16), np.arange(n - 16)])
    got = []
    for slot, bits in ((far, _lib.KVQ_DEVERR_POSITION), (np.concatenate([np.full(16, -1), np.arange(n - 16)]),
                                                         _lib.KVQ_DEVERR_POSITION)):
        c, err = KVCache(2 * mbps, H, **FORMATS[fmt]), _i([0])
        _write(how, c, q, k, v, rope, _i(seq), _i(slot), table, 2, mbps, err)
        assert int(err) == bits
        got.append(_pools(c))
    for a, b in zip(*got):
        assert torch.equal(a, b) and a.any()


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("how,n", [("append", 48), ("rope", 48), ("rope", 1000)])
def test_rows_of_a_table_that_covers_every_position(fmt, how, n):
    """2^27 + 1 entries a row: 16 times as many positions pass 32 bits."""
    from quantized_kv_cache_07_gb300.cache import KVCache, RopeTable
    rng = np.random.default_rng(2)
    H, Hq, mbps = 3, 26, 2 ** 27 + 1
    q, k, v = _bits(rng, n, Hq, 128), _bits(rng, n, H, 128), _bits(rng, n, H, 128)
    rope, blocks, first = RopeTable(1), n // 16 + 2, 2 ** 31 - 16 * 70
    wide = torch.full((1, mbps), -1, dtype=torch.int32, device="cuda")
    order = _i(rng.permutation(blocks))
    wide[0, first // 16:first // 16 + blocks] = order
    got = []
    for slot, table in ((first + np.arange(n), wide), (np.arange(n), order[None])):
        c, err = KVCache(blocks, H, **FORMATS[fmt]), _i([0])
        _write(how, c, q, k, v, rope, _i(np.zeros(n)), _i(slot), table, 1, table.shape[1], err)
        assert int(err) == 0
        got.append(_pools(c))
    for a, b in zip(*got):
        assert torch.equal(a, b) and a.any()


@pytest.mark.parametrize("kw", [dict(), dict(window=32), dict(k_bits=16, v_bits=16, q_heads=14)])
@pytest.mark.parametrize("batch", [2, 9])     # shared prefixes on 16-vector tiles; on tcgen05 (not bf16)
def test_attention_over_a_table_that_covers_every_position(kw, batch):
    """The same results from tables of 2^27 + 1 entries a row as from short ones, in every call that reads a table."""
    from harness import DeviceRun, small_workload
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import DecodeWorkspace, SharedWorkspace
    from synth import make_inputs
    w = small_workload("wide_table", **dict(dict(batch=batch, q_heads=16, kv_heads=2, len_range=(100, 160)), **kw))
    inp = make_inputs(w)
    inp.block_table[:, :4] = inp.block_table[0, :4]
    run = DeviceRun(inp)
    Hq, H, W = w.q_heads, w.kv_heads, w.window
    wide = torch.full((batch, 2 ** 27 + 1), -1, dtype=torch.int32, device="cuda")
    wide[:, :inp.max_blocks] = run.table
    got = []
    for table in (run.table, wide):
        mbps, err = table.shape[1], _i([0])
        new = lambda *shape, t=torch.float32: torch.zeros(*shape, dtype=t, device="cuda")
        res = [new(batch, Hq, 128), new(batch, Hq), new(batch, Hq, 128), new(batch, Hq), new(batch, H, 160)]
        ws, sw = DecodeWorkspace(run.cache, batch, Hq), SharedWorkspace(run.cache, batch, Hq, 1)
        _lib.kvq_decode(run.cache.desc, run.q, batch, Hq, run.lens, table, mbps, res[0], lse=res[1], workspace=ws.buf,
                        workspace_bytes=ws.nbytes, err_word=err)
        _lib.kvq_decode_shared(run.cache.desc, run.q, batch, Hq, run.lens, table, mbps, 1, _i([0, batch]), _i([4]), res[2],
                               lse=res[3], workspace=sw.buf, workspace_bytes=sw.nbytes, err_word=err)
        _lib.kvq_attn_mass(run.cache.desc, run.q, batch, Hq, res[1], run.lens, table, mbps, res[4], err_word=err)
        source, lens = new(batch, H, 160, t=torch.int32), new(batch, t=torch.int32)
        if not W:
            seq, pos = torch.arange(batch, device="cuda").int(), run.lens - 1
            for ctas in (5, -1) if w.k_bits != 16 else (5,):
                out = new(batch, Hq, 128)
                nb = _lib.kvq_prefill_workspace_size(run.cache.desc, batch, Hq, ctas)
                pw = new(max(nb, 16), t=torch.uint8)
                _lib.kvq_prefill(run.cache.desc, run.q, Hq, seq, pos, table, batch, mbps, out, workspace=pw,
                                 workspace_bytes=nb, stream_ctas=ctas, err_word=err)
                res.append(out)
        pools = [t for t in (run.cache.k_codes, run.cache.v_codes, run.cache.meta) if t is not None]
        before = [t.clone() for t in pools]
        _lib.kvq_evict(run.cache.desc, res[4], None, run.lens, run.lens - 64, table, batch, mbps, source, lens,
                       protect_first=64, err_word=err)
        res += [source] + [t.clone() for t in pools] + [lens]
        for t, old in zip(pools, before):      # the eviction's moves back
            t.copy_(old)
        assert int(err) == 0
        got.append(res)
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert bool((got[0][-1] < run.lens).all())


@pytest.mark.parametrize("kw", [dict(window=32), dict(window=32, k_bits=4, asym=True, q_heads=16), dict(), dict(k_bits=4)])
@pytest.mark.parametrize("stride", [20, 64, 100])
def test_attention_mass_of_sequences_longer_than_their_row(kw, stride):
    """Flagged, and what the row holds is the sums of its tokens: the window's last tokens are those of the whole sequence."""
    from harness import DeviceRun, small_workload
    from quantized_kv_cache_07_gb300 import _lib
    from synth import make_inputs
    w = small_workload("short_rows", **dict(dict(batch=6, len_range=(40, 130)), **kw))
    run = DeviceRun(make_inputs(w))
    assert (run.lens > stride).any()
    _, lse = run.decode()
    lse = torch.from_numpy(lse).cuda()
    got = []
    for width in (160, stride):
        # a guard row behind the last: nothing may be written there
        mass, err = torch.ones(w.batch + 1, w.kv_heads, width, device="cuda"), _i([0])
        _lib.kvq_attn_mass(run.cache.desc, run.q, w.batch, w.q_heads, lse, run.lens, run.table, run.inp.max_blocks,
                           mass[:w.batch], decay=0.5, err_word=err)
        assert int(err) == (0 if width == 160 else _lib.KVQ_DEVERR_SEQ_LEN) and bool((mass[w.batch] == 1).all())
        got.append(mass[:w.batch])
    assert torch.equal(got[0][..., :stride], got[1])
