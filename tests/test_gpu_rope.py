"""Rotary positions with the cache write (kvq_rope_table, kvq_rope_append).

The rotation's definition is checked in float64: rotated values are the exact
ones rounded to float32 and then to bf16, so queries are compared bit for bit,
and the stored cache is compared, bit for bit, with kvq_append of the rotated keys.
"""
import numpy as np
import pytest

from oracle import kvq_oracle as O
from synth import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

FORMATS = {
    "int8": dict(k_bits=8, v_bits=8), "int4_factor": dict(k_bits=4, v_bits=4, factor=True),
    "asym_k4v8": dict(k_bits=4, v_bits=8, asym=True), "k8v4_chan": dict(k_bits=8, v_bits=4, factor=True,
                                                                       k_per_channel=True),
    "int2": dict(k_bits=2, v_bits=2), "asym_int2": dict(k_bits=2, v_bits=2, asym=True),
    "bf16": dict(k_bits=16, v_bits=16),
}


def _t(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def _i(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def rotate(bits, cs, interleaved):
    """bf16 bits [n, heads, 128] turned by cs [n, pairs, 2] (float64 of the table): bf16 bits."""
    x = O.bf16_to_f64(bits)
    pairs = cs.shape[1]
    j = np.arange(pairs)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + pairs)
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return f32_to_bf16_bits(y.astype(np.float32))


def _cache(fmt, H, blocks, rng, **kw):
    from quantized_kv_cache_07_gb300.cache import KVCache
    f = dict(FORMATS[fmt])
    factor = (0.5 + rng.random((H, 128))).astype(np.float32) if f.pop("factor", False) else None
    if f.get("k_per_channel"):
        factor /= 40.0
    return KVCache(blocks, H, channel_factor=factor, **f, **kw)


def _pools(c):
    return [None if t is None else t.view(torch.uint8).cpu().numpy()
            for t in (c.k_codes, c.v_codes, c.meta, c.k_window, c.v_window)]


def _same(a, b):
    for x, y in zip(_pools(a), _pools(b)):
        assert (x is None) == (y is None)
        if x is not None:
            np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("scaling,kw", [
    ("plain", {}), ("plain", dict(base=500000.0, rotary_dim=64, amplitude=1.25)), ("linear", dict(factor=4.0)),
    ("ntk", dict(factor=8.0, rotary_dim=96)),
    ("bands", dict(base=500000.0, factor=8.0, original_len=8192, low_turns=1.0, high_turns=4.0)),
])
def test_table_against_float64(scaling, kw):
    from quantized_kv_cache_07_gb300.cache import RopeTable
    n = 131072 if scaling == "plain" else 4099
    t = RopeTable(n, scaling=scaling, **kw)
    R, base, f = kw.get("rotary_dim", 128), kw.get("base", 10000.0), kw.get("factor", 1.0)
    if scaling == "ntk":
        base = base * f ** (R / (R - 2))
    w = base ** (-2.0 * np.arange(R // 2) / R)
    if scaling == "linear":
        w = w / f
    if scaling == "bands":
        turns = kw["original_len"] * w / (2 * np.pi)
        keep = np.clip((turns - kw["low_turns"]) / (kw["high_turns"] - kw["low_turns"]), 0, 1)
        assert 0 < np.sum((keep > 0) & (keep < 1)) and keep[0] == 1 and keep[-1] == 0
        w = keep * w + (1 - keep) * w / f
    at = np.unique(np.concatenate([np.arange(40), np.random.default_rng(1).integers(0, n, 500), [n - 1]]))
    angle = at[:, None] * w
    ref = kw.get("amplitude", 1.0) * np.stack([np.cos(angle), np.sin(angle)], -1)
    got = t.table.cpu().numpy()[at]
    # half a step of float32 below 2, and 1e-10 for the angle's own rounding (131071 times 2^-53 and a few operations)
    np.testing.assert_allclose(got, ref, rtol=2.0 ** -24, atol=1e-10)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("interleaved,R", [(False, 128), (True, 128), (False, 64), (True, 96), (False, 8)])
def test_rotated_queries_and_stored_keys_bit_for_bit(fmt, interleaved, R):
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import RopeTable
    rng = np.random.default_rng(3)
    Hq, H, lens = 6, 2, (37, 1, 50)
    n = sum(lens)
    seq = np.repeat(np.arange(3), lens)
    slot = np.concatenate([np.arange(l) for l in lens])
    pos = slot + np.repeat([1000, 7, 4000], lens)           # positions far from the slots
    table = _i(rng.permutation(12).reshape(3, 4))
    qkv = f32_to_bf16_bits(rng.standard_normal((n, (Hq + 2 * H) * 128)).astype(np.float32))
    qkv[5] = 0                                              # a zero row
    rope = RopeTable(4096, rotary_dim=R, interleaved=interleaved)
    x = _t(qkv)
    q, k, v = x[:, :Hq * 128], x[:, Hq * 128:(Hq + H) * 128], x[:, (Hq + H) * 128:]
    q_out = torch.full((n, Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    state = rng.bit_generator.state
    c = _cache(fmt, H, 12, rng)
    _lib.kvq_rope_append(c.desc, rope.desc, q, Hq, q_out, k, v, _i(pos), _i(seq), _i(slot), _lib.APPEND_QUANT, table,
                         3, 4, err_word=err)
    cs = rope.table.cpu().numpy().astype(np.float64)[pos]
    heads = qkv.reshape(n, -1, 128)
    np.testing.assert_array_equal(q_out.view(torch.int16).cpu().numpy().view(np.uint16),
                                  rotate(heads[:, :Hq], cs, interleaved))
    rng.bit_generator.state = state
    ref = _cache(fmt, H, 12, rng)
    _lib.kvq_append(ref.desc, _t(rotate(heads[:, Hq:Hq + H], cs, interleaved)), _t(heads[:, Hq + H:]), _i(seq),
                    _i(slot), _lib.APPEND_QUANT, table, 3, 4, err_word=err)
    _same(c, ref)
    assert int(err.item()) == 0


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("interleaved,R,lens", [
    (False, 128, (300, 1, 50)),      # runs of whole blocks that are not aligned with the call's rows, and their ends
    (True, 64, (16, 17, 15, 240)), (False, 96, (512,)),
])
def test_prompts_bit_for_bit(fmt, interleaved, R, lens):
    """Enough rows for the 16-row windows: whole blocks, their ragged ends, chunks that begin inside a block, rows out
    of order, and rows that are flagged in between."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import RopeTable
    rng = np.random.default_rng(13)
    Hq, H, B = 11, 3, len(lens)
    n = sum(lens)
    seq = np.repeat(np.arange(B), lens)
    start = np.array([0, 32, 5, 16][:B]) if FORMATS[fmt]["k_bits"] != 2 else np.zeros(B, int)
    slot = np.concatenate([s + np.arange(l) for s, l in zip(start, lens)])
    pos = slot + np.repeat([1000, 7, 4000, 20][:B], lens)
    order = np.arange(n)
    if fmt in ("int8", "asym_k4v8"):   # the last rows shuffled: no runs there
        order[-40:] = rng.permutation(order[-40:])
    seq, slot, pos = seq[order], slot[order], pos[order]
    bad = np.zeros(n, bool)
    if fmt in ("int8", "bf16", "int4_factor"):
        bad[[20, n - 7]] = True
        pos[bad] = 9000                # no such row in the table
    blocks = 34
    perm = rng.permutation(blocks * B).reshape(B, blocks)
    table = _i(perm)
    qkv = f32_to_bf16_bits(rng.standard_normal((n, (Hq + 2 * H) * 128)).astype(np.float32))
    rope = RopeTable(8192, rotary_dim=R, interleaved=interleaved)
    x = _t(qkv)
    q, k, v = x[:, :Hq * 128], x[:, Hq * 128:(Hq + H) * 128], x[:, (Hq + H) * 128:]
    q_out = torch.full((n, Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    state = rng.bit_generator.state
    c = _cache(fmt, H, blocks * B, rng)
    _lib.kvq_rope_append(c.desc, rope.desc, q, Hq, q_out, k, v, _i(pos), _i(seq), _i(slot), _lib.APPEND_QUANT, table,
                         B, blocks, err_word=err)
    assert int(err.item()) == (_lib.KVQ_DEVERR_POSITION if bad.any() else 0)
    ok = ~bad
    cs = rope.table.cpu().numpy().astype(np.float64)[np.where(bad, 0, pos)]
    heads = qkv.reshape(n, -1, 128)
    got = q_out.view(torch.int16).cpu().numpy().view(np.uint16)
    np.testing.assert_array_equal(got[ok], rotate(heads[:, :Hq], cs, interleaved)[ok])
    assert torch.all(q_out[torch.from_numpy(bad)] == 7)
    rng.bit_generator.state = state
    ref = _cache(fmt, H, blocks * B, rng)
    # one row at a time would do as well: kvq_append of the rotated rows that are good
    _lib.kvq_append(ref.desc, _t(rotate(heads[:, Hq:Hq + H], cs, interleaved)[ok]), _t(heads[:, Hq + H:][ok]),
                    _i(seq[ok]), _i(slot[ok]), _lib.APPEND_QUANT, table, B, blocks)
    _same(c, ref)
    # and read back, many slots and few
    where = _i(perm[seq, slot // 16] * 16 + slot % 16)
    many = [torch.empty(n, H, 128, device="cuda") for _ in range(2)]
    _lib.kvq_dequant(c.desc, where, *many)
    for a in range(0, n, 100):
        few = [torch.empty(min(100, n - a), H, 128, device="cuda") for _ in range(2)]
        _lib.kvq_dequant(c.desc, where[a:a + 100].contiguous(), *few)
        for m, f in zip(many, few):
            assert torch.equal(m[a:a + 100], f)


@pytest.mark.parametrize("fmt", ["int8", "int4_factor", "asym_k4v8"])
def test_steps_through_the_window(fmt):
    """Token by token through the bf16 window (KVQ_APPEND_STEP), every step with its own positions."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import RopeTable
    rng = np.random.default_rng(4)
    B, H, W, steps = 3, 2, 16, 41
    rope = RopeTable(512, rotary_dim=64)
    table = _i(rng.permutation(9).reshape(3, 3))
    state = rng.bit_generator.state
    a = _cache(fmt, H, 9, rng, window=W, window_batch=B)
    rng.bit_generator.state = state
    b = _cache(fmt, H, 9, rng, window=W, window_batch=B)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    tab = rope.table.cpu().numpy().astype(np.float64)
    for p in range(steps):
        k = f32_to_bf16_bits(rng.standard_normal((B, H, 128)).astype(np.float32))
        v = f32_to_bf16_bits(rng.standard_normal((B, H, 128)).astype(np.float32))
        slot, pos = np.full(B, p), p + np.array([0, 100, 400])
        _lib.kvq_rope_append(a.desc, rope.desc, None, 0, None, _t(k), _t(v), _i(pos), _i(np.arange(B)), _i(slot),
                             _lib.APPEND_STEP, table, B, 3, err_word=err)
        _lib.kvq_append(b.desc, _t(rotate(k, tab[pos], False)), _t(v), _i(np.arange(B)), _i(slot), _lib.APPEND_STEP,
                        table, B, 3, err_word=err)
    _same(a, b)
    assert int(err.item()) == 0


def test_bad_positions_are_flagged_and_their_rows_left_alone():
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache, RopeTable
    rng = np.random.default_rng(5)
    rope = RopeTable(64)
    x = _t(f32_to_bf16_bits(rng.standard_normal((5, 2, 128)).astype(np.float32)))
    for fmt in (dict(k_bits=8, v_bits=8), dict(k_bits=2, v_bits=2)):
        c = KVCache(4, 2, **fmt)
        c.k_codes.fill_(9)
        q_out = torch.full((5, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        # every row at the start of a block of its own; rows 1 and 3 have no such position
        _lib.kvq_rope_append(c.desc, rope.desc, x, 2, q_out, x, x, _i([0, -1, 63, 64, 5]), _i([0, 0, 0, 0, 9]),
                             _i([0, 16, 32, 48, 0]), _lib.APPEND_QUANT, _i([[0, 1, 2, 3]]), 1, 4, err_word=err)
        assert int(err.item()) == _lib.KVQ_DEVERR_POSITION
        assert torch.all(q_out[[1, 3]] == 7) and not torch.any(torch.all((q_out[[0, 2, 4]] == 7).flatten(1), 1))
        blocks = c.k_codes.view(2, 4, -1)
        assert torch.all(blocks[:, [1, 3]] == 9) and torch.any(blocks[:, 0] != 9) and torch.any(blocks[:, 2] != 9)


def test_queries_alone_in_place_and_keys_alone():
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache, RopeTable
    rng = np.random.default_rng(6)
    rope = RopeTable(300, interleaved=True)
    bits = f32_to_bf16_bits(rng.standard_normal((9, 5, 128)).astype(np.float32))
    pos = rng.integers(0, 300, 9)
    want = rotate(bits, rope.table.cpu().numpy().astype(np.float64)[pos], True)
    c = KVCache(1, 5, 8, 8)
    q = _t(bits)
    _lib.kvq_rope_append(c.desc, rope.desc, q, 5, q, None, None, _i(pos), None, None, _lib.APPEND_QUANT, None, 0, 0)
    np.testing.assert_array_equal(q.view(torch.int16).cpu().numpy().view(np.uint16), want)
    assert not torch.any(c.k_codes)
    # keys alone, the cache slot standing for the position
    slot = np.arange(9)
    cs = rope.table.cpu().numpy().astype(np.float64)[slot]
    _lib.kvq_rope_append(c.desc, rope.desc, None, 0, None, _t(bits), _t(bits), None, _i(slot * 0), _i(slot),
                         _lib.APPEND_QUANT, _i([[0]]), 1, 1)
    ref = KVCache(1, 5, 8, 8)
    _lib.kvq_append(ref.desc, _t(rotate(bits, cs, True)), _t(bits), _i(slot * 0), _i(slot), _lib.APPEND_QUANT,
                    _i([[0]]), 1, 1)
    _same(c, ref)
    # no rows
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    z = torch.empty(0, 5, 128, dtype=torch.bfloat16, device="cuda")
    _lib.kvq_rope_append(c.desc, rope.desc, z, 5, z, z, z, e, e, e, _lib.APPEND_QUANT, _i([[0]]), 1, 1)


def test_the_binding_refuses_what_the_library_cannot_see():
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache, RopeTable
    rope, c = RopeTable(64), KVCache(1, 2, 8, 8)
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    i = _i([0, 1, 2])

    def call(q=x, q_out=x, k=x, v=x, pos=i, slot=i):
        _lib.kvq_rope_append(c.desc, rope.desc, q, 2, q_out, k, v, pos, i * 0, slot, _lib.APPEND_QUANT, _i([[0]]), 1, 1)

    call(q_out=torch.empty_like(x))
    for kw in (dict(q=x.float()), dict(k=x.cpu()), dict(v=x[:, :1]), dict(q=x.transpose(1, 2)), dict(pos=i.long()),
               dict(q_out=x.half()), dict(slot=i.repeat(2)[::2])):
        with pytest.raises(_lib.KvqError) as e:
            call(**kw)
        assert e.value.status == _lib.KVQ_ERR_INVALID_ARG


def test_captured_and_replayed_on_a_side_stream():
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache, RopeTable
    rng = np.random.default_rng(8)
    rope, c = RopeTable(200), KVCache(2, 2, 8, 8)
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    out, pos, slot = torch.zeros_like(x), _i([0, 0, 0, 0]), _i([0, 1, 0, 1])
    seq, table = _i([0, 0, 1, 1]), _i([[0], [1]])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        _lib.kvq_rope_append(c.desc, rope.desc, x, 2, out, x, x, pos, seq, slot, _lib.APPEND_QUANT, table, 2, 1)
    for _ in range(2):
        bits = f32_to_bf16_bits(rng.standard_normal((4, 2, 128)).astype(np.float32))
        p = rng.integers(0, 200, 4)
        x.copy_(_t(bits))
        pos.copy_(_i(p))
        g.replay()
        torch.cuda.synchronize()
        want = rotate(bits, rope.table.cpu().numpy().astype(np.float64)[p], False)
        np.testing.assert_array_equal(out.view(torch.int16).cpu().numpy().view(np.uint16), want)


@pytest.mark.parametrize("k_bits,v_bits,asym,kchan", [(8, 8, False, False), (4, 4, True, False), (4, 8, False, False),
                                                      (8, 4, False, True), (16, 16, False, False)])
@pytest.mark.parametrize("shift", [0, 1])
def test_read_back_of_many_slots(k_bits, v_bits, asym, kchan, shift):
    """Whole blocks at any row of the call, parts of blocks, repeated, missing and foreign slots, in one call and a few
    at a time; outputs that are not aligned to 16 bytes."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache
    rng = np.random.default_rng(k_bits + v_bits)
    H, nb = 2, 40
    factor = rng.random((H, 128)) + 0.5 if kchan else None
    c = KVCache(nb, H, k_bits, v_bits, asym=asym, channel_factor=factor, k_per_channel=kchan)
    for pool in (c.k_codes, c.v_codes):
        raw = rng.standard_normal(pool.numel() // 2).astype(np.float32) if k_bits == 16 else None
        if raw is None:
            pool.copy_(torch.from_numpy(rng.integers(1, 256, pool.numel()).astype(np.uint8)))
        else:
            pool.copy_(torch.from_numpy(raw).bfloat16().view(torch.uint8))
    if c.meta is not None:
        c.meta.copy_(torch.from_numpy(rng.random(c.meta.numel()).astype(np.float32)))
    block = lambda b: np.arange(16 * b, 16 * b + 16)
    parts = [block(3), block(5)[2:], block(7), [-1, 16 * nb, 16 * nb + 16], block(7), block(8), block(9)[:15], block(11),
             [3], block(12), block(13)[::-1], block(39), block(2)[1:], block(2)[:1], block(20), [-5], block(21)]
    slots = np.concatenate([np.asarray(p, np.int32) for p in (parts + parts[::-1]) * 8 + [[7]]])
    assert slots.size * 2 * H >= 152 * 64 and slots.size % 16 != 0
    n = slots.size
    s = torch.from_numpy(slots).cuda()
    whole = [torch.full((n * H * 128 + shift,), 7.0, device="cuda")[shift:] for _ in range(2)]
    _lib.kvq_dequant(c.desc, s, *whole)
    few = [torch.zeros(n, H, 128, device="cuda") for _ in range(2)]
    for r in range(0, n, 100):
        _lib.kvq_dequant(c.desc, s[r:r + 100], few[0][r:], few[1][r:])
    for x, y in zip(whole, few):
        assert torch.equal(x.view(n, H, 128), y)
        assert not x.view(n, H, 128)[s < 0].any() and x.view(n, H, 128)[s == 48].any()


@pytest.mark.parametrize("k_bits,v_bits,asym,factor,interleaved,R", [
    (8, 8, False, False, False, 128), (4, 4, True, True, True, 64), (4, 8, False, True, False, 96),
    (8, 4, True, False, True, 128), (16, 16, False, False, False, 64)])
def test_many_rows_as_in_small_calls(k_bits, v_bits, asym, factor, interleaved, R):
    """Enough rows for windows of 16, runs of whole blocks at any row, parts of blocks, bad positions: the same bits as
    calls of a few rows (which are compared with the oracle above)."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache, RopeTable
    rng = np.random.default_rng(R + k_bits)
    H, Hq, lens = 3, 6, [1000, 1, 37, 16, 15, 1531, 17]
    n, mbps, B = sum(lens), 96, len(lens)
    assert n * (Hq + 2 * H) >= 3 * 152 * 64
    rope = RopeTable(2000, rotary_dim=R, interleaved=interleaved)
    i = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    x = torch.from_numpy(rng.standard_normal((n, (Hq + 2 * H) * 128)).astype(np.float32)).bfloat16().cuda()
    q, k, v = x[:, :Hq * 128], x[:, Hq * 128:(Hq + H) * 128], x[:, (Hq + H) * 128:]
    seq = np.repeat(np.arange(B), lens)
    first = rng.integers(0, 3, B) * 8          # some sequences start inside a block
    slot = np.concatenate([np.arange(m) + f for m, f in zip(lens, first)])
    pos = rng.integers(0, 2000, n)
    pos[[5, 1010, 2000]] = [-1, 2000, -7]      # flagged, their rows left alone
    table = i(rng.permutation(B * mbps).reshape(B, mbps))
    c_f = rng.random((H, 128)) + 0.5 if factor else None
    got = []
    for step in (n, 100):
        c = KVCache(B * mbps, H, k_bits, v_bits, asym=asym, channel_factor=c_f)
        out, err = torch.zeros(n, Hq, 128, dtype=torch.bfloat16, device="cuda"), i([0])
        for r in range(0, n, step):
            e = min(n, r + step)
            _lib.kvq_rope_append(c.desc, rope.desc, q[r:e], Hq, out[r:e], k[r:e], v[r:e], i(pos[r:e]), i(seq[r:e]),
                                 i(slot[r:e]), _lib.APPEND_QUANT, table, B, mbps, err_word=err)
        assert int(err) == _lib.KVQ_DEVERR_POSITION
        got.append([out.view(torch.int16), c.k_codes, c.v_codes] + ([] if c.meta is None else [c.meta.view(torch.int32)]))
    for a, b in zip(*got):
        assert torch.equal(a, b)
