"""The rotary write of many rows (windows of 16) in every format it takes, queries alone, and the write into the ring:
rotated values and stored bytes compared bit for bit, as in test_gpu_rope.py."""
import numpy as np
import pytest

from synth import f32_to_bf16_bits
from test_gpu_rope import _cache, _i, _same, _t, rotate

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

WINDOWS = 3 * 152 * 64      # vectors of a call from which rows go 16 at a time


@pytest.mark.parametrize("fmt", ["int8", "int4_factor", "asym_k4v8", "k8v4_chan", "bf16"])
@pytest.mark.parametrize("interleaved,R,lens,start", [
    (False, 128, (700, 300), (0, 0)),              # prompts from a block's start
    (True, 64, (333, 16, 1, 17, 640), (0, 32, 5, 16, 7)),   # chunks behind cached tokens, inside and at the end of a block
])
def test_chunks_bit_for_bit(fmt, interleaved, R, lens, start):
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import RopeTable
    rng = np.random.default_rng(21)
    Hq, H, B, n = 24, 3, len(lens), sum(lens)
    assert n * (Hq + 2 * H) >= WINDOWS
    seq = np.repeat(np.arange(B), lens)
    slot = np.concatenate([s + np.arange(m) for s, m in zip(start, lens)])
    pos = rng.integers(0, 4096, n)
    order = np.arange(n)
    order[-60:] = rng.permutation(order[-60:])     # no runs there
    seq, slot, pos = seq[order], slot[order], pos[order]
    bad = np.zeros(n, bool)
    bad[[20, 333, n - 7]] = True
    pos[bad] = 5000                                # no such row in the table
    mbps = 64
    perm = rng.permutation(mbps * B).reshape(B, mbps)
    table = _i(perm)
    qkv = f32_to_bf16_bits(rng.standard_normal((n, (Hq + 2 * H) * 128)).astype(np.float32))
    qkv[40] = 0
    rope = RopeTable(4096, rotary_dim=R, interleaved=interleaved)
    x = _t(qkv)
    q_out = torch.full((n, Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    state = rng.bit_generator.state
    c = _cache(fmt, H, mbps * B, rng)
    _lib.kvq_rope_append(c.desc, rope.desc, x[:, :Hq * 128], Hq, q_out, x[:, Hq * 128:(Hq + H) * 128],
                         x[:, (Hq + H) * 128:], _i(pos), _i(seq), _i(slot), _lib.APPEND_QUANT, table, B, mbps, err_word=err)
    assert int(err) == _lib.KVQ_DEVERR_POSITION
    ok, heads = ~bad, qkv.reshape(n, -1, 128)
    cs = rope.table.cpu().numpy().astype(np.float64)[np.where(bad, 0, pos)]
    np.testing.assert_array_equal(q_out.view(torch.int16).cpu().numpy().view(np.uint16)[ok],
                                  rotate(heads[:, :Hq], cs, interleaved)[ok])
    assert torch.all(q_out[torch.from_numpy(bad).cuda()] == 7)
    rng.bit_generator.state = state
    ref = _cache(fmt, H, mbps * B, rng)
    _lib.kvq_append(ref.desc, _t(rotate(heads[:, Hq:Hq + H], cs, interleaved)[ok]), _t(heads[:, Hq + H:][ok]),
                    _i(seq[ok]), _i(slot[ok]), _lib.APPEND_QUANT, table, B, mbps)
    _same(c, ref)
    # read back in one call and a hundred at a time
    where = _i(perm[seq, slot // 16] * 16 + slot % 16)
    many = [torch.empty(n, H, 128, device="cuda") for _ in range(2)]
    _lib.kvq_dequant(c.desc, where, *many)
    for a in range(0, n, 100):
        few = [torch.empty(min(100, n - a), H, 128, device="cuda") for _ in range(2)]
        _lib.kvq_dequant(c.desc, where[a:a + 100].contiguous(), *few)
        for m, f in zip(many, few):
            assert torch.equal(m[a:a + 100], f)


@pytest.mark.parametrize("fmt", ["int8", "int4_factor", "int2", "bf16"])
@pytest.mark.parametrize("Hq,in_place", [(32, False), (32, True), (27, False), (1, False)])
def test_many_queries_alone(fmt, Hq, in_place):
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import RopeTable
    rng = np.random.default_rng(22)
    n = -(-WINDOWS // Hq) + 5
    bits = f32_to_bf16_bits(rng.standard_normal((n, Hq, 128)).astype(np.float32))
    pos = rng.integers(0, 3000, n)
    pos[[3, n - 1]] = [-1, 3000]
    rope, c = RopeTable(3000, rotary_dim=96), _cache(fmt, 2, 1, rng)
    q = _t(bits)
    out, err = q if in_place else torch.zeros_like(q), _i([0])
    _lib.kvq_rope_append(c.desc, rope.desc, q, Hq, out, None, None, _i(pos), None, None, _lib.APPEND_QUANT, None, 0, 0,
                         err_word=err)
    assert int(err) == _lib.KVQ_DEVERR_POSITION
    ok = (pos >= 0) & (pos < 3000)
    want = rotate(bits, rope.table.cpu().numpy().astype(np.float64)[np.where(ok, pos, 0)], False)
    want[~ok] = bits[~ok] if in_place else 0
    np.testing.assert_array_equal(out.view(torch.int16).cpu().numpy().view(np.uint16), want)
    assert not c.k_codes.any() and not c.v_codes.any()


@pytest.mark.parametrize("fmt", ["int8", "asym_k4v8", "int2", "int4_factor"])
@pytest.mark.parametrize("n,W", [(37, 16), (1000, 48)])      # the latter more vectors than windows of rows start from
def test_write_into_the_ring(fmt, n, W):
    """KVQ_APPEND_RING: the last W of each sequence's rows, in any order of the call, and one row of no sequence."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import RopeTable
    rng = np.random.default_rng(23)
    Hq, H = 24, 3
    B = -(-n // W)
    seq, slot = np.arange(n) % B, 100 + np.arange(n) // B    # fewer than W rows of a sequence
    pos = rng.integers(0, 4000, n)
    seq[11] = B
    q = f32_to_bf16_bits(rng.standard_normal((n, Hq, 128)).astype(np.float32))
    k = f32_to_bf16_bits(rng.standard_normal((n, H, 128)).astype(np.float32))
    v = f32_to_bf16_bits(rng.standard_normal((n, H, 128)).astype(np.float32))
    rope = RopeTable(4000, interleaved=True)
    cs = rope.table.cpu().numpy().astype(np.float64)[pos]
    state = rng.bit_generator.state
    a = _cache(fmt, H, 1, rng, window=W, window_batch=B)
    rng.bit_generator.state = state
    b = _cache(fmt, H, 1, rng, window=W, window_batch=B)
    out, err, err_b = torch.zeros(n, Hq, 128, dtype=torch.bfloat16, device="cuda"), _i([0]), _i([0])
    _lib.kvq_rope_append(a.desc, rope.desc, _t(q), Hq, out, _t(k), _t(v), _i(pos), _i(seq), _i(slot), _lib.APPEND_RING,
                         None, B, 0, err_word=err)
    _lib.kvq_append(b.desc, _t(rotate(k, cs, True)), _t(v), _i(seq), _i(slot), _lib.APPEND_RING, None, B, 0, err_word=err_b)
    _same(a, b)
    assert a.k_window.any() and int(err) == int(err_b) == _lib.KVQ_DEVERR_POSITION
    np.testing.assert_array_equal(out.view(torch.int16).cpu().numpy().view(np.uint16), rotate(q, cs, True))
