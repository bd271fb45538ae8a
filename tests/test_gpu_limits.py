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
