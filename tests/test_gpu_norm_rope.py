"""Norms of the heads and rotary positions with the cache write (kvq_norm_rope_append).

The definition is evaluated in float64.  Keys are that rounded to float32 and then to bf16: the stored cache is compared,
bit for bit, with kvq_append of the keys so computed.  Queries are float32 rounded once: half a bf16 step, and before
that 2^-20 of the two terms of a turn (float32's 12 roundings of 2^-24 at most, and 2^-22 of the root).
"""
import numpy as np
import pytest

from oracle import kvq_oracle as O
from synth import f32_to_bf16_bits
from test_gpu_rope import FORMATS, _cache, _i, _same, _t

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def normed(bits, weight, eps, cs, interleaved, rounded=True):
    """bf16 bits [n, heads, 128]: each head over the root of its mean square, weighted, turned by cs [n, pairs, 2].  As
    bf16 bits, or in float64 with the sum of the terms' sizes."""
    x = O.bf16_to_f64(bits)
    eps = float(np.float32(eps))
    with np.errstate(all="ignore"):
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            x = x * weight.astype(np.float64)
        pairs = cs.shape[1]
        j = np.arange(pairs)
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + pairs)
        c, s = cs[:, None, :, 0], cs[:, None, :, 1]
        y, size = x.copy(), np.abs(x)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
        size[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
        size[..., b] = np.abs(x[..., a] * s) + np.abs(x[..., b] * c)
        return f32_to_bf16_bits(y.astype(np.float32)) if rounded else (y, size)


def check_queries(got, bits, weight, eps, cs, interleaved):
    """Half a bf16 step of the largest value it can be (2^-8 of it, and subnormals' 2^-134), and 2^-20 of the terms."""
    want, size = normed(bits, weight, eps, cs, interleaved, rounded=False)
    early = size * 2.0 ** -20 + 2.0 ** -134
    ok = np.isfinite(want) & (np.abs(want) < 3e38)
    y = O.bf16_to_f64(got)
    assert np.all(np.isnan(y) == np.isnan(want))
    assert np.all((np.abs(y - want) <= early + (np.abs(want) + early) * 2.0 ** -8)[ok])


def heads_of(rng, n, heads, spread=3.0):
    """Heads of very different sizes, a few of zeros."""
    x = rng.standard_normal((n, heads, 128)) * np.exp(rng.standard_normal((n, heads, 1)) * spread)
    x[rng.random((n, heads)) < 0.02] = 0
    return f32_to_bf16_bits(x.astype(np.float32))


def weights_of(rng, kind, Hq, H):
    if kind == "none":
        return None, None
    if kind == "one":
        return None, (0.5 + rng.random(128)).astype(np.float32)
    shape = (lambda h: (h, 128)) if kind == "heads" else (lambda h: (128,))
    return tuple((rng.standard_normal(shape(h)) + 1).astype(np.float32) for h in (Hq, H))


@pytest.mark.parametrize("n,Hq,H,R,inter,fmt,kind,eps", [
    (1, 4, 4, 128, False, "int8", "all", 1e-6), (5, 10, 2, 64, True, "int4_factor", "heads", 1e-5),
    (64, 32, 8, 128, False, "asym_k4v8", "none", 1e-6), (33, 7, 1, 8, False, "bf16", "one", 1e-12),
    (40, 8, 8, 96, True, "k8v4_chan", "heads", 0.1), (48, 6, 3, 32, False, "int2", "all", 1e-6),
    (1500, 32, 8, 128, False, "int8", "all", 1e-6), (1339, 33, 4, 64, True, "int4_factor", "heads", 1e-6),
    (1201, 20, 10, 104, False, "bf16", "heads", 1e-6), (900, 24, 24, 128, False, "asym_k4v8", "one", 1e-6),
    (901, 64, 8, 128, True, "k8v4_chan", "none", 1e-6), (2000, 12, 12, 128, False, "int2", "heads", 1e-6),
])
def test_bits_and_codes_of_the_definition(n, Hq, H, R, inter, fmt, kind, eps):
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import HeadNorm, RopeTable
    rng = np.random.default_rng(n + R)
    rope = RopeTable(5000, rotary_dim=R, interleaved=inter)
    wq, wk = weights_of(rng, kind, Hq, H)
    norm = HeadNorm(wq, wk, eps=eps)
    seqs = 3
    seq = np.sort(rng.integers(0, seqs, n))
    slot = np.concatenate([np.arange((seq == b).sum()) for b in range(seqs)])
    pos = rng.integers(0, 5000, n)
    mb = n // 16 + 1
    table = _i(rng.permutation(seqs * mb).reshape(seqs, mb))
    q, k, v = heads_of(rng, n, Hq), heads_of(rng, n, H), heads_of(rng, n, H, 1.0)
    qkv = np.concatenate([x.reshape(n, -1) for x in (q, k, v)], 1)
    flat = _t(np.concatenate([qkv, np.zeros((n, 12), qkv.dtype)], 1))  # slices of a wider row
    at = np.cumsum([0, Hq * 128, H * 128, H * 128])
    c, ref = _cache(fmt, H, seqs * mb, np.random.default_rng(1)), _cache(fmt, H, seqs * mb, np.random.default_rng(1))
    out = torch.zeros(n, Hq, 128, dtype=torch.bfloat16, device="cuda")
    err = _i([0])
    _lib.kvq_norm_rope_append(c.desc, rope.desc, norm.desc, flat[:, at[0]:at[1]], Hq, out, flat[:, at[1]:at[2]],
                              flat[:, at[2]:at[3]], _i(pos), _i(seq), _i(slot), _lib.APPEND_QUANT, table, seqs, mb,
                              err_word=err)
    cs = rope.table.cpu().numpy().astype(np.float64)[pos]
    got = out.view(torch.int16).cpu().numpy().view(np.uint16)
    check_queries(got, q, wq, eps, cs, inter)
    key = normed(k, wk, eps, cs, inter)
    _lib.kvq_append(ref.desc, _t(key), _t(v), _i(seq), _i(slot), _lib.APPEND_QUANT, table, seqs, mb)
    torch.cuda.synchronize()
    assert err.item() == 0
    _same(c, ref)


@pytest.mark.parametrize("n", [3, 1300])
def test_sizes_beyond_float32_squares_and_no_numbers(n):
    """Heads whose squares overflow or vanish in float32, infinities and NaN, as queries and (bf16 cache) as keys."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import HeadNorm, KVCache, RopeTable
    rng = np.random.default_rng(n)
    Hq = 40
    rope, norm = RopeTable(2000), HeadNorm(weights_of(rng, "all", Hq, 1)[0], None)
    x = rng.standard_normal((n, Hq, 128))
    x *= np.resize([1e-38, 1e-30, 1e-20, 1e-9, 1.0, 1e15, 1e18, 3e19, 1e30, 7e37], Hq)[:, None]
    x[0, 20, 5], x[1, 21, 77], x[2, 22, 100] = np.inf, -np.inf, np.nan
    q = f32_to_bf16_bits(x.astype(np.float32))
    c = KVCache(1, 1, 8, 8)
    out = torch.zeros(n, Hq, 128, dtype=torch.bfloat16, device="cuda")
    pos = rng.integers(0, 2000, n)
    _lib.kvq_norm_rope_append(c.desc, rope.desc, norm.desc, _t(q), Hq, out, None, None, _i(pos), None, None,
                              _lib.APPEND_QUANT, None, 0, 0)
    cs = rope.table.cpu().numpy().astype(np.float64)[pos]
    w = norm.q_weight.cpu().numpy()
    want = normed(q, w, 1e-6, cs, False)
    got = out.view(torch.int16).cpu().numpy().view(np.uint16)
    none = np.isnan(O.bf16_to_f64(want))
    assert none.sum() >= 128
    check_queries(got, q, w, 1e-6, cs, False)
    # the same as keys: the definition's bits, where it has any
    cache = KVCache(n // 16 + 1, Hq, 16, 16)
    at = np.arange(n)
    _lib.kvq_norm_rope_append(cache.desc, rope.desc, HeadNorm(None, w).desc, None, 0, None, _t(q), _t(q), _i(pos), _i(at * 0),
                              _i(at), _lib.APPEND_QUANT, _i([np.arange(n // 16 + 1)]), 1, n // 16 + 1)
    k, v = torch.empty(n, Hq, 128, device="cuda"), torch.empty(n, Hq, 128, device="cuda")
    _lib.kvq_dequant(cache.desc, _i(at), k, v)
    got = f32_to_bf16_bits(k.cpu().numpy())
    assert np.all(np.isnan(k.cpu().numpy()) == none)
    np.testing.assert_array_equal(got[~none], want[~none])


@pytest.mark.parametrize("mode", ["RING", "STEP"])
def test_window_modes(mode):
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import HeadNorm, KVCache, RopeTable
    rng = np.random.default_rng(3)
    B, H, W, mb = 9, 3, 32, 8
    rope = RopeTable(500)
    w = weights_of(rng, "heads", 1, H)
    norm = HeadNorm(None, w[1], eps=1e-5)
    caches = [KVCache(B * mb, H, 4, 4, window=W, window_batch=B) for _ in range(2)]
    table = _i(rng.permutation(B * mb).reshape(B, mb))
    m = getattr(_lib, "APPEND_" + mode)
    for step in range(40, 44):
        pos = np.arange(B) + step
        k, v = heads_of(rng, B, H, 1.0), heads_of(rng, B, H, 1.0)
        args = (_i(np.arange(B)), _i(pos), m, table, B, mb)
        _lib.kvq_norm_rope_append(caches[0].desc, rope.desc, norm.desc, None, 0, None, _t(k), _t(v), None, *args)
        cs = rope.table.cpu().numpy().astype(np.float64)[pos]
        _lib.kvq_append(caches[1].desc, _t(normed(k, w[1], 1e-5, cs, False)), _t(v), *args)
    torch.cuda.synchronize()
    _same(*caches)


@pytest.mark.parametrize("n", [6, 4000])
def test_positions_out_of_range_and_in_place(n):
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import HeadNorm, KVCache, RopeTable
    rng = np.random.default_rng(4)
    Hq = 9
    rope, norm = RopeTable(50), HeadNorm(np.full(128, 2.0))
    q = _t(heads_of(rng, n, Hq))
    pos, err, c = np.resize([0, 49, 50, -1, 7, 8], n), _i([0]), KVCache(1, 1, 8, 8)
    out = torch.full_like(q, 5)
    call = lambda o: _lib.kvq_norm_rope_append(c.desc, rope.desc, norm.desc, q, Hq, o, None, None, _i(pos), None, None,
                                               _lib.APPEND_QUANT, None, 0, 0, err_word=err)
    call(out)
    bad = (pos < 0) | (pos > 49)
    assert err.item() == _lib.KVQ_DEVERR_POSITION and (out[bad] == 5).all() and not (out[~bad] == 5).all(-1).any()
    kept = q.clone()
    call(q)
    bits = lambda t, rows: t[rows].view(torch.int16)
    assert torch.equal(bits(q, ~bad), bits(out, ~bad)) and torch.equal(bits(q, bad), bits(kept, bad))
