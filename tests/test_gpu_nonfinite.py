"""Keys and values that are not finite, and scales below float32's normal range: what one token's vector stores is its
own alone.  The rule: NaN counts as nothing in the largest value and stores code 0; under an infinite scale every code is
0; codes stay within their bounds whatever the quotient."""
import numpy as np
import pytest

from layout_ref import meta_by_block, unpack_blocks
from oracle import kvq_oracle as O
from synth import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

TOP = {8: 127, 4: 7}
LOW = {8: -127, 4: -8}
FORMATS = {"int8": dict(k_bits=8, v_bits=8), "int4": dict(k_bits=4, v_bits=4), "k4v8": dict(k_bits=4, v_bits=8),
           "k8v4": dict(k_bits=8, v_bits=4), "asym_int8": dict(k_bits=8, v_bits=8, asym=True),
           "asym_int4": dict(k_bits=4, v_bits=4, asym=True)}


def _t(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def _i(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def _pools(c):
    return [t.view(torch.uint8).cpu().numpy() for t in (c.k_codes, c.v_codes, c.meta)]


def symmetric(x, bits):
    """Codes and float32 scales of float32 vectors along the last axis, by the rule above."""
    x = x.astype(np.float64)
    a = np.nanmax(np.abs(x), -1, keepdims=True)
    with np.errstate(all="ignore"):
        s = np.where(a == 0, 1.0, (a / TOP[bits])).astype(np.float32)
        q = np.rint(x / s.astype(np.float64))
    return np.where(np.isnan(q), 0, np.clip(q, LOW[bits], TOP[bits])).astype(np.int32), s[..., 0]


def bad_rows(rng, n, H):
    """Vectors [n, H, 128] of bf16 bits with NaN and infinities in some rows (their numbers come back), each kind alone."""
    x = rng.standard_normal((n, H, 128)).astype(np.float32)
    rows = np.array([3, 7, 8, 12, 17, n - 2])
    x[3, :, 5] = np.nan
    x[7, 0, 100] = np.inf
    x[8, H - 1, 0:4] = np.nan          # one lane's four
    x[12, :, [0, 64, 127]] = -np.inf
    x[17, 0, ::2] = np.nan
    x[n - 2, :, 31], x[n - 2, :, 32] = np.inf, np.nan
    return f32_to_bf16_bits(x), rows


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_append_stores_bad_values_in_their_own_place(fmt):
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache
    rng = np.random.default_rng(1)
    n, H = 40, 2
    k, rows = bad_rows(rng, n, H)
    v, _ = bad_rows(rng, n, H)
    got = []
    for zero in (False, True):
        kk, vv = k.copy(), v.copy()
        if zero:
            kk[rows], vv[rows] = 0, 0
        c = KVCache(3, H, **FORMATS[fmt])
        _lib.kvq_append(c.desc, _t(kk), _t(vv), _i(np.zeros(n)), _i(np.arange(n)), _lib.APPEND_QUANT,
                        _i([[2, 0, 1]]), 1, 3)
        got.append(_pools(c))
    blocks = np.array([2, 0, 1])
    at = (blocks[np.arange(n) // 16], np.arange(n) % 16)
    others = np.setdiff1d(np.arange(n), rows)
    for i, (name, x) in enumerate((("k_bits", k), ("v_bits", v))):
        bits, asym = FORMATS[fmt][name], FORMATS[fmt].get("asym", False)
        codes = [unpack_blocks(g[i], bits, i == 0, H, asym).transpose(0, 2, 1, 3)[at] for g in got]
        np.testing.assert_array_equal(codes[0][others], codes[1][others])
        if not asym:
            want, s = symmetric(O.bf16_to_f64(x), bits)
            np.testing.assert_array_equal(codes[0], want)
            scale = meta_by_block(got[0][2].view(np.float32), H)["v_scale" if i else "k_scale"]
            np.testing.assert_array_equal(scale.transpose(0, 2, 1)[at], s)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("n", [40, 1000])     # a warp a vector; windows of 16 rows
def test_rotary_write_as_the_append_of_the_rotated_rows(fmt, n):
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache, RopeTable
    rng = np.random.default_rng(2)
    H, Hq, blocks = 3, 26, 64
    assert n < 1000 or n * (Hq + 2 * H) >= 3 * 152 * 64
    k, _ = bad_rows(rng, n, H)
    v, _ = bad_rows(rng, n, H)
    q = f32_to_bf16_bits(rng.standard_normal((n, Hq, 128)).astype(np.float32))
    rope = RopeTable(2000)
    pos = 1 + rng.integers(0, 1999, n)
    cs = rope.table.cpu().numpy().astype(np.float64)[pos][:, None]
    x = O.bf16_to_f64(k)
    with np.errstate(all="ignore"):
        y = np.concatenate([x[..., :64] * cs[..., 0] - x[..., 64:] * cs[..., 1],
                            x[..., :64] * cs[..., 1] + x[..., 64:] * cs[..., 0]], -1).astype(np.float32)
    y[np.isnan(y)] = np.nan
    table = _i(rng.permutation(blocks)[None])
    a, b = (KVCache(blocks, H, **FORMATS[fmt]) for _ in range(2))
    out = torch.empty(n, Hq, 128, dtype=torch.bfloat16, device="cuda")
    zero, slot = _i(np.zeros(n)), _i(np.arange(n))
    _lib.kvq_rope_append(a.desc, rope.desc, _t(q), Hq, out, _t(k), _t(v), _i(pos), zero, slot, _lib.APPEND_QUANT, table, 1,
                         blocks)
    _lib.kvq_append(b.desc, _t(f32_to_bf16_bits(y)), _t(v), zero, slot, _lib.APPEND_QUANT, table, 1, blocks)
    for p, r in zip(_pools(a), _pools(b)):
        np.testing.assert_array_equal(p, r)
    assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("rope", [False, True])
def test_codes_stay_within_their_bounds_under_subnormal_scales(bits, rope):
    """Keys over a large key factor: largest values of a few steps of 2^-149, whose scale is one step or 0."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache, RopeTable
    rng = np.random.default_rng(3)
    n, top = 32, TOP[bits]
    steps = np.concatenate([[1, 2, 3, 10, 50, 63, 64, 90, 127, 128, 188, 190, 191, 200, 255], 1 + np.arange(17) * 14])[:n]
    x = (rng.integers(-8, 9, (n, 1, 128)) * (steps[:, None, None] // 8)).astype(np.float64)
    x[:, 0, 1], x[:, 0, 2], x[:, 0, 3] = steps, -steps, 0
    k = f32_to_bf16_bits((x * 2.0 ** -49).astype(np.float32))
    kq = O.bf16_to_f64(k) * 2.0 ** -100       # exact: multiples of 2^-149
    np.testing.assert_array_equal(kq, x * 2.0 ** -149)
    c = KVCache(2, 1, k_bits=bits, v_bits=bits, channel_factor=np.full((1, 128), 2.0 ** 100, np.float32))
    table, seq, pos = _i([[0, 1]]), _i(np.zeros(n)), _i(np.arange(n))
    if rope:      # position 0: cosine 1, sine 0
        turns = RopeTable(1)
        _lib.kvq_rope_append(c.desc, turns.desc, None, 0, None, _t(k), _t(k), seq, seq, pos, _lib.APPEND_QUANT,
                             table, 1, 2)
    else:
        _lib.kvq_append(c.desc, _t(k), _t(k), seq, pos, _lib.APPEND_QUANT, table, 1, 2)
    want, s = symmetric(kq.astype(np.float32), bits)
    assert (s == 0).any() and (s == 2.0 ** -149).any() and (np.abs(kq) > top * s[..., None].astype(np.float64)).any()
    codes = unpack_blocks(_pools(c)[0], bits, True, 1).transpose(0, 2, 1, 3).reshape(n, 1, 128)
    np.testing.assert_array_equal(codes, want)


SHARED = {
    # query vectors of a group: few (16-vector tiles), many (tcgen05, one and two warpgroups' worth)
    "tiles_int8": dict(batch=6), "tiles_asym_int4_factor": dict(batch=6, k_bits=4, v_bits=4, asym=True, channel_factor=True),
    "tiles_int2": dict(batch=6, k_bits=2, v_bits=2), "tiles_q32_int8": dict(batch=20, q_bits=32, q_heads=16),
    "int8": dict(batch=20), "k8v4": dict(batch=40, v_bits=4, q_heads=16), "asym_k4v8": dict(batch=20, k_bits=4, asym=True),
    "asym_int8": dict(batch=40, q_heads=16, asym=True), "int4_factor": dict(batch=20, k_bits=4, v_bits=4, channel_factor=True),
    "asym_int4_factor": dict(batch=20, k_bits=4, v_bits=4, asym=True, channel_factor=True),
    "asym_int2": dict(batch=20, k_bits=2, v_bits=2, asym=True),
}


@pytest.mark.parametrize("fmt", list(SHARED))
@pytest.mark.parametrize("bad", ["inf", "-inf", "nan", "1e36"])
def test_a_prefix_token_reaches_only_the_sequences_that_hold_it(fmt, bad):
    """Token 150 of a shared prefix of 208 has a value that is not finite, or far out of the others' range: sequences that
    end before it are as kvq_decode has them; for those that hold it the log-sum-exp and what is not finite are."""
    from harness import DeviceRun, small_workload
    from test_gpu_shared import decode_shared, shared_inputs
    w = small_workload("shared_masked", **dict(dict(len_range=(300, 420), paged=True), **SHARED[fmt]))
    groups = [(0, w.batch, 13)]
    inp = shared_inputs(w, groups)
    lead = int(np.argmax(inp.lengths))
    value = np.array([float(bad)], np.float32)
    for b in range(w.batch):
        at = inp.seq_offsets[b] + 150
        if bad == "nan":       # every dim: no number is left to give a scale
            inp.v[at] = f32_to_bf16_bits(value)[0]
        else:
            inp.v[at, :, 77] = f32_to_bf16_bits(value)[0]
    assert inp.lengths[lead] > 208
    run = DeviceRun(inp)
    lens = np.array(inp.lengths)
    before = np.arange(w.batch) % 3 != 1
    lens[before] = np.resize([149, 150, 37, 1, 144, 100, 64, 129], int(before.sum()))
    if w.k_bits == 2:          # the token's block has one scale: only what lies before the block is apart from it
        lens[before] = np.minimum(lens[before], 144)
    lens_t = torch.from_numpy(lens.astype(np.int32)).cuda()
    ref, ref_lse = run.decode(lens=lens_t)
    out, lse = decode_shared(run, groups, lens=lens_t)
    assert np.isfinite(ref[before]).all() and run.err_bits() == 0
    np.testing.assert_allclose(out[before], ref[before], rtol=0, atol=2e-3)
    np.testing.assert_allclose(lse, ref_lse, rtol=0, atol=2e-3)
    out, ref = out[~before], ref[~before]
    np.testing.assert_array_equal(np.isfinite(out), np.isfinite(ref))
    if bad == "1e36":
        # the token's weight times its value scale decides: one fp16 rounding (2^-11) in each call; under a key factor
        # kvq_decode's query is one fp16 part, and its score off by 2^-11 of the products' sum, below 12 here
        tol = 2.0 ** -10 + (12 * 2.0 ** -11 if w.channel_factor else 0.0)
        # an asymmetric 2-bit group's 16 tokens all have the scale s = 10^36 / 3, and code 0 as 2 s from the middle code's
        # value: 2^-11 of each weight times 2 s, the weights' sum below 1, in each call
        atol = 2.0 ** -10 * 2 / 3 * 1e36 if w.k_bits == 2 and w.asym else 0.0
        assert np.all(np.abs(out - ref) <= tol * np.abs(ref).max(-1, keepdims=True) + atol)
    elif not (w.k_bits == 2 and bad == "nan"):      # a 2-bit group's scale comes from its numbers
        assert not np.isfinite(ref).any()


@pytest.mark.parametrize("kw", [dict(k_bits=16, v_bits=16, q_heads=14), dict(k_bits=16, v_bits=16, q_heads=14, paged=True),
                                dict(window=32), dict(window=32, k_bits=4, asym=True)])
@pytest.mark.parametrize("batch", [5, 20])
def test_slots_without_a_token_hold_anything(kw, batch):
    """Block stores and rings full of NaN before the tokens are written: lengths of 1, inside and at the end of a block, in
    kvq_decode, kvq_decode_shared and kvq_attn_mass as from zeroed memory."""
    from harness import DeviceRun, small_workload
    from quantized_kv_cache_07_gb300 import _lib
    from synth import make_inputs
    from test_gpu_shared import decode_shared
    w = small_workload("stale", **dict(dict(batch=batch, len_range=(33, 120)), **kw))
    window = w.window
    inp = make_inputs(w)
    run = DeviceRun(inp)
    if window:       # rings that are not full: 1 to 31 tokens each
        short = torch.from_numpy(np.resize([1, 5, 16, 17, 31], batch).astype(np.int32)).cuda()
    else:            # prefixes of 2 blocks of which less is held
        short = torch.from_numpy(np.resize([1, 19, 16, 17, 8], batch).astype(np.int32)).cuda()
    got = []
    for stale in (0, 0x7FC1):
        for t in (run.cache.k_codes, run.cache.v_codes, run.cache.meta, run.cache.k_window, run.cache.v_window):
            if t is not None:
                t.view(torch.int16).fill_(stale)
        n = int(short.sum())
        seq = torch.repeat_interleave(torch.arange(batch, device="cuda").int(), short.long())
        pos = (torch.arange(n, device="cuda") - torch.repeat_interleave(short.cumsum(0) - short, short.long())).int()
        g = torch.Generator(device="cuda").manual_seed(1)
        rows = torch.randn(2, 40, w.kv_heads, 128, generator=g, device="cuda").bfloat16()
        k, v = rows[0][pos.long()], rows[1][pos.long()]      # the same tokens in every sequence: a shared prefix
        table = run.table.clone()
        table[:, :2] = table[0, :2]
        one = torch.ones_like(seq, dtype=torch.bool) if window else seq == 1        # the longest, for all
        _lib.kvq_append(run.cache.desc, k[one].contiguous(), v[one].contiguous(), seq[one].contiguous(),
                        pos[one].contiguous(), _lib.APPEND_RING if window else _lib.APPEND_QUANT, table, batch, inp.max_blocks)
        run.table = table
        o, l = run.decode(lens=short)
        groups = [(0, batch, 0 if window else 2)]
        so, sl = decode_shared(run, groups, lens=short)
        mass = torch.zeros(batch, w.kv_heads, 64, device="cuda")
        _lib.kvq_attn_mass(run.cache.desc, run.q, batch, w.q_heads, torch.from_numpy(l).cuda(), short, table, inp.max_blocks, mass)
        got.append((o, l, so, sl, mass.cpu().numpy()))
    for a, b in zip(*got):
        assert np.isfinite(b).all()
        np.testing.assert_array_equal(a, b)
