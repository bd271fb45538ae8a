"""Attention mass and eviction (kvq_attn_mass, kvq_evict) against float64 and NumPy.

The mass of a token is a sum of exponentials of scores, so its relative error
is the scores' absolute error: the tolerance counts float32 half-steps of the
quantities that are summed (see _mass_tolerance).  Evictions are compared bit for bit.
"""
import numpy as np
import pytest

from harness import DeviceRun, compare_outputs, oracle_decode, oracle_state, small_workload
from layout_ref import meta_by_block, unpack_blocks
from oracle import kvq_oracle as O
from synth import make_inputs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

MASS = {
    "int8_g4": dict(),
    "int8_g1": dict(q_heads=4, kv_heads=4, len_range=(1, 200)),
    "int4_factor_g8": dict(batch=4, q_heads=16, k_bits=4, v_bits=4, channel_factor=True, outlier_channels=4),
    "k4v8_g3": dict(q_heads=6, k_bits=4, k_dist="t3", paged=True),
    "window32_int8": dict(batch=5, len_range=(1, 120), window=32),
    "window32_qint8_asym_k4": dict(batch=5, k_bits=4, len_range=(1, 120), window=32, q_bits=8, asym=True),
    "bf16_g5": dict(q_heads=10, k_bits=16, v_bits=16),
    "asym_int8_factor": dict(asym=True, channel_factor=True),
    "asym_int4": dict(asym=True, k_bits=4, v_bits=4, paged=True),
    "kchan_int8": dict(channel_factor=True, k_per_channel=True),
    "qint8_int4_factor": dict(k_bits=4, v_bits=4, channel_factor=True, q_bits=8),
    "q32_int8": dict(q_bits=32),
    "int2": dict(k_bits=2, v_bits=2), "asym_int2_factor": dict(k_bits=2, v_bits=2, asym=True, channel_factor=True),
}


def _reference(inp, lse):
    """Weights [batch, kv_heads, longest] in float64 for float32 lse, and the tolerance of each."""
    w = inp.workload
    n = int(inp.lengths.max())
    mass, tol = np.zeros((w.batch, w.kv_heads, n)), np.zeros((w.batch, w.kv_heads, n))
    for b in range(w.batch):
        st = oracle_state(inp, b)
        q = O.bf16_to_f64(inp.q[b])
        for h in range(w.kv_heads):
            k_hat, _ = O.reconstruct_sequence(st, h)
            qh = q[h * w.group:(h + 1) * w.group]
            if w.q_bits == 8:
                qh = O.effective_query(qh, None if st["c"] is None else st["c"][h])
            l = lse[b, h * w.group:(h + 1) * w.group].astype(np.float64)[:, None]
            p = np.exp(qh @ k_hat.T / np.sqrt(128.0) - l)
            # float32 half-steps (2^-24) of the score's absolute sum: 8 products of 16 terms each added one
            # after another, the low query parts and the key factor, three scale factors: below 32 of them;
            # of |lse| and of the exponent: one each, and 2^-22 of ex2
            size = np.abs(qh) @ np.abs(k_hat).T / np.sqrt(128.0)
            if w.asym:  # the code dot and the zero-point term are each larger than their sum
                size = 4 * size + 4 * np.abs(qh).sum(1, keepdims=True) * np.abs(k_hat).max(1) / np.sqrt(128.0)
            mass[b, h, :k_hat.shape[0]] = p.sum(0)
            tol[b, h, :k_hat.shape[0]] = (p * (32 * size + 2 * np.abs(l) + 8)).sum(0) * 2.0 ** -24
    return mass, tol


@pytest.mark.parametrize("name", list(MASS))
def test_mass_of_every_token(name):
    inp = make_inputs(small_workload(name, **MASS[name]))
    w = inp.workload
    run = DeviceRun(inp)
    _, lse = run.decode()
    ref, tol = _reference(inp, lse)
    n = (int(inp.lengths.max()) + 7) // 4 * 4
    start = np.random.default_rng(2).random((w.batch, w.kv_heads, n)).astype(np.float32)
    mass = torch.from_numpy(start.copy()).cuda()
    run.lib.kvq_attn_mass(run.cache.desc, run.q, w.batch, w.q_heads, torch.from_numpy(lse).cuda(), run.lens, run.table,
                          inp.max_blocks, mass, decay=0.75, err_word=run.err)
    got = mass.cpu().numpy()
    for b in range(w.batch):
        L = int(inp.lengths[b])
        want = 0.75 * start[b, :, :L].astype(np.float64) + ref[b, :, :L]
        assert np.all(np.abs(got[b, :, :L] - want) <= tol[b, :, :L] + 2.0 ** -23 * want), name
        np.testing.assert_array_equal(got[b, :, L:], start[b, :, L:])   # behind the sequence
        # every query's weights sum to 1
        total = (got[b, :, :L].astype(np.float64) - 0.75 * start[b, :, :L]).sum(1)
        np.testing.assert_allclose(total, w.group, rtol=2e-3)
    assert run.err_bits() == 0


def test_mass_is_the_same_every_time_and_empty_queries_add_nothing():
    inp = make_inputs(small_workload("mass_again", batch=7, len_range=(1, 900), paged=True))
    w = inp.workload
    run = DeviceRun(inp)
    _, lse = run.decode()
    lse_t = torch.from_numpy(lse).cuda()
    lens = run.lens.clone()
    lens[2] = 0
    lse_t[3] = -float("inf")

    def once():
        m = torch.full((w.batch, w.kv_heads, inp.max_blocks * 16), 0.5, device="cuda")
        run.lib.kvq_attn_mass(run.cache.desc, run.q, w.batch, w.q_heads, lse_t, lens, run.table, inp.max_blocks, m,
                              err_word=run.err)
        return m
    a = once()
    assert torch.equal(a, once())
    assert torch.all(a[2] == 0.5) and torch.all(a[3] == 0.5) and torch.any(a[4] != 0.5)
    assert run.err_bits() == 0


def test_mass_flags_bad_lengths_and_blocks():
    inp = make_inputs(small_workload("mass_bad", batch=4, len_range=(100, 200)))
    w = inp.workload
    run = DeviceRun(inp)
    lse = torch.zeros(w.batch, w.q_heads, device="cuda")
    cap = inp.max_blocks * 16

    def call(lens, table, stride=cap):
        m = torch.zeros(w.batch, w.kv_heads, stride, device="cuda")
        run.err.zero_()
        run.lib.kvq_attn_mass(run.cache.desc, run.q, w.batch, w.q_heads, lse, lens, table, inp.max_blocks, m,
                              err_word=run.err)
        return m, run.err_bits()
    lens = run.lens.clone()
    lens[1] = -3
    m, err = call(lens, run.table)
    assert err == run.lib.KVQ_DEVERR_SEQ_LEN and not torch.any(m[1]) and torch.any(m[0])
    lens[1] = cap + 1
    assert call(lens, run.table)[1] & run.lib.KVQ_DEVERR_SEQ_LEN
    table = run.table.clone()
    table[2, 1] = inp.num_blocks
    table[3, 0] = -7
    m, err = call(run.lens, table)
    assert err == run.lib.KVQ_DEVERR_BLOCK_ID
    assert not torch.any(m[2, :, 16:32]) and torch.all(m[2, :, :16] > 0) and not torch.any(m[3, :, :16])
    # rows shorter than the sequences: cut, nothing behind a row is touched
    m, err = call(run.lens, run.table, stride=52)
    assert err == run.lib.KVQ_DEVERR_SEQ_LEN and torch.all(m > 0)


def test_mass_of_a_long_sequence_beyond_the_table_window():
    """Many blocks per warp and units of very different lengths in one range."""
    inp = make_inputs(small_workload("mass_long", batch=3, q_heads=16, len_range=(1, 9000), k_bits=4, paged=True))
    w = inp.workload
    run = DeviceRun(inp)
    _, lse = run.decode()
    ref, tol = _reference(inp, lse)
    mass = torch.zeros(w.batch, w.kv_heads, inp.max_blocks * 16, device="cuda")
    run.lib.kvq_attn_mass(run.cache.desc, run.q, w.batch, w.q_heads, torch.from_numpy(lse).cuda(), run.lens, run.table,
                          inp.max_blocks, mass, err_word=run.err)
    got = mass.cpu().numpy()[:, :, :ref.shape[2]]
    assert np.all(np.abs(got - ref) <= tol + 2.0 ** -23 * ref) and run.err_bits() == 0


# ------------------------------------------------------------------ eviction

def choose(mass, L, keep, first, recent, window, pos=None, next_pos=None):
    """The source of every remaining slot of one row, by the definition."""
    Lq = max(L - window, 0)
    n = min(max(L - keep, 0), Lq)
    if window:
        n -= n % window
    K = Lq - n
    p = np.arange(Lq) if pos is None else pos[:Lq]
    protected = (np.arange(Lq) < first) | (p >= (L if next_pos is None else next_pos) - recent)
    m = mass[:Lq].astype(np.float64)
    # among the protected ones the lowest slot counts alone
    key = [(0, 0.0, False, s) if protected[s] else (1, np.inf if np.isnan(m[s]) else -m[s], np.isnan(m[s]), s)
           for s in range(Lq)]
    kept = np.zeros(Lq, bool)
    for k in sorted(key)[:K]:
        kept[k[3]] = True
    src = np.arange(K)
    src[~kept[:K]] = np.nonzero(kept[K:])[0] + K
    return np.concatenate([src, np.arange(K, L - n) + n]).astype(np.int32), K


EVICT = {
    "int8": dict(), "int4": dict(k_bits=4, v_bits=4), "asym_k4v8": dict(k_bits=4, v_bits=8, asym=True),
    "k8v4": dict(k_bits=8, v_bits=4), "asym_int8_factor": dict(asym=True, channel_factor=True),
    "bf16": dict(k_bits=16, v_bits=16), "window32": dict(window=32, batch=4), "kchan": dict(channel_factor=True,
                                                                                           k_per_channel=True),
}


def _logical(run, inp):
    """Everything stored, by (head, physical block, token)."""
    w, p = inp.workload, run.pools()
    k = unpack_blocks(p["k_codes"], w.k_bits, True, w.kv_heads, asym=w.asym)
    v = unpack_blocks(p["v_codes"], w.v_bits, False, w.kv_heads, asym=w.asym)
    meta = [] if w.k_bits == 16 else [m.copy() for m in meta_by_block(p["meta"], w.kv_heads, w.asym).values()]
    return [k, v] + meta


@pytest.mark.parametrize("name", list(EVICT))
@pytest.mark.parametrize("in_place", [False, True])
def test_evicted_cache_bit_for_bit(name, in_place):
    inp = make_inputs(small_workload(name, **dict(dict(batch=5, len_range=(60, 400), paged=True), **EVICT[name])))
    w = inp.workload
    run = DeviceRun(inp)
    rng = np.random.default_rng(11)
    cap = inp.max_blocks * 16 + 4 + w.window
    L = inp.lengths.astype(int)
    mass = rng.choice([0.0, 0.5, 1.0, 2.5, 7.0], (w.batch, w.kv_heads, cap)).astype(np.float32)   # many ties
    mass[0, 0, 3:30] = np.nan
    mass[0, 0, 40:45] = np.inf
    mass[1, 0] = -np.inf
    mass[1, 1, ::2] = -0.0
    keep = np.array([L[0] // 2, L[1] - 1, 17, L[3] + 5, 0, 33][:w.batch], dtype=np.int32)
    first, recent = 3, 9
    pos = np.stack([np.stack([rng.permutation(cap) for _ in range(w.kv_heads)]) for _ in range(w.batch)]).astype(np.int32)
    nxt = np.full(w.batch, cap - 20, dtype=np.int32)
    before = _logical(run, inp)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    m_in, p_in = t(mass), t(pos)
    m_out = m_in if in_place else torch.full_like(m_in, -5.0)
    p_out = p_in if in_place else torch.full_like(p_in, -5)
    src = torch.full_like(p_in, -7)
    new = torch.zeros(w.batch, dtype=torch.int32, device="cuda")
    run.lib.kvq_evict(run.cache.desc, m_in, m_out, run.lens, t(keep), run.table, w.batch, inp.max_blocks, src, new,
                      protect_first=first, protect_recent=recent, token_pos=p_in, token_pos_out=p_out, next_pos=t(nxt),
                      err_word=run.err)
    assert run.err_bits() == 0
    want = [x.copy() for x in before]
    for b in range(w.batch):
        for h in range(w.kv_heads):
            s, K = choose(mass[b, h], L[b], keep[b], first, recent, w.window, pos[b, h], nxt[b])
            n = len(s)
            assert int(new[b]) == n
            np.testing.assert_array_equal(src[b, h, :n].cpu().numpy(), s)
            np.testing.assert_array_equal(m_out[b, h, :n].cpu().numpy(), mass[b, h][s])
            np.testing.assert_array_equal(p_out[b, h, :n].cpu().numpy(), pos[b, h][s])
            assert torch.all(src[b, h, n:] == -7)
            np.testing.assert_array_equal(m_out[b, h, n:].cpu().numpy(), mass[b, h, n:] if in_place else -5.0)
            dst, tab = np.arange(K), inp.block_table[b]
            for x, y in zip(want, before):
                x[tab[dst // 16], h, dst % 16] = y[tab[s[:K] // 16], h, s[:K] % 16]
    for x, y in zip(_logical(run, inp), want):
        np.testing.assert_array_equal(x.view(np.uint32) if x.dtype == np.float32 else x,
                                      y.view(np.uint32) if y.dtype == np.float32 else y)


@pytest.mark.parametrize("L,keep", [(1, 1), (1, 0), (16, 15), (17, 16), (33, 1), (50000, 25000), (70001, 1000)])
def test_eviction_of_one_row(L, keep):
    """Lengths of one, block borders, and more moves than one walk matches; the heavy tokens lie at the end."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache
    rng = np.random.default_rng(L)
    nb = (L + 15) // 16
    c = KVCache(nb, 1, 8, 8)
    codes = rng.integers(1, 256, nb * 2048).astype(np.uint8)
    c.k_codes.copy_(torch.from_numpy(codes).cuda())
    c.v_codes.copy_(torch.from_numpy(codes[::-1].copy()).cuda())
    mass = (np.arange(L) + rng.random(L)).astype(np.float32)[None, None]
    new = torch.zeros(1, dtype=torch.int32, device="cuda")
    src = torch.zeros(1, 1, L, dtype=torch.int32, device="cuda")
    i = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
    _lib.kvq_evict(c.desc, torch.from_numpy(mass).cuda(), None, i([L]), i([keep]), torch.arange(nb).int().cuda()[None],
                   1, nb, src, new)
    s, K = choose(mass[0, 0], L, keep, 0, 0, 0)
    assert int(new) == len(s)
    np.testing.assert_array_equal(src[0, 0, :len(s)].cpu().numpy(), s)
    for pool, old, is_key in ((c.k_codes, codes, True), (c.v_codes, codes[::-1], False)):
        got = unpack_blocks(pool.cpu().numpy(), 8, is_key, 1)[:, 0].reshape(-1, 128)
        ref = unpack_blocks(np.ascontiguousarray(old), 8, is_key, 1)[:, 0].reshape(-1, 128)
        np.testing.assert_array_equal(got[:K], ref[s])
        np.testing.assert_array_equal(got[K:], ref[K:])


@pytest.mark.parametrize("L,keep,order", [(32768, 20000, "spread"), (32769, 20000, "spread"), (60000, 30000, "rising"),
                                          (60000, 30000, "equal"), (40000, 8000, "steps")])
def test_sums_and_positions_follow_in_place(L, keep, order):
    """Rows about and beyond what stays on the chip, more moves than one walk matches, many equal sums."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache
    rng = np.random.default_rng(L + keep)
    nb = (L + 15) // 16
    c = KVCache(nb, 2, 4, 4)
    x = dict(spread=rng.random((2, L)), rising=np.arange(2 * L).reshape(2, L), equal=np.ones((2, L)),
             steps=rng.integers(0, 4, (2, L)))[order].astype(np.float32)
    pos = np.sort(rng.permutation(2 * L)[:L]).astype(np.int32)
    i = lambda v: torch.as_tensor(v, dtype=torch.int32).cuda()
    mass = torch.from_numpy(x).cuda()[None].contiguous()
    tp = i(np.stack([pos, pos]))[None].contiguous()
    new = torch.zeros(1, dtype=torch.int32, device="cuda")
    src = torch.zeros(1, 2, L, dtype=torch.int32, device="cuda")
    _lib.kvq_evict(c.desc, mass, mass, i([L]), i([keep]), torch.arange(nb).int().cuda()[None], 1, nb, src, new,
                   token_pos=tp, token_pos_out=tp, next_pos=i([2 * L]))
    for h in range(2):
        s, _ = choose(x[h], L, keep, 0, 0, 0, pos, 2 * L)
        assert int(new) == len(s)
        np.testing.assert_array_equal(src[0, h, :len(s)].cpu().numpy(), s)
        np.testing.assert_array_equal(mass[0, h, :len(s)].cpu().numpy(), x[h][s])
        np.testing.assert_array_equal(tp[0, h, :len(s)].cpu().numpy(), pos[s])
        np.testing.assert_array_equal(mass[0, h, len(s):].cpu().numpy(), x[h][len(s):])


def test_eviction_flags_bad_lengths_and_blocks():
    inp = make_inputs(small_workload("evict_bad", batch=3, len_range=(100, 200)))
    w = inp.workload
    run = DeviceRun(inp)
    cap = inp.max_blocks * 16
    rng = np.random.default_rng(0)
    mass = torch.from_numpy(rng.random((3, w.kv_heads, cap)).astype(np.float32)).cuda()
    src, new = torch.zeros(3, w.kv_heads, cap, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32).cuda()
    i = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
    run.lib.kvq_evict(run.cache.desc, mass, None, i([-4, 90, cap + 9]), i([10, -1, cap + 50]), run.table, 3,
                      inp.max_blocks, src, new, err_word=run.err)
    assert run.err_bits() == run.lib.KVQ_DEVERR_SEQ_LEN and new.tolist() == [0, 0, cap]
    run.err.zero_()
    table = run.table.clone()
    table[:, 5] = -1                       # a source block that is not there: its tokens are not moved
    before = run.cache.k_codes.clone()
    run.lib.kvq_evict(run.cache.desc, mass, None, run.lens, i([40, 40, 40]), table, 3, inp.max_blocks, src, new,
                      err_word=run.err)
    assert run.err_bits() == run.lib.KVQ_DEVERR_BLOCK_ID and not torch.equal(before, run.cache.k_codes)


@pytest.mark.parametrize("fmt", [dict(), dict(k_bits=4, v_bits=4, channel_factor=True), dict(window=16)])
def test_a_run_of_decode_mass_and_eviction(fmt):
    """Decode, add the weights, evict, append behind the kept tokens, decode again: attention over the kept
    tokens and the new one, and weights that are kept with their tokens."""
    inp = make_inputs(small_workload("evict_run", **dict(dict(batch=3, len_range=(150, 300), paged=True), **fmt)))
    w = inp.workload
    run = DeviceRun(inp)
    lib = run.lib
    _, lse = run.decode()
    cap = inp.max_blocks * 16 + w.window
    mass = torch.zeros(w.batch, w.kv_heads, cap, device="cuda")
    lib.kvq_attn_mass(run.cache.desc, run.q, w.batch, w.q_heads, torch.from_numpy(lse).cuda(), run.lens, run.table,
                      inp.max_blocks, mass, err_word=run.err)
    before = mass.cpu().numpy()
    keep = (run.lens // 2).int()
    src = torch.zeros(w.batch, w.kv_heads, cap, dtype=torch.int32, device="cuda")
    new = torch.zeros(w.batch, dtype=torch.int32, device="cuda")
    lib.kvq_evict(run.cache.desc, mass, mass, run.lens, keep, run.table, w.batch, inp.max_blocks, src, new,
                  protect_first=4, protect_recent=20, err_word=run.err)
    out, lse2 = run.decode(lens=new)
    assert run.err_bits() == 0
    new, src = new.cpu().numpy(), src.cpu().numpy()
    G = w.group
    for b in range(w.batch):
        st = oracle_state(inp, b)
        for h in range(w.kv_heads):
            s = src[b, h, :new[b]]
            assert len(set(s)) == len(s) and set(range(4)) <= set(s)
            assert set(range(inp.lengths[b] - 20, inp.lengths[b])) <= set(s)
            np.testing.assert_array_equal(mass[b, h, :new[b]].cpu().numpy(), before[b, h][s])
            k, v = O.reconstruct_sequence(st, h)
            o, l = O.attention(O.bf16_to_f64(inp.q[b, h * G:(h + 1) * G]), k[s], v[s])
            assert np.max(np.abs(out[b, h * G:(h + 1) * G] - o)) <= 2e-3
            assert np.max(np.abs(lse2[b, h * G:(h + 1) * G] - l)) <= 2e-3


def test_captured_eviction_is_replayed_on_new_sums():
    inp = make_inputs(small_workload("evict_graph", batch=2, len_range=(80, 160)))
    w = inp.workload
    run = DeviceRun(inp)
    cap = inp.max_blocks * 16
    mass = torch.zeros(2, w.kv_heads, cap, device="cuda")
    src, new = torch.zeros(2, w.kv_heads, cap, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32).cuda()
    keep = (run.lens // 3).int()
    lse = torch.zeros(2, w.q_heads, device="cuda")

    def call():
        run.lib.kvq_attn_mass(run.cache.desc, run.q, 2, w.q_heads, lse, run.lens, run.table, inp.max_blocks, mass,
                              decay=0.0)
        run.lib.kvq_evict(run.cache.desc, mass, None, run.lens, keep, run.table, 2, inp.max_blocks, src, new)
    call()  # launches once outside the capture
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for _ in range(2):
        run.q.normal_()
        g.replay()
        torch.cuda.synchronize()
        m = mass.cpu().numpy()
        for b in range(2):
            for h in range(w.kv_heads):
                want, _ = choose(m[b, h], int(inp.lengths[b]), int(keep[b]), 0, 0, 0)
                np.testing.assert_array_equal(src[b, h, :len(want)].cpu().numpy(), want)
