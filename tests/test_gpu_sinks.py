"""Attention with sinks and a sliding window (kvq_decode_sinks, kvq_prefill_sinks) against the float64 oracle.

A query at position p sees tokens i <= p with i < sinks or i > p - span: the oracle gets those tokens
alone.  Every test runs on a block table whose other blocks have been freed (-1).  Tolerances are
those of kvq_decode (harness.TOL; bf16 outputs add half a step).
"""
import numpy as np
import pytest

from harness import DeviceRun, TOL, bf16_half_ulp, oracle_state, small_workload
from oracle import kvq_oracle as O
from synth import f32_to_bf16_bits, make_inputs, query_rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

FORMATS = {
    "int8_g4": dict(), "int8_g1_paged": dict(q_heads=4, kv_heads=4, paged=True),
    "int4_factor_g8": dict(q_heads=16, k_bits=4, v_bits=4, channel_factor=True),
    "k4v8_g3": dict(q_heads=6, k_bits=4, paged=True), "k8v4_g5": dict(q_heads=10, v_bits=4, paged=True),
    "bf16_g7": dict(q_heads=14, k_bits=16, v_bits=16), "bf16_g1": dict(q_heads=2, k_bits=16, v_bits=16),
    "asym_int8": dict(asym=True, outlier_channels=4), "asym_int4_factor": dict(asym=True, k_bits=4, v_bits=4,
                                                                              channel_factor=True),
    "kchan_int8": dict(channel_factor=True, k_per_channel=True), "qint8_asym_k8v4": dict(q_bits=8, asym=True, v_bits=4),
    "q32_int8": dict(q_bits=32), "q32_asym_k4v8": dict(q_bits=32, asym=True, k_bits=4),
    "int2": dict(k_bits=2, v_bits=2), "asym_int2_g8": dict(k_bits=2, v_bits=2, asym=True, q_heads=16),
    "q32_int2": dict(k_bits=2, v_bits=2, q_bits=32),
}
WINDOWS = {"window32_int8": dict(window=32), "window16_asym_k4v8": dict(window=16, k_bits=4, asym=True, q_heads=16),
           "window128_bf16": dict(window=128, k_bits=16, v_bits=16)}
# the window ends inside a block, at its border, reaches into the sinks, is a single token; sinks of none, part of a
# block, whole blocks, more than there are tokens
SPANS = [(4, 100), (0, 64), (16, 33), (5, 1), (40, 16), (300, 20), (3, 1000)]


def seen(L, sinks, span):
    i = np.arange(L)
    return (i < sinks) | (i >= L - span)


def freed(table, lens, low, sinks, window=0):
    """The table without the blocks that no query of lengths low..lens sees."""
    t = table.clone()
    for b, L in enumerate(lens):
        stored = max(int(L) - window, 0)
        for j in range(t.shape[1]):
            used = 16 * j < stored and (16 * j < sinks or 16 * (j + 1) > low[b])
            if not used:
                t[b, j] = -1
    return t


def decode(run, sinks, span, lens=None, table=None, out_fp32=True, lse=True, stream_ctas=0, ws=None, stream=None):
    from quantized_kv_cache_07_gb300.cache import DecodeWorkspace
    w = run.inp.workload
    lens = run.lens if lens is None else lens
    out = torch.full((w.batch, w.q_heads, 128), float("nan"), device="cuda",
                     dtype=torch.float32 if out_fp32 else torch.bfloat16)
    l = torch.full((w.batch, w.q_heads), float("nan"), device="cuda") if lse else None
    ws = ws or DecodeWorkspace(run.cache, w.batch, w.q_heads, stream_ctas)
    run.lib.kvq_decode_sinks(run.cache.desc, run.q, w.batch, w.q_heads, lens, run.table if table is None else table,
                             run.inp.max_blocks, sinks, span, out, lse=l, workspace=ws.buf, workspace_bytes=ws.nbytes,
                             stream_ctas=stream_ctas, err_word=run.err, stream=stream)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), None if l is None else l.cpu().numpy()


class Oracle:
    def __init__(self, inp):
        self.inp = inp
        self.kv = [[O.reconstruct_sequence(oracle_state(inp, b), h) for h in range(inp.workload.kv_heads)]
                   for b in range(inp.workload.batch)]
        self.c = None if inp.channel_factor is None else inp.channel_factor.astype(np.float64)

    def __call__(self, b, h, q, L, sinks, span):
        """q [G, 128] float64 over the first L tokens of sequence b."""
        if self.inp.workload.q_bits == 8:
            q = O.effective_query(q, None if self.c is None else self.c[h])
        k, v = self.kv[b][h]
        s = seen(L, sinks, span)
        return O.attention(q, k[:L][s], v[:L][s])


def worst(out, lse, ref_o, ref_l, bf16=False):
    tol = TOL + (bf16_half_ulp(ref_o) if bf16 else 0.0)
    w = float(np.max(np.abs(out - ref_o) / tol))
    return w if lse is None else max(w, float(np.max(np.abs(lse - ref_l)) / TOL))


@pytest.mark.parametrize("fmt", list(FORMATS) + list(WINDOWS))
def test_decode_matches_the_oracle(fmt):
    kw = FORMATS[fmt] if fmt in FORMATS else WINDOWS[fmt]
    w = small_workload(fmt, **dict(dict(batch=5, len_range=(150, 420)), **kw))
    inp = make_inputs(w, 0)
    run, ref, G = DeviceRun(inp), Oracle(inp), w.group
    for sinks, span in SPANS:
        span = max(span, w.window)
        table = freed(run.table, inp.lengths, [int(L) - span for L in inp.lengths], sinks, w.window)
        o = np.zeros((w.batch, w.q_heads, 128))
        l = np.zeros((w.batch, w.q_heads))
        for b in range(w.batch):
            q = O.bf16_to_f64(inp.q[b])
            for h in range(w.kv_heads):
                g = slice(h * G, (h + 1) * G)
                o[b, g], l[b, g] = ref(b, h, q[g], int(inp.lengths[b]), sinks, span)
        for ctas in (0, 1, 7):
            assert worst(*decode(run, sinks, span, table=table, stream_ctas=ctas), o, l) <= 1.0, (sinks, span, ctas)
        assert worst(*decode(run, sinks, span, table=table, out_fp32=False, lse=False), o, l, True) <= 1.0
    assert run.err_bits() == 0


@pytest.mark.parametrize("fmt", ["int8_g4", "asym_int4_factor", "bf16_g7", "int2"])
def test_short_sequences(fmt):
    """Lengths of zero, one, the sinks, the window, both, one more: with span >= L the result is kvq_decode's."""
    w = small_workload(fmt, **dict(dict(batch=9, len_range=(300, 420)), **FORMATS[fmt]))
    inp = make_inputs(w, 1)
    run, ref, G = DeviceRun(inp), Oracle(inp), w.group
    sinks, span = 20, 40
    lens = np.array([0, 1, 16, 20, 40, 60, 61, 80, inp.lengths[8]])
    lens_t = torch.from_numpy(lens.astype(np.int32)).cuda()
    out, lse = decode(run, sinks, span, lens=lens_t)
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[0]))
    for b in range(1, 9):
        q = O.bf16_to_f64(inp.q[b])
        for h in range(w.kv_heads):
            g = slice(h * G, (h + 1) * G)
            assert worst(out[b, g], lse[b, g], *ref(b, h, q[g], int(lens[b]), sinks, span)) <= 1.0, b
    out, lse = decode(run, 0, 10 ** 6, lens=lens_t)
    o, l = run.decode(lens=lens_t)
    np.testing.assert_allclose(out, o, rtol=0, atol=TOL)
    np.testing.assert_allclose(lse[1:], l[1:], rtol=0, atol=TOL)
    assert run.err_bits() == 0


def _poison(run, b, positions, value):
    """Keys and values of `value` at these positions of sequence b."""
    w, n = run.inp.workload, len(positions)
    x = torch.full((n, w.kv_heads, 128), value, dtype=torch.bfloat16, device="cuda")
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    run.lib.kvq_append(run.cache.desc, x, x, i([b] * n), i(list(positions)), run.lib.APPEND_QUANT, run.table, w.batch,
                       run.inp.max_blocks)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("fmt", ["int8_g4", "int4_factor_g8", "asym_int8", "q32_asym_k4v8", "bf16_g7", "qint8_asym_k8v4"])
def test_hidden_tokens_have_no_effect(fmt, value):
    """Not-a-numbers, infinities and the largest values in hidden tokens of the blocks that are read: same bits."""
    w = small_workload(fmt, **dict(dict(batch=2, len_range=(200, 300)), **FORMATS[fmt]))
    inp = make_inputs(w, 2)
    run = DeviceRun(inp)
    for sinks, span in ((5, 70), (0, 33), (18, 9)):
        before = decode(run, sinks, span)
        for b in range(2):
            L = int(inp.lengths[b])
            _poison(run, b, np.nonzero(~seen(L, sinks, span))[0], value)
        after = decode(run, sinks, span)
        np.testing.assert_array_equal(before[0], after[0])
        np.testing.assert_array_equal(before[1], after[1])
        run = DeviceRun(inp)


def prefill(run, seq, pos, qbits, sinks, span, stream_ctas=0, table=None, fused_rows=None, out_fp32=True):
    w, lib, n = run.inp.workload, run.lib, len(seq)
    i = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()
    t = lambda bits: torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)
    out = torch.full((n, w.q_heads, 128), float("nan"), dtype=torch.float32 if out_fp32 else torch.bfloat16, device="cuda")
    lse = torch.full((n, w.q_heads), float("nan"), device="cuda")
    nb = lib.kvq_prefill_workspace_size(run.cache.desc, n, w.q_heads, max(stream_ctas, 0))
    ws = torch.zeros(max(nb, 16), dtype=torch.uint8, device="cuda")
    new = {} if fused_rows is None else dict(k_new=t(run.inp.k[fused_rows]), v_new=t(run.inp.v[fused_rows]))
    lib.kvq_prefill_sinks(run.cache.desc, t(qbits), w.q_heads, i(seq), i(pos), run.table if table is None else table,
                          w.batch, run.inp.max_blocks, sinks, span, out, lse=lse, workspace=ws, workspace_bytes=nb,
                          stream_ctas=stream_ctas, err_word=run.err, **new)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), lse.cpu().numpy()


def _rows(order, lens, start):
    pairs = [(b, p) for b in range(len(lens)) for p in range(start[b], int(lens[b]))]
    if order == "mixed":
        pairs = sorted(pairs, key=lambda x: (x[1] * 7919) % 101)
    return np.array([b for b, _ in pairs]), np.array([p for _, p in pairs])


@pytest.mark.parametrize("order", ["seq", "mixed"])
@pytest.mark.parametrize("fmt", list(FORMATS))
def test_prefill_matches_the_oracle(fmt, order):
    w = small_workload(fmt, **dict(dict(batch=3, len_range=(100, 200)), **FORMATS[fmt]))
    inp = make_inputs(w, 3)
    run, ref, G = DeviceRun(inp), Oracle(inp), w.group
    start = [0, 70, int(inp.lengths[2]) - 1]
    seq, pos = _rows(order, inp.lengths, start)
    qbits = query_rows(len(seq), w.q_heads, 5)
    for sinks, span in ((4, 50), (0, 16), (21, 1), (0, 1000)):
        table = freed(run.table, inp.lengths, [s + 1 - span for s in start], sinks)
        o = np.zeros((len(seq), w.q_heads, 128))
        l = np.zeros((len(seq), w.q_heads))
        for r, (b, p) in enumerate(zip(seq, pos)):
            q = O.bf16_to_f64(qbits[r])
            for h in range(w.kv_heads):
                g = slice(h * G, (h + 1) * G)
                o[r, g], l[r, g] = ref(b, h, q[g], p + 1, sinks, span)
        for ctas in (0, 5) if w.k_bits == 16 else (0, -1, 5) if w.q_bits == 32 else (0, -1, -2, 5):
            assert worst(*prefill(run, seq, pos, qbits, sinks, span, ctas, table), o, l) <= 1.0, (sinks, span, ctas)
    assert run.err_bits() == 0


@pytest.mark.parametrize("ctas", [-1, -2, 3])
@pytest.mark.parametrize("fmt", ["int8_g4", "int4_factor_g8", "asym_int8", "bf16_g7"])
def test_prefill_rows_that_hide_a_token(fmt, ctas):
    """A token that is no number, or infinite, changes the rows that see it and no others of their tile."""
    if fmt == "bf16_g7" and ctas < 0:
        pytest.skip("a bf16 cache takes split rows")
    w = small_workload(fmt, **dict(dict(batch=1, len_range=(150, 150)), **FORMATS[fmt]))
    inp = make_inputs(w, 4)
    seq, pos = _rows("seq", inp.lengths, [60])
    qbits = query_rows(len(seq), w.q_heads, 6)
    sinks, span = 3, 30
    before = prefill(DeviceRun(inp), seq, pos, qbits, sinks, span, ctas)
    for at, value in ((100, float("nan")), (77, float("inf"))):
        run = DeviceRun(inp)
        _poison(run, 0, [at], value)
        after = prefill(run, seq, pos, qbits, sinks, span, ctas)
        hidden = (pos < at) | (pos - span >= at)
        np.testing.assert_array_equal(before[0][hidden], after[0][hidden])
        np.testing.assert_array_equal(before[1][hidden], after[1][hidden])
        assert np.all(~np.isfinite(after[0][~hidden]).all(axis=(1, 2)))


@pytest.mark.parametrize("fmt", ["int8_g4", "int4_factor_g8", "asym_int8", "k4v8_g3", "int8_g1_paged", "asym_int2_g8"])
@pytest.mark.parametrize("case", ["one long", "ragged", "few rows", "many sequences"])
def test_units_of_many_rows(fmt, case):
    """Units with several tiles, several units, sequences that share a unit, empty and invalid rows among them."""
    B, lo, hi = {"one long": (1, 900, 900), "ragged": (4, 150, 500), "few rows": (2, 700, 800),
                 "many sequences": (20, 1, 90)}[case]
    w = small_workload(fmt, **dict(dict(batch=B, len_range=(lo, hi)), **FORMATS[fmt]))
    inp = make_inputs(w, 9)
    run, ref, G = DeviceRun(inp), Oracle(inp), w.group
    start = [0] * B if case != "few rows" else [int(L) - 3 for L in inp.lengths]
    seq, pos = _rows("seq", inp.lengths, start)
    bad = np.zeros(len(seq), bool)
    if case in ("ragged", "many sequences"):
        seq, pos = seq.copy(), pos.copy()
        bad[5::41] = True
        pos[5::41] = -1          # nothing to attend to
        seq[46::82], bad[46::82] = B + 3, True
    qbits = query_rows(len(seq), w.q_heads, 11)
    for sinks, span in ((4, 130), (70, 1), (0, 333)):
        table = freed(run.table, inp.lengths, [s + 1 - span for s in start], sinks)
        out, lse = prefill(run, seq, pos, qbits, sinks, span, -2, table)
        assert run.err_bits() & ~run.lib.KVQ_DEVERR_POSITION == 0
        assert np.all(out[bad] == 0) and np.all(np.isneginf(lse[bad]))
        bf, _ = prefill(run, seq, pos, qbits, sinks, span, -2, table, out_fp32=False)
        for r in np.nonzero(~bad)[0][::7]:
            q = O.bf16_to_f64(qbits[r])
            for h in range(w.kv_heads):
                g = slice(h * G, (h + 1) * G)
                o, l = ref(seq[r], h, q[g], pos[r] + 1, sinks, span)
                assert worst(out[r, g], lse[r, g], o, l) <= 1.0, (r, h, sinks, span)
                assert worst(bf[r, g], None, o, l, True) <= 1.0


@pytest.mark.parametrize("fmt", ["int8_g4", "int4_factor_g8", "asym_int8", "k4v8_g3", "asym_int2_g8", "asym_int4_factor"])
@pytest.mark.parametrize("batch", [1, 3])
def test_units_that_clusters_share(fmt, batch):
    """Few units on long windows: 2, 4 and 8 CTAs a unit (8, 16 and 32 tiles at least), one pass or several in a unit, the last
    ones with fewer tiles than CTAs."""
    w = small_workload(fmt, **dict(dict(batch=batch, len_range=(2250, 2400)), **FORMATS[fmt]))
    inp = make_inputs(w, 14)
    run, ref, G = DeviceRun(inp), Oracle(inp), w.group
    ends = np.array(inp.lengths)
    if batch == 3:   # rows of the second sequence's front: a pass of two tiles, shared all the same
        ends[1] = 120
    start = [int(L) - n for L, n in zip(ends, [90, 30, 41])]
    seq, pos = _rows("seq", ends, start)
    qbits = query_rows(len(seq), w.q_heads, 15)
    for sinks, span in ((4, 560), (130, 1150), (0, 2200), (7, 10 ** 9)):
        low = [max(s + 1 - span, 0) for s in start]
        table = freed(run.table, ends, low, sinks)
        out, lse = prefill(run, seq, pos, qbits, sinks, span, -2, table)
        tiles, tiles_lse = prefill(run, seq, pos, qbits, sinks, span, -1, table)
        assert np.max(np.abs(out - tiles)) <= 2 * TOL and np.max(np.abs(lse - tiles_lse)) <= 2 * TOL
        for r in range(0, len(seq), 17):
            q = O.bf16_to_f64(qbits[r])
            for h in range(w.kv_heads):
                g = slice(h * G, (h + 1) * G)
                assert worst(out[r, g], lse[r, g], *ref(seq[r], h, q[g], pos[r] + 1, sinks, span)) <= 1.0, (r, h, sinks, span)
    assert run.err_bits() == 0


@pytest.mark.parametrize("fmt", ["int8_g4", "asym_int8", "int4_factor_g8", "qint8_asym_k8v4"])
def test_units_of_queries_of_any_size(fmt):
    """Large and tiny queries, zeros, infinities and no numbers among the rows of a unit: each row its own result."""
    w = small_workload(fmt, **dict(dict(batch=1, len_range=(400, 400)), **FORMATS[fmt]))
    inp = make_inputs(w, 12)
    run, ref, G = DeviceRun(inp), Oracle(inp), w.group
    seq, pos = _rows("seq", inp.lengths, [200])
    qbits = query_rows(len(seq), w.q_heads, 13).copy()
    size = np.resize([1.0, 200.0, 1e-9, 0.0, 1.0, 1e-30], len(seq))
    qbits[:] = f32_to_bf16_bits((O.bf16_to_f64(qbits) * size[:, None, None]).astype(np.float32))
    qbits[10], qbits[33] = 0x7FC0, 0x7F80  # not a number, infinity
    none = np.isin(np.arange(len(seq)), (10, 33))
    out, lse = prefill(run, seq, pos, qbits, 4, 150, -2)
    if w.q_bits != 8:  # (8-bit query codes hold a number for everything)
        assert np.isnan(out[10]).all() and not np.isfinite(lse[none]).any()
    for r in np.nonzero(~none)[0][::3]:
        q = O.bf16_to_f64(qbits[r])
        for h in range(w.kv_heads):
            g = slice(h * G, (h + 1) * G)
            o, l = ref(0, h, q[g], pos[r] + 1, 4, 150)
            # scores of the large rows reach 10^3 and more: float32 holds them to 2^-24, twice rounded
            s = 2.0 ** -22 * np.abs(l).max()
            assert np.max(np.abs(lse[r, g] - l)) <= TOL + s, r
            # and a weight moves by its exponent's error
            assert np.max(np.abs(out[r, g] - o)) <= TOL + 2 * s * np.abs(ref.kv[0][h][1]).max(), r


@pytest.mark.parametrize("ctas", [-1, -2])
@pytest.mark.parametrize("power", [-40, -26, -17, 6, 30])
@pytest.mark.parametrize("fmt", ["int8_g4", "asym_int8", "int4_factor_g8"])
def test_queries_and_keys_that_trade_a_power_of_two(fmt, power, ctas):
    """Queries times 2^p on keys times 2^-p: every code, product and sum of the definition stays as it was."""
    w = small_workload(fmt, **dict(dict(batch=1, len_range=(300, 300)), **FORMATS[fmt]))
    inp = make_inputs(w, 17)
    seq, pos = _rows("seq", inp.lengths, [150])
    qbits = query_rows(len(seq), w.q_heads, 18)
    want, want_lse = prefill(DeviceRun(inp), seq, pos, qbits, 4, 150, ctas)
    times = lambda bits, p: f32_to_bf16_bits((O.bf16_to_f64(bits) * 2.0 ** p).astype(np.float32))
    inp.k = times(inp.k, -power)
    out, lse = prefill(DeviceRun(inp), seq, pos, times(qbits, power), 4, 150, ctas)
    assert np.max(np.abs(out - want)) <= 2 * TOL and np.max(np.abs(lse - want_lse)) <= 2 * TOL


def test_prefill_writes_its_chunk_first():
    w = small_workload("w", batch=2, len_range=(90, 120))
    inp = make_inputs(w, 5)
    whole = DeviceRun(inp)
    seq, pos = _rows("seq", inp.lengths, [0, 0])
    qbits = query_rows(len(seq), w.q_heads, 7)
    want = prefill(whole, seq, pos, qbits, 4, 30)
    blank = DeviceRun(inp)
    for t in (blank.cache.k_codes, blank.cache.v_codes, blank.cache.meta):
        t.zero_()
    got = prefill(blank, seq, pos, qbits, 4, 30, fused_rows=inp.seq_offsets[seq] + pos)
    np.testing.assert_array_equal(want[0], got[0])


def test_device_errors_and_table_capacity():
    w = small_workload("e", batch=3, len_range=(100, 140))
    inp = make_inputs(w, 6)
    run = DeviceRun(inp)
    good = decode(run, 4, 40)
    # an entry that is needed and out of range; one that is not needed
    t = run.table.clone()
    t[0, 2] = 10 ** 6
    np.testing.assert_array_equal(decode(run, 4, 40, table=t)[0], good[0])
    assert run.err_bits() == 0
    t[1, 0] = -1
    out, _ = decode(run, 4, 40, table=t)
    assert run.err_bits() == run.lib.KVQ_DEVERR_BLOCK_ID
    np.testing.assert_array_equal(out[[0, 2]], good[0][[0, 2]])
    run.err.zero_()
    lens = run.lens.clone()
    lens[2] = -5
    out, lse = decode(run, 4, 40, lens=lens)
    assert run.err_bits() == run.lib.KVQ_DEVERR_SEQ_LEN and np.all(out[2] == 0) and np.all(np.isneginf(lse[2]))
    # the work is cut by all lengths, so the other rows are summed in other pieces: within the output tolerance
    np.testing.assert_allclose(out[:2], good[0][:2], rtol=0, atol=TOL)


def test_refusals():
    w = small_workload("r", batch=2, window=32, len_range=(50, 60))
    run = DeviceRun(make_inputs(w, 7))
    lib = run.lib
    for sinks, span, status in ((-1, 64, lib.KVQ_ERR_INVALID_ARG), (0, 0, lib.KVQ_ERR_INVALID_ARG),
                                (4, 31, lib.KVQ_ERR_UNSUPPORTED)):
        with pytest.raises(lib.KvqError) as e:
            decode(run, sinks, span)
        assert e.value.status == status
    q32 = DeviceRun(make_inputs(small_workload("q", batch=1, q_bits=32, len_range=(50, 60)), 7))
    with pytest.raises(lib.KvqError) as e:  # units carry the weights in one part
        prefill(q32, [0], [3], query_rows(1, 8, 0), 4, 64, lib.PREFILL_UNITS)
    assert e.value.status == lib.KVQ_ERR_UNSUPPORTED
    with pytest.raises(lib.KvqError) as e:  # a chunk needs its positions in blocks
        prefill(run, [0], [3], query_rows(1, w.q_heads, 0), 4, 64)
    assert e.value.status == lib.KVQ_ERR_UNSUPPORTED


def test_captured_replayed_and_on_two_streams():
    from quantized_kv_cache_07_gb300.cache import DecodeWorkspace
    w = small_workload("g", batch=4, q_heads=16, kv_heads=4, len_range=(900, 1500))
    inp = make_inputs(w, 8)
    run = DeviceRun(inp)
    want = decode(run, 4, 300)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [DecodeWorkspace(run.cache, w.batch, w.q_heads) for _ in range(2)]
    outs = [torch.zeros(w.batch, w.q_heads, 128, device="cuda") for _ in range(3)]

    def call(i, ws, stream):
        run.lib.kvq_decode_sinks(run.cache.desc, run.q, w.batch, w.q_heads, run.lens, run.table, inp.max_blocks, 4, 300,
                                 outs[i], workspace=ws.buf, workspace_bytes=ws.nbytes, stream=stream)
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            call(i, ws[i], streams[i])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(2, ws[0], None)
    run.lens.sub_(1)
    graph.replay()
    torch.cuda.synchronize()
    shorter = outs[2].cpu().numpy()
    run.lens.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        np.testing.assert_array_equal(o.cpu().numpy(), want[0])
    assert not np.array_equal(shorter, want[0])
