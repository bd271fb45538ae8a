"""Decode over shared prefixes (kvq_decode_shared) against the float64 oracle and kvq_decode.

Inputs are ordinary decode inputs whose sequences are made to share the tokens
and blocks of their group's prefix; the oracle sees every sequence whole.
"""
import numpy as np
import pytest

from harness import DeviceRun, compare_outputs, oracle_decode, small_workload
from synth import make_inputs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def shared_inputs(w, groups, seed=0):
    """make_inputs(w) with groups [(first, last + 1, prefix blocks)]: the sequences of a group hold the tokens and the
    blocks of its longest sequence's prefix (of their own length, where they are shorter)."""
    inp = make_inputs(w, seed)
    for a, e, P in groups:
        if e <= a or P == 0:
            continue
        lead = a + int(np.argmax(inp.lengths[a:e]))
        assert inp.lengths[lead] >= 16 * P, "no sequence of the group holds the whole prefix"
        for b in range(a, e):
            n = min(16 * P, int(inp.lengths[b]))
            src, dst = inp.seq_offsets[lead], inp.seq_offsets[b]
            inp.k[dst:dst + n] = inp.k[src:src + n]
            inp.v[dst:dst + n] = inp.v[src:src + n]
            inp.block_table[b, :P] = inp.block_table[lead, :P]
    return inp


def decode_shared(run, groups, out_fp32=True, lens=None, ws=None, lse=True, num=None, start=None, blocks=None):
    from quantized_kv_cache_07_gb300.cache import SharedWorkspace
    w, inp = run.inp.workload, run.inp
    start = [g[0] for g in groups] + [groups[-1][1]] if start is None else start
    blocks = [g[2] for g in groups] if blocks is None else blocks
    i = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
    out = torch.full((w.batch, w.q_heads, 128), float("nan"), device="cuda",
                     dtype=torch.float32 if out_fp32 else torch.bfloat16)
    l = torch.full((w.batch, w.q_heads), float("nan"), device="cuda") if lse else None
    ws = ws or SharedWorkspace(run.cache, w.batch, w.q_heads, len(blocks))
    run.lib.kvq_decode_shared(run.cache.desc, run.q, w.batch, w.q_heads, run.lens if lens is None else lens, run.table,
                              inp.max_blocks, len(blocks), i(start), i(blocks), out, lse=l, workspace=ws.buf,
                              workspace_bytes=ws.nbytes, err_word=run.err)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), None if l is None else l.cpu().numpy()


FORMATS = {
    "int8_g4": dict(),
    "int8_g1": dict(q_heads=4, kv_heads=4),
    "int4_factor_g8": dict(q_heads=16, k_bits=4, v_bits=4, channel_factor=True),
    "k4v8_g3_t3": dict(q_heads=6, k_bits=4, k_dist="t3", paged=True),
    "k8v4_g5": dict(q_heads=10, v_bits=4, paged=True),
    "window32_int8": dict(window=32),
    "window16_asym_k4v8": dict(window=16, k_bits=4, asym=True, q_heads=16),
    "bf16_g7": dict(q_heads=14, k_bits=16, v_bits=16),
    "asym_int8": dict(asym=True, outlier_channels=4), "asym_int4_factor": dict(asym=True, k_bits=4, v_bits=4,
                                                                              channel_factor=True),
    "kchan_int8": dict(channel_factor=True, k_per_channel=True),
    "qint8_int8": dict(q_bits=8), "qint8_asym_k8v4": dict(q_bits=8, asym=True, v_bits=4),
    "q32_int8": dict(q_bits=32), "q32_asym_int4_factor": dict(q_bits=32, asym=True, k_bits=4, v_bits=4,
                                                              channel_factor=True),
    "int2": dict(k_bits=2, v_bits=2), "asym_int2_g8": dict(k_bits=2, v_bits=2, asym=True, q_heads=16),
    "q32_int2": dict(k_bits=2, v_bits=2, q_bits=32),
}
# a group of many rows, one of one row, one without a prefix, one without rows
GROUPS = [(0, 9, 11), (9, 10, 7), (10, 12, 0), (12, 12, 3), (12, 15, 6)]


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_matches_the_oracle(fmt):
    w = small_workload(fmt, **dict(dict(batch=16, len_range=(200, 420)), **FORMATS[fmt]))
    inp = shared_inputs(w, GROUPS)     # sequence 15 is in no group
    run = DeviceRun(inp)
    ref = oracle_decode(inp)
    out, lse = decode_shared(run, GROUPS)
    assert compare_outputs(inp, out, lse, ref, False) <= 1.0
    out, lse = decode_shared(run, GROUPS, out_fp32=False, lse=False)
    assert lse is None and compare_outputs(inp, out, None, ref, True) <= 1.0
    assert run.err_bits() == 0


@pytest.mark.parametrize("fmt", ["int8_g4", "asym_int4_factor", "window32_int8", "bf16_g7", "int2"])
def test_sequences_shorter_than_their_prefix(fmt):
    """Lengths of zero, one, inside the prefix, exactly its end and one behind it."""
    kw = dict(dict(batch=8, len_range=(300, 420), paged=True), **FORMATS[fmt])
    w = small_workload(fmt, **kw)
    groups = [(0, 8, 12)]
    inp = shared_inputs(w, groups)
    run = DeviceRun(inp)
    if w.window:   # the ring's contents go by the length: only whole sequences and empty ones
        lens = np.array(inp.lengths)
        lens[2] = 0
    else:
        lens = np.array([0, 1, 17, 100, 191, 192, 193, inp.lengths[7]])
    lens_t = torch.from_numpy(lens.astype(np.int32)).cuda()
    out, lse = decode_shared(run, groups, lens=lens_t)
    o, l = run.decode(lens=lens_t)
    empty = lens == 0
    assert np.all(out[empty] == 0) and np.all(np.isneginf(lse[empty]))
    np.testing.assert_allclose(out[~empty], o[~empty], rtol=0, atol=2e-3)
    np.testing.assert_allclose(lse[~empty], l[~empty], rtol=0, atol=2e-3)
    assert run.err_bits() == 0


@pytest.mark.parametrize("fmt", ["int8_g4", "int4_factor_g8", "k4v8_g3_t3", "k8v4_g5", "window32_int8",
                                 "window16_asym_k4v8", "asym_int8", "kchan_int8", "qint8_asym_k8v4", "int2",
                                 "asym_int2_g8"])
def test_full_tiles_of_every_format(fmt):
    """Groups of enough vectors for the 128-vector tiles, over more than one unit per CTA, with rows that end before,
    inside and behind the prefix."""
    w = small_workload(fmt, **dict(dict(batch=50, len_range=(500, 640), paged=True), **FORMATS[fmt]))
    groups = [(0, 41, 29), (41, 50, 9)]
    inp = shared_inputs(w, groups)
    run = DeviceRun(inp)
    lens = np.array(inp.lengths)
    if not w.window:
        lens[[3, 8, 20, 33, 42, 45]] = [0, 1, 463, 464, 143, 200]
    lens[7] = 0
    lens_t = torch.from_numpy(lens.astype(np.int32)).cuda()
    out, lse = decode_shared(run, groups, lens=lens_t)
    o, l = run.decode(lens=lens_t)
    empty = lens == 0
    assert np.all(out[empty] == 0) and np.all(np.isneginf(lse[empty]))
    np.testing.assert_allclose(out[~empty], o[~empty], rtol=0, atol=2e-3)
    np.testing.assert_allclose(lse[~empty], l[~empty], rtol=0, atol=2e-3)
    whole = {(b, h) for b in range(0, 50, 6) if lens[b] == inp.lengths[b] for h in range(w.kv_heads)}
    assert compare_outputs(inp, out, lse, oracle_decode(inp, whole), False) <= 1.0
    assert run.err_bits() == 0


@pytest.mark.parametrize("kw,groups", [
    (dict(batch=40, q_heads=32, kv_heads=8, len_range=(2100, 2300)), [(0, 40, 130)]),       # 160 vectors, long
    (dict(batch=3, q_heads=4, kv_heads=4, len_range=(9000, 9100), k_bits=4), [(0, 3, 560)]),  # few vectors, many CTAs
    (dict(batch=70, q_heads=16, kv_heads=2, len_range=(90, 130), v_bits=4), [(0, 70, 5)]),   # 560 vectors, short
    (dict(batch=33, q_heads=8, kv_heads=1, len_range=(700, 900), asym=True), [(0, 17, 40), (17, 33, 3)]),
    (dict(batch=20, q_heads=16, kv_heads=2, len_range=(600, 700), k_bits=2, v_bits=2), [(0, 20, 37)]),
    (dict(batch=20, q_heads=16, kv_heads=2, len_range=(600, 700), q_bits=32), [(0, 20, 37)]),
    (dict(batch=20, q_heads=16, kv_heads=2, len_range=(600, 700), q_bits=8, asym=True), [(0, 20, 37)]),
    (dict(batch=20, q_heads=16, kv_heads=2, len_range=(600, 700), channel_factor=True, k_per_channel=True),
     [(0, 20, 37)]),
    (dict(batch=20, q_heads=10, kv_heads=2, len_range=(600, 700), k_bits=16, v_bits=16), [(0, 20, 37)]),
])
def test_many_vectors_and_long_prefixes(kw, groups):
    w = small_workload("shared_sizes", **dict(dict(paged=True), **kw))
    inp = shared_inputs(w, groups)
    run = DeviceRun(inp)
    rng = np.random.default_rng(1)
    units = {(int(b), int(h)) for b, h in zip(rng.integers(0, w.batch, 12), rng.integers(0, w.kv_heads, 12))}
    ref = oracle_decode(inp, units)
    out, lse = decode_shared(run, groups)
    assert np.all(np.isfinite(out)) and compare_outputs(inp, out, lse, ref, False) <= 1.0
    # twice on one workspace: the same bits
    from quantized_kv_cache_07_gb300.cache import SharedWorkspace
    ws = SharedWorkspace(run.cache, w.batch, w.q_heads, len(groups))
    for _ in range(2):
        again = decode_shared(run, groups, ws=ws)
        np.testing.assert_array_equal(again[0], out)
        np.testing.assert_array_equal(again[1], lse)
    assert run.err_bits() == 0


@pytest.mark.parametrize("kw", [dict(k_bits=4, v_bits=4, asym=True), dict(k_bits=2, v_bits=2), dict(),
                                dict(k_bits=4, v_bits=4, asym=True, q_heads=16), dict(k_bits=2, v_bits=2, q_heads=16),
                                dict(q_heads=16), dict(q_heads=16, channel_factor=True)])
@pytest.mark.parametrize("P", [1, 4, 7, 12, 23])
def test_short_prefixes_again_and_again(kw, P):
    """A few tiles per CTA, where the conversion runs furthest ahead of the softmax: the same bits every time."""
    w = small_workload("shared_again", **dict(dict(batch=8, len_range=(400, 420), paged=True), **kw))
    groups = [(0, 8, P)]
    inp = shared_inputs(w, groups)
    run = DeviceRun(inp)
    ref, ref_lse = run.decode()
    first = decode_shared(run, groups)
    np.testing.assert_allclose(first[0], ref, rtol=0, atol=2e-3)
    np.testing.assert_allclose(first[1], ref_lse, rtol=0, atol=2e-3)
    for _ in range(25):
        out, lse = decode_shared(run, groups)
        assert run.err_bits() == 0
        np.testing.assert_array_equal(out, first[0])
        np.testing.assert_array_equal(lse, first[1])


def test_large_scores_and_extreme_value_scales():
    """Scores that need the running maximum to move, and values of very different sizes."""
    w = small_workload("shared_extreme", batch=24, q_heads=16, kv_heads=2, len_range=(900, 1000))
    groups = [(0, 24, 50)]
    inp = make_inputs(w)
    from oracle import kvq_oracle as O
    from synth import f32_to_bf16_bits
    rng = np.random.default_rng(5)
    size = np.exp(rng.uniform(-12, 6, inp.v.shape[0])).astype(np.float32)
    inp.v[:] = f32_to_bf16_bits(O.bf16_to_f64(inp.v).astype(np.float32) * size[:, None, None])
    ramp = np.linspace(0.1, 3, inp.k.shape[0]).astype(np.float32)
    inp.k[:] = f32_to_bf16_bits(O.bf16_to_f64(inp.k).astype(np.float32) * ramp[:, None, None])
    lead = int(np.argmax(inp.lengths))
    for b in range(24):
        a, s = inp.seq_offsets[b], inp.seq_offsets[lead]
        inp.k[a:a + 800], inp.v[a:a + 800] = inp.k[s:s + 800].copy(), inp.v[s:s + 800].copy()
        inp.block_table[b, :50] = inp.block_table[lead, :50]
    run = DeviceRun(inp)
    ref = oracle_decode(inp)
    out, lse = decode_shared(run, groups)
    for (b, h), (o, l) in ref.items():
        # fp16 weights: half a step (2^-12 of the largest value, here up to 400 times 4) on each of the terms
        atol = 2e-3 + 2.0 ** -11 * np.abs(o).max()
        assert np.max(np.abs(out[b, 8 * h:8 * h + 8] - o)) <= atol
        assert np.max(np.abs(lse[b, 8 * h:8 * h + 8] - l)) <= 2e-3


def test_bad_groups_are_flagged_and_cleaned():
    w = small_workload("shared_bad", batch=6, len_range=(100, 160))
    groups = [(0, 3, 4), (3, 6, 5)]
    inp = shared_inputs(w, groups)
    run = DeviceRun(inp)
    ref, ref_lse = decode_shared(run, groups)
    lib = run.lib

    def flagged(start, blocks, bits):
        run.err.zero_()
        out, lse = decode_shared(run, groups, start=start, blocks=blocks)
        assert run.err_bits() == bits
        return out, lse
    # a start behind the batch, one that falls, one below zero: the sequences still get their own attention
    for start in ([0, 3, 9], [0, 3, 2], [-2, 3, 6]):
        out, lse = flagged(start, [4, 5], lib.KVQ_DEVERR_POSITION)
        np.testing.assert_allclose(out, ref, rtol=0, atol=2e-3)
        np.testing.assert_allclose(lse, ref_lse, rtol=0, atol=2e-3)
    out, _ = flagged([0, 3, 6], [-1, 5], lib.KVQ_DEVERR_SEQ_LEN)       # no prefix: every sequence by itself
    np.testing.assert_allclose(out, ref, rtol=0, atol=2e-3)
    lens = run.lens.clone()
    lens[1] = inp.max_blocks * 16 + 1
    lens[4] = -1
    run.err.zero_()
    out, lse = decode_shared(run, groups, lens=lens)
    assert run.err_bits() & lib.KVQ_DEVERR_SEQ_LEN and np.all(out[4] == 0)
    np.testing.assert_allclose(out[[0, 2, 3, 5]], ref[[0, 2, 3, 5]], rtol=0, atol=2e-3)
    # a prefix block that is not there
    run.err.zero_()
    run.table[0, 2] = inp.num_blocks
    out, _ = decode_shared(run, groups)
    assert run.err_bits() == lib.KVQ_DEVERR_BLOCK_ID
    np.testing.assert_allclose(out[3:], ref[3:], rtol=0, atol=2e-3)


def test_the_workspace_is_checked():
    w = small_workload("shared_ws", batch=4, len_range=(100, 160))
    inp = shared_inputs(w, [(0, 4, 4)])
    run = DeviceRun(inp)
    nb = run.lib.kvq_decode_shared_workspace_size(run.cache.desc, 4, w.q_heads, 1)

    class Small:
        buf, nbytes = torch.zeros(nb, dtype=torch.uint8, device="cuda"), nb - 1
    with pytest.raises(run.lib.KvqError) as e:
        decode_shared(run, [(0, 4, 4)], ws=Small)
    assert e.value.status == run.lib.KVQ_ERR_WORKSPACE


def test_captured_and_replayed_with_other_groups():
    """One captured call, replayed with other lengths, groups and queries in the same buffers."""
    from quantized_kv_cache_07_gb300.cache import SharedWorkspace
    w = small_workload("shared_graph", batch=12, len_range=(300, 420))
    inp = shared_inputs(w, [(0, 12, 15)])
    run = DeviceRun(inp)
    ws = SharedWorkspace(run.cache, 12, w.q_heads, 2)
    start, blocks = torch.tensor([0, 5, 12], dtype=torch.int32).cuda(), torch.tensor([15, 7], dtype=torch.int32).cuda()
    out = torch.zeros(12, w.q_heads, 128, device="cuda")

    def call():
        run.lib.kvq_decode_shared(run.cache.desc, run.q, 12, w.q_heads, run.lens, run.table, inp.max_blocks, 2, start,
                                  blocks, out, workspace=ws.buf, workspace_bytes=ws.nbytes)
    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for a, p in (([0, 12, 12], [10, 0]), ([2, 4, 9], [15, 3])):
        start.copy_(torch.tensor(a))
        blocks.copy_(torch.tensor(p))
        run.q.normal_()
        run.lens.sub_(7)
        g.replay()
        torch.cuda.synchronize()
        ref, _ = run.decode()
        np.testing.assert_allclose(out.cpu().numpy(), ref, rtol=0, atol=2e-3)


@pytest.mark.parametrize("kw", [dict(), dict(k_bits=4, v_bits=4, channel_factor=True), dict(q_bits=32)])
def test_groups_without_a_prefix(kw):
    """Nothing is shared: the prefix kernel has no work, the result is kvq_decode's."""
    run = DeviceRun(make_inputs(small_workload("shared_none", **dict(dict(batch=16, len_range=(1, 300)), **kw))))
    out, lse = decode_shared(run, [(0, 16, 0)])
    ref, ref_lse = run.decode()
    np.testing.assert_allclose(out, ref, rtol=0, atol=2e-3)
    np.testing.assert_allclose(lse, ref_lse, rtol=0, atol=2e-3)
    assert run.err_bits() == 0


@pytest.mark.parametrize("batch,kw", [(16, dict()), (16, dict(q_heads=16)), (3, dict()),
                                      (16, dict(k_bits=4, v_bits=4, channel_factor=True, q_heads=16))])
def test_inputs_written_by_the_kernels_just_before(batch, kw):
    """Queries, lengths, groups and the table change between calls that are queued without a wait."""
    from quantized_kv_cache_07_gb300.cache import SharedWorkspace
    w = small_workload("shared_queued", **dict(dict(batch=batch, len_range=(400, 420), paged=True), **kw))
    inp = shared_inputs(w, [(0, batch, 20)])
    run = DeviceRun(inp)
    ws = SharedWorkspace(run.cache, batch, w.q_heads, 2)
    i = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    g = torch.Generator(device="cuda").manual_seed(5)
    sets = []
    for k in range(12):
        P = (20, 13, 1, 17)[k % 4]
        # other blocks for the sequences' own tokens: two swapped rows behind the prefix
        table = run.table.clone()
        table[:, 20:] = table[:, 20:].roll(k % 3, 0)
        sets.append((torch.randn(run.q.shape, generator=g, device="cuda").bfloat16(),
                     torch.randint(330, 400, (batch,), generator=g, device="cuda").int(), table,
                     i([0, (k * 5) % (batch + 1), batch]), i([P, (P + k) % 21])))
    q, lens, table, start, blocks = (t.clone() for t in sets[0])
    outs = [torch.empty(batch, w.q_heads, 128, device="cuda") for _ in sets]
    torch.cuda.synchronize()
    for s, out in zip(sets, outs):
        for dst, src in zip((q, lens, table, start, blocks), s):
            dst.copy_(src)
        run.lib.kvq_decode_shared(run.cache.desc, q, batch, w.q_heads, lens, table, inp.max_blocks, 2, start, blocks, out,
                                  workspace=ws.buf, workspace_bytes=ws.nbytes, err_word=run.err)
    for s, out in zip(sets, outs):
        run.q.copy_(s[0])
        run.table.copy_(s[2])
        ref, _ = run.decode(lens=s[1])
        np.testing.assert_allclose(out.cpu().numpy(), ref, rtol=0, atol=2e-3)
    assert run.err_bits() == 0


@pytest.mark.parametrize("batch", [40, 3])
@pytest.mark.parametrize("kw", [dict(), dict(k_bits=4, v_bits=4), dict(k_bits=4, asym=True), dict(k_per_channel=True),
                                dict(window=32)])
def test_log_sum_exp_under_a_key_factor(batch, kw):
    """The query times the factor does not fit in fp16's 11 bits: its log-sum-exp holds float32's precision all the same."""
    from harness import oracle_state
    from oracle import kvq_oracle as O
    w = small_workload("shared_lse", **dict(dict(batch=batch, len_range=(300, 420), channel_factor=True,
                                                 outlier_channels=4), **kw))
    inp = shared_inputs(w, [(0, batch, 15)])
    run = DeviceRun(inp)
    _, lse = decode_shared(run, [(0, batch, 15)])
    for b in range(batch):
        st = oracle_state(inp, b)
        q = O.bf16_to_f64(inp.q[b])
        for h in range(w.kv_heads):
            k_hat, _ = O.reconstruct_sequence(st, h)
            qh = q[h * w.group:(h + 1) * w.group]
            s = qh @ k_hat.T / np.sqrt(128.0)
            top = s.max(1, keepdims=True)
            ref = top[:, 0] + np.log(np.exp(s - top).sum(1))
            # float32 half-steps (2^-24) of the score's absolute sum: 8 products of 16 terms each added one after
            # another, the low query parts and the factor, three scale factors: below 32 of them, and as many again
            # where the tensor cores cut instead of rounding; of the exponents and of lse one each; 2^-22 of ex2,
            # log2 and the sums' merges each
            size = np.abs(qh) @ np.abs(k_hat).T / np.sqrt(128.0)
            if w.asym:  # the code dot and the zero-point term are each larger than their sum
                size = 4 * size + 4 * np.abs(qh).sum(1, keepdims=True) * np.abs(k_hat).max(1) / np.sqrt(128.0)
            p = np.exp(s - ref[:, None])
            tol = (p * (64 * size + np.abs(s) + np.abs(ref[:, None]))).sum(1) * 2.0 ** -24 + 3 * 2.0 ** -22
            assert np.all(np.abs(lse[b, h * w.group:(h + 1) * w.group] - ref) <= tol), (b, h)
    assert run.err_bits() == 0
