"""Attention with sinks and a sliding window: rows of a chunk that lie far apart, and positions at the end of 32 bits."""
import numpy as np
import pytest

from harness import DeviceRun, small_workload
from synth import make_inputs, query_rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from oracle import kvq_oracle as O  # noqa: E402
from test_gpu_sinks import FORMATS, Oracle, prefill, worst  # noqa: E402


def paths(w):
    """Every path of the format: automatic, tiles, units, split rows."""
    return (0, 5) if w.k_bits == 16 else (0, -1, 5) if w.q_bits == 32 else (0, -1, -2, 5)


def seen_by(pos, L, sinks, span):
    """Which of L tokens one at least of the rows at `pos` sees."""
    i, p = np.arange(L), np.asarray(pos)[:, None]
    return ((i <= p) & ((i < sinks) | (i > p - span))).any(0)


# positions of one sequence's rows and (sinks, span): windows that leave blocks, parts of blocks or nothing between them
APART = [([2, 700], 4, 64), ([700, 2, 3, 350, 351, 352], 4, 20), ([5, 40, 41, 90, 640, 1020], 0, 33), ([17, 18], 0, 1),
         ([900, 60, 480], 40, 16), (list(range(100, 180)) + list(range(800, 860)), 3, 50), (list(range(0, 1000, 37)), 16, 5),
         (list(range(200, 330)), 2, 7), ([800, 30, 31, 32, 801, 33], 4, 10), ([3, 3, 3, 6], 0, 1), ([64, 500, 64, 500], 0, 40)]


@pytest.mark.parametrize("pos,sinks,span", APART)
@pytest.mark.parametrize("fmt", ["int8_g4", "int4_factor_g8", "asym_int8", "q32_asym_k4v8", "asym_int2_g8", "bf16_g7", "kchan_int8",
                                 "int8_g1_paged"])
def test_rows_far_apart(fmt, pos, sinks, span):
    """Blocks that no row of the chunk sees may be gone: no error and the oracle's results on every path."""
    w = small_workload(fmt, **dict(dict(batch=2, len_range=(1030, 1100)), **FORMATS[fmt]))
    inp = make_inputs(w, 21)
    run, ref, G = DeviceRun(inp), Oracle(inp), w.group
    seq = np.array([1] * len(pos) + [0])  # and a row of another sequence behind them
    pos = np.array(pos + [900])
    qbits = query_rows(len(seq), w.q_heads, 22)
    table = run.table.clone()
    for b in range(2):
        s = seen_by(pos[seq == b], 16 * table.shape[1], sinks, span).reshape(-1, 16).any(1)
        table[b, torch.from_numpy(~s).cuda()] = -1
    o, l = np.zeros((len(seq), w.q_heads, 128)), np.zeros((len(seq), w.q_heads))
    for r, (b, p) in enumerate(zip(seq, pos)):
        q = O.bf16_to_f64(qbits[r])
        for h in range(w.kv_heads):
            g = slice(h * G, (h + 1) * G)
            o[r, g], l[r, g] = ref(b, h, q[g], p + 1, sinks, span)
    for ctas in paths(w):
        out = prefill(run, seq, pos, qbits, sinks, span, ctas, table)
        assert run.err_bits() == 0, ctas
        assert worst(*out, o, l) <= 1.0, ctas


@pytest.mark.parametrize("fmt,what", [(f, "records") for f in ("int8_g4", "asym_int8", "q32_asym_k4v8", "asym_int4_factor")] + [
    (f, "zero points") for f in ("asym_int8", "q32_asym_k4v8", "asym_int4_factor")])
def test_tokens_between_the_windows_are_not_data(fmt, what):
    """What the scales and zero points of tokens that no row sees hold changes no bit: in whole blocks and in parts."""
    w = small_workload(fmt, **dict(dict(batch=1, len_range=(1030, 1030)), **FORMATS[fmt]))
    inp = make_inputs(w, 23)
    for pos, sinks, span in APART:
        run = DeviceRun(inp)
        qbits, seq = query_rows(len(pos), w.q_heads, 24), np.zeros(len(pos), int)
        before = [prefill(run, seq, np.array(pos), qbits, sinks, span, ctas) for ctas in paths(w)]
        M = run.cache.meta_floats
        meta = run.cache.meta.view(w.kv_heads, run.cache.num_blocks, M // 16, 16)
        s = seen_by(pos, 16 * run.table.shape[1], sinks, span).reshape(-1, 16)
        hidden = torch.zeros(run.cache.num_blocks, 16, dtype=torch.bool)
        hidden[run.table[0].long().cpu()] = torch.from_numpy(~s)
        fields = [1, 3] if what == "zero points" else list(range(M // 16))
        for f in fields:
            meta[:, :, f][:, hidden.cuda()] = float("nan")
        for ctas, want in zip(paths(w), before):
            got = prefill(run, seq, np.array(pos), qbits, sinks, span, ctas)
            np.testing.assert_array_equal(want[0], got[0], err_msg=str(ctas))
            np.testing.assert_array_equal(want[1], got[1], err_msg=str(ctas))
        assert run.err_bits() == 0


@pytest.mark.parametrize("fmt", ["int8_g4", "q32_int8", "bf16_g7"])
def test_a_missing_block_between_the_windows_that_a_row_sees(fmt):
    """The same rows, and one entry that a single row of them needs: reported on every path."""
    w = small_workload(fmt, **dict(dict(batch=1, len_range=(1030, 1030)), **FORMATS[fmt]))
    run = DeviceRun(make_inputs(w, 25))
    pos = np.array([700, 2, 3, 350, 351, 352])
    table = run.table.clone()
    table[0, 21] = 10 ** 6   # tokens 336 .. 351
    for ctas in paths(w):
        prefill(run, pos * 0, pos, query_rows(len(pos), w.q_heads, 26), 4, 20, ctas, table)
        assert run.err_bits() == run.lib.KVQ_DEVERR_BLOCK_ID, ctas
        run.err.zero_()


@pytest.mark.parametrize("windowed", [True, False])
@pytest.mark.parametrize("fmt", ["int8_g4", "asym_int2_g8", "bf16_g7"])
def test_the_last_position_is_cut_to_the_table_on_every_path(fmt, windowed):
    """A row at 2^31 - 1 is reported and attends as the table's last position does, as any position behind the table."""
    w = small_workload(fmt, **dict(dict(batch=1, len_range=(300, 300)), **FORMATS[fmt]))
    run = DeviceRun(make_inputs(w, 27))
    lib, table, q_heads = run.lib, run.table, w.q_heads
    pos, qbits, end = np.arange(250, 290), query_rows(40, q_heads, 28), 16 * run.inp.max_blocks - 1
    i = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()

    def whole(pos, ctas):
        q = torch.from_numpy(qbits.view(np.int16)).cuda().view(torch.bfloat16)
        out, lse = torch.empty(40, q_heads, 128, device="cuda"), torch.empty(40, q_heads, device="cuda")
        ws = torch.zeros(lib.kvq_prefill_workspace_size(run.cache.desc, 40, q_heads, max(ctas, 0)) + 16, dtype=torch.uint8,
                         device="cuda")
        lib.kvq_prefill(run.cache.desc, q, q_heads, i(pos * 0), i(pos), table, 1, run.inp.max_blocks, out, lse=lse,
                        workspace=ws, workspace_bytes=ws.numel(), stream_ctas=ctas, err_word=run.err)
        return out.cpu().numpy(), lse.cpu().numpy()
    for ctas in paths(w):
        if ctas == -2 and not windowed:
            continue
        got = []
        for p, bits in ((end, 0), (end + 1, lib.KVQ_DEVERR_SEQ_LEN), (2 ** 31 - 2, lib.KVQ_DEVERR_SEQ_LEN),
                        (2 ** 31 - 1, lib.KVQ_DEVERR_SEQ_LEN)):
            at = pos.copy()
            at[13] = p
            got.append(prefill(run, pos * 0, at, qbits, 4, 64, ctas) if windowed else whole(at, ctas))
            assert run.err_bits() == bits, (ctas, p)
            run.err.zero_()
            np.testing.assert_array_equal(got[0][0], got[-1][0], err_msg=str((ctas, p)))
            np.testing.assert_array_equal(got[0][1], got[-1][1], err_msg=str((ctas, p)))
