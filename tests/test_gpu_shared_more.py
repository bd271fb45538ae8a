"""Shared prefixes: the two-part queries of asymmetric caches on tcgen05, many groups, and groups that are mixed."""
import numpy as np
import pytest

from harness import DeviceRun, compare_outputs, oracle_state, small_workload
from oracle import kvq_oracle as O
from test_gpu_shared import decode_shared, shared_inputs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


@pytest.mark.parametrize("kw", [dict(k_bits=4, v_bits=4), dict(), dict(k_bits=4), dict(v_bits=4), dict(k_bits=2, v_bits=2)])
@pytest.mark.parametrize("batch,q_heads", [(50, 8), (50, 16), (17, 8)])     # 164 and 36 vectors, 328 and 72, 68 in one
def test_asymmetric_caches_under_a_key_factor(kw, batch, q_heads):
    """Outputs and log-sum-exps of full tiles, with rows that end before, inside and behind the prefix."""
    w = small_workload("shared_two", **dict(dict(batch=batch, q_heads=q_heads, len_range=(500, 640), paged=True, asym=True,
                                                 channel_factor=True, outlier_channels=4), **kw))
    groups = [(0, 41, 29), (41, 50, 9)] if batch == 50 else [(0, 17, 29)]
    inp = shared_inputs(w, groups)
    run = DeviceRun(inp)
    lens = np.array(inp.lengths)
    lens[[3, 8, 11, 13, 7]] = [0, 1, 463, 464, 143]
    lens_t = torch.from_numpy(lens.astype(np.int32)).cuda()
    # the definition for every length (kvq_decode carries the query times the factor in one fp16 part: its score may be
    # 2^-11 of the products' sum off, more than the tolerance for 2-bit keys)
    ref = {}
    for b in range(batch):
        st = oracle_state(inp, b)
        for h in range(w.kv_heads):
            k_hat, v_hat = O.reconstruct_sequence(st, h)
            ref[(b, h)] = O.attention(O.bf16_to_f64(inp.q[b, h * w.group:(h + 1) * w.group]), k_hat[:lens[b]], v_hat[:lens[b]])
    for fp32 in (True, False):
        out, lse = decode_shared(run, groups, out_fp32=fp32, lens=lens_t)
        assert compare_outputs(inp, out, lse, ref, not fp32) <= 1.0
    assert np.all(out[3] == 0) and np.all(np.isneginf(lse[3]))
    assert run.err_bits() == 0


@pytest.mark.parametrize("num,each,q_heads", [(33, 2, 8), (256, 2, 8), (33, 8, 16), (64, 9, 16), (256, 8, 16)])
def test_many_groups(num, each, q_heads):
    """More groups than one round of 32 lanes cleans and adds up, on 16-vector tiles and on tcgen05: prefixes of 0 to 3
    blocks, groups without rows, and every start checked by its own sequences' results."""
    rng = np.random.default_rng(num)
    batch = num * each + 3
    w = small_workload("shared_groups", batch=batch, q_heads=q_heads, len_range=(50, 90))
    cuts = np.sort(rng.integers(0, batch + 1, num - 1))
    start = np.concatenate([[0], cuts, [batch]])
    blocks = rng.integers(0, 4, num)
    groups = [(int(a), int(b), int(p)) for a, b, p in zip(start[:-1], start[1:], blocks)]
    assert any(a == b for a, b, _ in groups)
    inp = shared_inputs(w, groups)
    run = DeviceRun(inp)
    out, lse = decode_shared(run, groups)
    o, l = run.decode()
    np.testing.assert_allclose(out, o, rtol=0, atol=2e-3)
    np.testing.assert_allclose(lse, l, rtol=0, atol=2e-3)
    assert run.err_bits() == 0
    # a start that falls, far behind the first 32: cleaned and flagged, the results as before
    if num > 40:
        fallen = start.copy()
        fallen[40] = max(int(start[39]) - 5, 0) if start[39] > 0 else -1
        assert fallen[40] < start[39]
        again, _ = decode_shared(run, groups, start=fallen.tolist(), blocks=[0] * 41 + [0] * (num - 41))
        assert run.err_bits() == run.lib.KVQ_DEVERR_POSITION
        np.testing.assert_allclose(again, o, rtol=0, atol=2e-3)


def test_a_large_group_beside_small_ones():
    """240 vectors in one group and two in each of seven: the average decides the path, the results are the same."""
    w = small_workload("shared_mixed", batch=74, q_heads=8, len_range=(200, 260))
    groups = [(0, 60, 11)] + [(60 + 2 * i, 62 + 2 * i, 3 + i) for i in range(7)]
    inp = shared_inputs(w, groups)
    run = DeviceRun(inp)
    out, lse = decode_shared(run, groups)
    o, l = run.decode()
    np.testing.assert_allclose(out, o, rtol=0, atol=2e-3)
    np.testing.assert_allclose(lse, l, rtol=0, atol=2e-3)
    assert run.err_bits() == 0
