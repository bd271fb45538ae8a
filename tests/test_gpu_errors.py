"""A call that could not be launched leaves nothing behind: the next one is judged by itself."""
import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def _i(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def calls():
    """name -> a call on a given stream, on one small cache."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import DecodeWorkspace, KVCache, RopeTable, SharedWorkspace
    B, H, Hq = 2, 2, 4
    c, rope = KVCache(8, H, 8, 8), RopeTable(64)
    table, lens, seq, pos = _i(np.arange(8).reshape(2, 4)), _i([20, 20]), _i([0, 1]), _i([19, 19])
    x, q = torch.randn(B, H, 128, device="cuda").bfloat16(), torch.randn(B, Hq, 128, device="cuda").bfloat16()
    out, lse, mass = torch.zeros_like(q), torch.zeros(B, Hq, device="cuda"), torch.zeros(B, H, 64, device="cuda")
    ws, sw = DecodeWorkspace(c, B, Hq), SharedWorkspace(c, B, Hq, 1)
    new, source, keep = _i([0, 0]), torch.zeros(B, H, 64, dtype=torch.int32, device="cuda"), _i([10, 10])
    k, v = (torch.zeros(2, H, 128, device="cuda") for _ in range(2))
    start, blocks = _i([0, 2]), _i([0])
    freqs = _lib.RopeFreqs(base=10000.0)
    return {
        "append": lambda s: _lib.kvq_append(c.desc, x, x, seq, pos, _lib.APPEND_QUANT, table, B, 4, stream=s),
        "rope": lambda s: _lib.kvq_rope_append(c.desc, rope.desc, q, Hq, out, x, x, pos, seq, pos, _lib.APPEND_QUANT, table,
                                               B, 4, stream=s),
        "rope_table": lambda s: _lib.kvq_rope_table(freqs, 128, 64, rope.table, stream=s),
        "decode": lambda s: _lib.kvq_decode(c.desc, q, B, Hq, lens, table, 4, out, workspace=ws.buf,
                                            workspace_bytes=ws.nbytes, stream=s),
        "shared": lambda s: _lib.kvq_decode_shared(c.desc, q, B, Hq, lens, table, 4, 1, start, blocks, out, lse=lse,
                                                   workspace=sw.buf, workspace_bytes=sw.nbytes, stream=s),
        "prefill": lambda s: _lib.kvq_prefill(c.desc, q, Hq, seq, pos, table, B, 4, out, stream_ctas=-1, stream=s),
        "mass": lambda s: _lib.kvq_attn_mass(c.desc, q, B, Hq, lse, lens, table, 4, mass, stream=s),
        "evict": lambda s: _lib.kvq_evict(c.desc, mass, None, lens, keep, table, B, 4, source, new, stream=s),
        "dequant": lambda s: _lib.kvq_dequant(c.desc, pos, k, v, stream=s),
    }, new


@pytest.mark.parametrize("name", ["append", "rope", "rope_table", "decode", "shared", "prefill", "mass", "evict", "dequant"])
def test_a_launch_that_failed_does_not_fail_the_next(name):
    """A stream whose capture has been invalidated takes no launch; once it has ended, the same call succeeds."""
    from quantized_kv_cache_07_gb300 import _lib
    by_name, new = calls()
    call = by_name[name]
    call(None)
    torch.cuda.synchronize()
    cu = ctypes.CDLL("libcuda.so.1")
    s = torch.cuda.Stream()
    h, graph = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p()
    assert cu.cuStreamBeginCapture_v2(h, 2) == 0
    try:
        assert cu.cuStreamSynchronize(h) != 0       # not allowed in a capture: it is invalid from here on
        with pytest.raises(_lib.KvqError) as e:
            call(s)
        assert e.value.status == _lib.KVQ_ERR_CUDA
    finally:
        assert cu.cuStreamEndCapture(h, ctypes.byref(graph)) != 0
    if name == "evict":
        new.zero_()
    call(None)
    call(s)
    torch.cuda.synchronize()
    assert name != "evict" or new.tolist() == [10, 10]
