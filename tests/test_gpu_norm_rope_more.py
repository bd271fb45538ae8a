"""Normed rotary write: a query's bits are its own, whatever else the call holds."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from synth import f32_to_bf16_bits  # noqa: E402
from test_gpu_norm_rope import heads_of, weights_of  # noqa: E402
from test_gpu_rope import _i, _t  # noqa: E402


@pytest.mark.parametrize("Hq,R,inter,kind", [(32, 128, False, "all"), (32, 64, True, "all"), (33, 104, False, "one"),
                                             (32, 128, True, "none"), (24, 96, False, "heads"), (32, 8, True, "heads")])
def test_a_querys_bits_do_not_depend_on_the_rows_beside_it(Hq, R, inter, kind):
    """A prompt in one call, in chunks and row by row: the same bits of every query."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import HeadNorm, KVCache, RopeTable
    rng = np.random.default_rng(R)
    n = 3 * 152 * 64 // Hq + 70   # many rows of their own kernel; the chunks below that
    rope, norm = RopeTable(3000, rotary_dim=R, interleaved=inter), HeadNorm(weights_of(rng, kind, Hq, 1)[0])
    bits = heads_of(rng, n, Hq)
    bits[7::50] = f32_to_bf16_bits((rng.standard_normal(bits[7::50].shape) * 1e18).astype(np.float32))  # squares that overflow
    q, pos, c = _t(bits), _i(rng.integers(0, 3000, n)), KVCache(1, 1, 8, 8)

    def call(rows):
        out = torch.zeros(rows.stop - rows.start, Hq, 128, dtype=torch.bfloat16, device="cuda")
        _lib.kvq_norm_rope_append(c.desc, rope.desc, norm.desc, q[rows], Hq, out, None, None, pos[rows], None, None,
                                  _lib.APPEND_QUANT, None, 0, 0)
        return out
    whole = call(slice(0, n))
    for step, last in ((200, n), (1, 20)):
        parts = torch.cat([call(slice(r, min(r + step, last))) for r in range(0, last, step)])
        assert torch.equal(parts.view(torch.int16), whole[:last].view(torch.int16)), step
