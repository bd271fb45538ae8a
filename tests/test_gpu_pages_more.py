"""Pages of a cache (kvq_pages_update and what moves them) at the ends of their arguments and between calls."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from test_gpu_pages import Run, same, update_rule  # noqa: E402


@pytest.mark.parametrize("window", [0, 32])
@pytest.mark.parametrize("sinks", [2 ** 31 - 1, 2 ** 31 - 15, 2 ** 31 - 16, 10 ** 9, 128, 100])
def test_sinks_beyond_every_length_free_nothing(sinks, window):
    """A span that hides most of a row, and as many sinks as an argument can hold: every block of every row stays."""
    B, width, blocks = 3, 9, 64
    run, lens = Run(blocks, B, width), np.array([130, 77, 16]) if window == 0 else np.array([130, 109, 40])
    table, page = np.full((B, width), -1), iter(range(blocks))
    for r in range(B):
        for j in range(-(-(lens[r] - window) // 16)):
            table[r, j] = next(page)
    refs = np.bincount(table[table >= 0], minlength=blocks)
    kw = dict(room=1, window=window, sinks=sinks, span=max(window, 5))
    got = run(refs, table, lens, None, **kw)
    assert run.err.item() == 0
    same(got, update_rule(refs, table, lens, None, **kw))
    if sinks >= 128:
        assert np.array_equal(got[1][table >= 0], table[table >= 0])
