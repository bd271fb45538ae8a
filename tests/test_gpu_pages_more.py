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


def both(calls, times=20000):
    """Each call over and over in a thread and on a stream of its own; the errors."""
    import threading
    failed, start = [], threading.Barrier(len(calls))

    def go(call):
        stream = torch.cuda.Stream()
        start.wait()
        try:
            for _ in range(times):
                call(stream)
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=go, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return failed


def test_two_threads_update_batches_of_different_sizes():
    """The launch of a large batch beside that of a small one: both go through."""
    from quantized_kv_cache_07_gb300 import _lib
    calls = []
    for B in (4096, 1, 1, 1):
        run = Run(4, B, 1)
        i = lambda n, v: torch.full((n,), v, dtype=torch.int32, device="cuda")
        refs, table, lens = i(4, 0), i(B, -1).view(B, 1), i(B, 0)

        def call(stream, run=run, args=(refs, table, lens)):
            _lib.kvq_pages_update(*args, *run.out, workspace=run.ws, stream=stream)
        calls.append(call)
    torch.cuda.synchronize()
    assert both(calls) == []


def test_two_threads_fork_windows_of_different_batches():
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache
    calls = []
    for B in (4096, 1, 1, 1):
        cache = KVCache(1, 1, 8, 8, window=16, window_batch=B)
        parent = torch.arange(B, dtype=torch.int32, device="cuda")

        def call(stream, caches=_lib.CacheList([cache.desc]), parent=parent, B=B, cache=cache):
            _lib.kvq_fork_windows(caches, parent, B, stream=stream)
        calls.append(call)
    torch.cuda.synchronize()
    assert both(calls) == []


def test_empty_blocks_of_a_larger_room_are_given_back():
    """Room for 64 tokens, then for one: a row keeps the blocks of its tokens and of this call's room; the others are
    free at once, for another row of the same call too.  The same room again changes nothing."""
    blocks, width = 16, 8
    run, none = Run(blocks, 2, width), [-1] * 8
    refs, table, lens = np.zeros(blocks, int), np.array([[9, 3] + [-1] * 6, none]), np.array([20, 0])
    refs[[9, 3]] = 1
    for _ in range(2):
        refs, table, lens, copies = (x.copy() for x in run(refs, table, lens, None, room=np.array([64, 0])))
        assert table.tolist() == [[9, 3, 0, 1, 2, 4, -1, -1], none] and len(copies) == 0
        assert np.nonzero(refs)[0].tolist() == [0, 1, 2, 3, 4, 9]
    refs, table, lens, copies = (x.copy() for x in run(refs, table, lens, None, room=np.array([1, 16])))
    assert table.tolist() == [[9, 3] + [-1] * 6, [0] + [-1] * 7] and np.nonzero(refs)[0].tolist() == [0, 3, 9]
    assert lens.tolist() == [20, 0] and run.err.item() == 0
