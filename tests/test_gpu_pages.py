"""Pages of a cache (kvq_pages_update, kvq_pages_compact, kvq_copy_blocks, kvq_fork_windows).

What they decide is compared, number for number, with the rules of include/kvq.h written out for one row and one page
at a time; what they move is compared byte for byte.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def _i(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def update_rule(refs, table, lens, parent, room=0, window=0, sinks=0, span=0):
    """(refs, table, lens, copies) after kvq_pages_update, or None where the free pages do not suffice; room: of all rows,
    or of each."""
    refs = list(map(int, refs))
    rooms = np.broadcast_to(room, len(lens))
    B, width = table.shape
    most = 16 * width + window
    rows = []
    for r in range(B):
        s = r if parent is None else int(parent[r])
        L = int(lens[s]) if s >= 0 else 0
        L = min(max(L, 0), most)
        count = -(-max(L - window, 0) // 16)
        need = -(-max(min(L + int(rooms[r]), most) - window, 0) // 16) if s >= 0 else 0
        row = [-1] * width
        for j in range(width if s >= 0 else 0):
            if j < count:
                keep = not span or 16 * j < sinks or 16 * (j + 1) > L - span
            else:
                keep = s == r and j < need
            if keep:
                row[j] = int(table[s][j])
        rows.append((s, L, count, need, row))
    for r in range(B):
        for e in table[r]:
            if e >= 0:
                refs[e] -= 1
    for _, _, _, _, row in rows:
        for e in row:
            if e >= 0:
                refs[e] += 1
    shared = [(r, j) for r, (_, _, count, need, row) in enumerate(rows) for j in range(count, need)
              if row[j] >= 0 and refs[row[j]] > 1]
    for r, j in shared:
        refs[rows[r][4][j]] -= 1
        rows[r][4][j] = -1
    last = {}
    for r, (s, L, count, need, row) in enumerate(rows):
        if s >= 0 and max(L - window, 0) % 16 and row[count - 1] >= 0:
            last.setdefault(row[count - 1], []).append(r)
    copying = {r for page, who in last.items() for r in who if not (len(who) == refs[page] and r == who[0])}
    free = [i for i, n in enumerate(refs) if n == 0]
    copies = []
    for r, (s, L, count, need, row) in enumerate(rows):
        places = [count - 1] if r in copying else []
        places += [j for j in range(count, need) if row[j] < 0]
        for j in places:
            if not free:
                return None
            page = free.pop(0)
            if j < count:
                copies.append((row[j], page))
                refs[row[j]] -= 1
            row[j] = page
            refs[page] = 1
    return refs, [x[4] for x in rows], [x[1] for x in rows], copies


class Run:
    """kvq_pages_update of one state, its outputs on the host."""

    def __init__(self, blocks, B, width):
        from quantized_kv_cache_07_gb300 import _lib
        self.lib = _lib
        self.err = _i([0])
        self.ws = torch.full((_lib.kvq_pages_workspace_size(blocks),), 0x5A, dtype=torch.uint8, device="cuda")
        self.out = [torch.full(s, -77, dtype=torch.int32, device="cuda") for s in ((blocks,), (B, width), (B,), (B, 2), (1,))]

    def __call__(self, refs, table, lens, parent, in_place=False, **kw):
        refs_d = _i(refs)
        if isinstance(kw.get("room"), np.ndarray):
            kw["room"] = _i(kw["room"])
        refs_out, table_out, lens_out, copies, num = self.out
        if in_place:
            refs_out = refs_d
        self.lib.kvq_pages_update(refs_d, _i(table), _i(lens), refs_out, table_out, lens_out, copies, num,
                                  parent=None if parent is None else _i(parent), workspace=self.ws, err_word=self.err, **kw)
        torch.cuda.synchronize()
        n = int(num.item())
        return [x.cpu().numpy() for x in (refs_out, table_out, lens_out, copies[:n])]


def same(got, want):
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g, np.asarray(w, dtype=np.int32).reshape(g.shape))


def random_state(rng, B, width, blocks, window=0):
    """Rows that share prefixes at random, cut back at random; refs with a few claims of the user's."""
    refs, table = np.zeros(blocks, int), np.full((B, width), -1)
    ids = list(rng.permutation(blocks))
    lens = np.zeros(B, int)
    for r in range(B):
        if rng.random() < 0.15:
            continue  # a row that is not in use
        lens[r] = rng.integers(0, 16 * width + window + 1)
        count = -(-max(lens[r] - window, 0) // 16)
        have = 0
        if r and rng.random() < 0.7:  # shares the front of an earlier row
            s = rng.integers(0, r)
            held = int((table[s] >= 0).sum())
            have = min(int(rng.integers(0, held + 1)), count)
            table[r, :have] = table[s, :have]
        for j in range(have, min(count + int(rng.integers(0, 3)), width)):
            if len(ids) > 4:
                table[r, j] = ids.pop()
            else:
                lens[r] = min(lens[r], 16 * j + window)
                break
        if rng.random() < 0.3:
            lens[r] = rng.integers(0, lens[r] + 1)  # cut back: pages behind its end stay its own
    for e in table[table >= 0]:
        refs[e] += 1
    for e in rng.choice(blocks, 3, replace=False):
        refs[e] += 1
    return refs, table, lens


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("B,width,blocks", [(1, 1, 1), (1, 40, 64), (5, 7, 50), (16, 33, 700), (70, 130, 9000), (300, 5, 1999)])
def test_update_follows_the_rules(B, width, blocks, seed):
    rng = np.random.default_rng(seed * 101 + B)
    window = int(rng.choice([0, 0, 16, 128]))
    blocks = max(blocks, 4)
    refs, table, lens = random_state(rng, B, width, blocks, window)
    run = Run(blocks, B, width)
    for trial in range(6):
        kind = rng.integers(0, 4)
        parent = [None, rng.integers(-1, B, B), rng.integers(0, B, B), np.full(B, rng.integers(0, B))][kind]
        span = int(rng.choice([0, 0, max(window, 1), window + 37, 500]))
        room = int(rng.choice([0, 1, 16, 40]))
        if rng.random() < 0.3:
            room = rng.integers(0, 50, B)
        kw = dict(room=room, window=window, sinks=int(rng.integers(0, 40)), span=span)
        if rng.random() < 0.8:
            lens = np.minimum(lens, 16 * width + window - np.max(room)).clip(0)
        want = update_rule(refs, table, lens, parent, **kw)
        got = run(refs, table, lens, parent, in_place=bool(rng.integers(0, 2)), **kw)
        err = int(run.err.item())
        run.err.zero_()
        if want is None:
            assert err & run.lib.KVQ_DEVERR_NO_BLOCKS
            same(got, (refs, table, lens, np.zeros((0, 2))))
            lens = lens // 2  # and go on with shorter rows
            continue
        # a last page that a window has freed is reported, and a row that its table has no room for
        whose = np.arange(B) if parent is None else parent
        full = bool(np.any((lens[whose] + room > 16 * width + window) & (whose >= 0)))
        assert err & ~run.lib.KVQ_DEVERR_BLOCK_ID == (run.lib.KVQ_DEVERR_SEQ_LEN if full else 0)
        same(got, want)
        refs, table, lens = (np.asarray(x) for x in want[:3])


@pytest.mark.parametrize("B,width,blocks", [(1500, 4, 9000), (4096, 2, 20000), (9, 20, 150000)])
def test_large_batches_and_pools(B, width, blocks):
    """Several rows a thread, and pools whose counts do not stay in registers."""
    rng = np.random.default_rng(B)
    refs, table, lens = random_state(rng, B, width, blocks)
    run = Run(blocks, B, width)
    for parent in (rng.integers(-1, B, B), np.zeros(B, int), None):
        lens = np.minimum(lens, 16 * width - 1)
        want = update_rule(refs, table, lens, parent, room=1)
        got = run(refs, table, lens, parent, room=1)
        assert run.err.item() == 0
        same(got, want)
        refs, table, lens = (np.asarray(x) for x in want[:3])


def test_too_few_pages_change_nothing():
    run = Run(6, 3, 4)
    table = np.array([[0, 1, -1, -1], [2, -1, -1, -1], [-1, -1, -1, -1]])
    refs, lens = np.array([1, 1, 1, 0, 0, 1]), [20, 16, 0]
    same(run(refs, table, lens, [0, 0, 0]), update_rule(refs, table, lens, [0, 0, 0]))   # two copies, two pages and one freed
    for in_place in (False, True):
        got = run(refs, table, lens, [0, 0, 0], in_place=in_place, room=30)
        same(got, (refs, table, lens, np.zeros((0, 2))))
        assert run.err.item() == run.lib.KVQ_DEVERR_NO_BLOCKS


def test_bad_entries_are_reported():
    lib = Run(1, 1, 1).lib
    run = Run(8, 2, 3)
    good = np.array([[0, 1, -1], [2, -1, -1]])
    refs = [1, 1, 1, 0, 0, 0, 0, 0]
    bad = good.copy()
    bad[0, 1] = 8
    got = run(refs, bad, [16, 10], None)
    assert run.err.item() == 0 or run.err.item() == lib.KVQ_DEVERR_BLOCK_ID
    assert run.err.item() == lib.KVQ_DEVERR_BLOCK_ID and got[1][0].tolist() == [0, -1, -1]
    run.err.zero_()
    got = run(refs, good, [16, 10], [-5, 7])   # no such parents: the rows stay themselves (but for the page kept for nothing)
    assert run.err.item() == lib.KVQ_DEVERR_POSITION
    same(got, update_rule(refs, good, [16, 10], None))
    run.err.zero_()
    got = run(refs, good, [-3, 1000], None)
    assert run.err.item() & lib.KVQ_DEVERR_SEQ_LEN and got[2].tolist() == [0, 48]


@pytest.mark.parametrize("B,width,blocks,seed", [(0, 0, 1, 0), (1, 3, 2, 1), (4, 9, 40, 2), (7, 300, 3001, 3), (20, 64, 20000, 4),
                                                 (3, 5, 8192, 5)])
@pytest.mark.parametrize("used", [0.0, 0.3, 0.7, 1.0])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_follows_the_rules(B, width, blocks, seed, used, in_place):
    from quantized_kv_cache_07_gb300 import _lib
    rng = np.random.default_rng(seed)
    refs = (rng.random(blocks) < used) * rng.integers(1, 4, blocks)
    on = np.nonzero(refs)[0]
    table = np.full((B, width), -1)
    if len(on):
        table = np.where(rng.random((B, width)) < 0.8, rng.choice(on, (B, width)), -1)
    live = len(on)
    holes, tails = [i for i in range(live) if refs[i] == 0], [i for i in range(live, blocks) if refs[i] > 0]
    to = {t: h for h, t in zip(holes, tails)}
    want_refs = refs.copy()
    for t, h in to.items():
        want_refs[h], want_refs[t] = refs[t], 0
    want_table = np.array([[to.get(int(e), int(e)) for e in row] for row in table]).reshape(B, width)
    refs_d, table_d, err = _i(refs), _i(table) if B else None, _i([0])
    moves, counts = torch.full((max(blocks // 2, 1), 2), -9, dtype=torch.int32, device="cuda"), _i([-9, -9])
    ws = torch.full((_lib.kvq_pages_workspace_size(blocks),), 0x5A, dtype=torch.uint8, device="cuda")
    refs_out = refs_d if in_place else torch.full_like(refs_d, -9)
    table_out = table_d if in_place or not B else torch.full_like(table_d, -9)
    _lib.kvq_pages_compact(refs_d, table_d, refs_out, table_out, moves, counts, workspace=ws, err_word=err)
    torch.cuda.synchronize()
    assert counts.tolist() == [len(to), live] and err.item() == 0
    np.testing.assert_array_equal(moves[:len(to)].cpu().numpy(), np.array(list(zip(tails, holes))).reshape(-1, 2))
    assert (moves[len(to):] == -9).all()
    np.testing.assert_array_equal(refs_out.cpu().numpy(), want_refs)
    if B:
        np.testing.assert_array_equal(table_out.cpu().numpy(), want_table)


def test_compact_reports_entries_of_free_pages():
    from quantized_kv_cache_07_gb300 import _lib
    refs, table, err = _i([0, 1, 0, 0]), _i([[1, 3, -1, 9]]), _i([0])
    moves, counts = _i([[0, 0]] * 2), _i([0, 0])
    ws = torch.empty(_lib.kvq_pages_workspace_size(4), dtype=torch.uint8, device="cuda")
    _lib.kvq_pages_compact(refs, table, refs, table, moves, counts, workspace=ws, err_word=err)
    assert table.tolist() == [[0, 3, -1, 9]] and refs.tolist() == [1, 0, 0, 0] and counts.tolist() == [1, 1]
    assert err.item() == _lib.KVQ_DEVERR_BLOCK_ID


def _caches(shapes, blocks, seed=0, **kw):
    from quantized_kv_cache_07_gb300.cache import KVCache
    gen = torch.Generator(device="cuda").manual_seed(seed)
    caches = []
    for H, k_bits, v_bits, asym in shapes:
        c = KVCache(blocks, H, k_bits, v_bits, asym=asym, **kw)
        for t in (c.k_codes, c.v_codes, c.meta, c.k_window, c.v_window):
            if t is not None:
                raw = t.view(torch.uint8)
                raw.copy_(torch.randint(0, 256, raw.shape, dtype=torch.uint8, generator=gen, device="cuda"))
        caches.append(c)
    return caches


@pytest.mark.parametrize("shapes", [
    [(8, 8, 8, False)] * 3, [(2, 4, 4, False)] * 70, [(3, 4, 8, True), (3, 4, 8, True), (1, 16, 16, False), (2, 2, 2, False),
                                                      (2, 2, 2, True), (5, 8, 4, False)]], ids=["int8", "70 layers", "mixed"])
@pytest.mark.parametrize("pairs", [0, 1, 37])
def test_copy_blocks(shapes, pairs):
    from quantized_kv_cache_07_gb300 import _lib
    blocks = 90
    caches = _caches(shapes, blocks)
    rng = np.random.default_rng(pairs)
    ids = rng.permutation(blocks)
    copies = np.stack([rng.choice(ids[40:], 40), ids[:40]], 1)
    copies[pairs:] = [0, 10 ** 6]   # behind the count: not read
    if pairs > 5:
        copies[3] = [-1, 2]
    before = [[None if t is None else t.view(torch.uint8).cpu().numpy().copy() for t in (c.k_codes, c.v_codes, c.meta)]
              for c in caches]
    err = _i([0])
    _lib.kvq_copy_blocks(_lib.CacheList([c.desc for c in caches]), _i(copies), _i([pairs]), err_word=err)
    torch.cuda.synchronize()
    assert err.item() == (_lib.KVQ_DEVERR_BLOCK_ID if pairs > 5 else 0)
    for c, old in zip(caches, before):
        for t, o in zip((c.k_codes, c.v_codes, c.meta), old):
            if o is None:
                continue
            want = o.reshape(c.kv_heads, blocks, -1).copy()
            for s, d in copies[:pairs]:
                if s >= 0:
                    want[:, d] = o.reshape(c.kv_heads, blocks, -1)[:, s]
            np.testing.assert_array_equal(t.view(torch.uint8).cpu().numpy().reshape(want.shape), want)


@pytest.mark.parametrize("B,H,window,layers", [(1, 1, 16, 1), (5, 3, 48, 2), (64, 2, 128, 3), (300, 1, 16, 2), (1500, 1, 16, 1)])
def test_fork_windows(B, H, window, layers):
    from quantized_kv_cache_07_gb300 import _lib
    caches = _caches([(H, 8, 8, False)] * layers, 4, window=window, window_batch=B + 2)
    rng = np.random.default_rng(B)
    for parent in (rng.integers(-1, B, B), rng.permutation(B), np.zeros(B, int), np.arange(B), np.full(B, -1)):
        before = [[t.view(torch.uint8).cpu().numpy().reshape(B + 2, -1) for t in (c.k_window, c.v_window)] for c in caches]
        err = _i([0])
        bad = parent.copy()
        if B > 4:
            bad[2] = B  # no such row: left as it is
        _lib.kvq_fork_windows(_lib.CacheList([c.desc for c in caches]), _i(bad), B, err_word=err)
        torch.cuda.synchronize()
        assert err.item() == (_lib.KVQ_DEVERR_POSITION if B > 4 else 0)
        source = np.where((bad >= 0) & (bad < B), bad, np.arange(B))
        for c, old in zip(caches, before):
            for t, o in zip((c.k_window, c.v_window), old):
                got = t.view(torch.uint8).cpu().numpy().reshape(B + 2, -1)
                np.testing.assert_array_equal(got[:B], o[source])
                np.testing.assert_array_equal(got[B:], o[B:])


def test_captured_with_its_copies_and_on_two_streams():
    """Update and copies replayed from a graph, with other parents each time; two workspaces on two streams."""
    from quantized_kv_cache_07_gb300 import _lib
    blocks, B, width = 500, 12, 30
    rng = np.random.default_rng(5)
    refs, table, lens = random_state(rng, B, width, blocks)
    lens = np.minimum(lens, 16 * width - 16)
    caches = _caches([(2, 8, 8, False)] * 4, blocks)
    cl = _lib.CacheList([c.desc for c in caches])
    refs_d, table_d, lens_d, parent_d = _i(refs), _i(table), _i(lens), _i(np.zeros(B))
    runs = [Run(blocks, B, width) for _ in range(2)]

    def call(run, stream=None, copy=True):
        _lib.kvq_pages_update(refs_d, table_d, lens_d, *run.out, parent=parent_d, room=16, workspace=run.ws, stream=stream)
        if copy:
            _lib.kvq_copy_blocks(cl, run.out[3], run.out[4], stream=stream)
    call(runs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(runs[0])
    for trial in range(4):
        parent = rng.integers(-1, B, B)
        parent_d.copy_(_i(parent))
        want = update_rule(refs, table, lens, parent, room=16)
        before = caches[3].k_codes.cpu().numpy().reshape(2, blocks, -1).copy()
        graph.replay()
        torch.cuda.synchronize()
        same([x.cpu().numpy() for x in runs[0].out[:3]], want[:3])
        for s, d in want[3]:
            before[:, d] = before[:, s]
        np.testing.assert_array_equal(caches[3].k_codes.cpu().numpy().reshape(2, blocks, -1), before)
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(10):
            for run, s in zip(runs, streams):
                call(run, s, copy=False)
        torch.cuda.synchronize()
        for run in runs:
            same([x.cpu().numpy() for x in run.out[:3]], want[:3])
