"""Sliding-window serving as a program runs it: prompts in chunks, normed rotary write, attention with sinks, rows that
fork, end and start again on shared pages, pages freed behind the window, a compaction, two layers.

The other side keeps every row's keys and values apart: each step writes them into a cache of its own pages from
scratch (kvq_append of the bf16 vectors that a bf16 cache gave back) and decodes there.  Blocks are the same bytes
under other numbers, so outputs are compared bit for bit.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

B, H, G, D, LAYERS = 7, 2, 4, 128, 2


def _i(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


class Apart:
    """Keys and values of every row and layer as bf16 tensors, and decode of them in pages of their own."""

    def __init__(self, fmt, window, mb):
        self.fmt, self.window, self.mb = fmt, window, mb
        self.rows = [[[] for _ in range(LAYERS)] for _ in range(B)]

    def decode(self, layer, q, sinks, span, fresh):
        from quantized_kv_cache_07_gb300 import _lib
        from quantized_kv_cache_07_gb300.cache import DecodeWorkspace
        cache, W = fresh(), self.window
        table = torch.arange(B * self.mb, device="cuda").int().view(B, self.mb)
        lens = [len(r[layer]) for r in self.rows]
        for mode in ("QUANT", "RING"):
            at = [(b, p) for b in range(B) for p in range(lens[b]) if (p >= lens[b] - W) == (mode == "RING")]
            if at:
                k, v = (torch.stack([self.rows[b][layer][p][x] for b, p in at]) for x in range(2))
                _lib.kvq_append(cache.desc, k, v, _i([b for b, _ in at]), _i([p for _, p in at]),
                                getattr(_lib, "APPEND_" + mode), table, B, self.mb)
        out, lse = torch.empty(B, G * H, D, device="cuda"), torch.empty(B, G * H, device="cuda")
        ws = DecodeWorkspace(cache, B, G * H)
        _lib.kvq_decode_sinks(cache.desc, q, B, G * H, _i(lens), table, self.mb, sinks, span, out, lse=lse, workspace=ws.buf,
                              workspace_bytes=ws.nbytes)
        return out, lse


@pytest.mark.parametrize("fmt,window", [(dict(k_bits=8, v_bits=8), 0), (dict(k_bits=4, v_bits=8, asym=True), 0),
                                        (dict(k_bits=8, v_bits=4), 32), (dict(k_bits=16, v_bits=16), 16)])
def test_serving_with_shared_pages(fmt, window):
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import DecodeWorkspace, HeadNorm, KVCache, Pages, RopeTable
    rng = np.random.default_rng(fmt["k_bits"] + window)
    gen = torch.Generator(device="cuda").manual_seed(window + 3)
    blocks, mb, sinks, span = 70, 24, 5, 70
    fresh = lambda n=None: KVCache(n or B * mb, H, window=window, window_batch=B, **fmt)
    caches, keep = [fresh(blocks) for _ in range(LAYERS)], KVCache(40, H, 16, 16)  # `keep` gives the written vectors back
    pages, apart = Pages(caches, B, mb, sinks=sinks, span=span), Apart(fmt, window, mb)
    rope, err = RopeTable(1024, rotary_dim=64), _i([0])
    norms = [HeadNorm(torch.rand(G * H, D, generator=gen, device="cuda") + 0.5,
                      torch.rand(H, D, generator=gen, device="cuda") + 0.5, eps=1e-5) for _ in range(LAYERS)]
    ws = DecodeWorkspace(caches[0], B, G * H)

    def write(layer, seq, pos, modes):
        """Rows (seq, pos) through the normed rotary write; the turned queries.  modes: (mode, rows) in turn."""
        n = len(seq)
        x = torch.randn(n, (G + 2) * H * D, generator=gen, device="cuda").mul(2).bfloat16()
        q, k, v = x[:, :G * H * D], x[:, G * H * D:(G + 1) * H * D], x[:, (G + 1) * H * D:]
        q_out = torch.empty(n, G * H, D, dtype=torch.bfloat16, device="cuda")
        norm = norms[layer]
        _lib.kvq_norm_rope_append(keep.desc, rope.desc, norm.desc, q, G * H, q_out, k, v, _i(pos), _i([0] * n), _i(range(n)),
                                  _lib.APPEND_QUANT, _i([range(40)]), 1, 40)
        for mode, rows in modes:
            if len(rows):
                at = torch.as_tensor(rows, device="cuda")
                _lib.kvq_norm_rope_append(caches[layer].desc, rope.desc, norm.desc, None, 0, None, k[at].contiguous(),
                                          v[at].contiguous(), None, _i(np.asarray(seq)[rows]), _i(np.asarray(pos)[rows]), mode,
                                          pages.table, B, mb, err_word=err)
        kr, vr = (torch.empty(n, H, D, device="cuda") for _ in range(2))
        _lib.kvq_dequant(keep.desc, _i(range(n)), kr, vr)
        for r, b in enumerate(seq):
            apart.rows[b][layer].append((kr[r].bfloat16(), vr[r].bfloat16()))
        return q_out

    def admit(row, n):
        """A prompt of n tokens into an empty row, in one chunk; without a bf16 window its attention too."""
        rooms = np.zeros(B)
        rooms[row] = n
        pages.update(room=_i(rooms), err_word=err)
        pos = list(range(n))
        for layer in range(LAYERS):
            stored = max(n - window, 0)
            q = write(layer, [row] * n, pos, [(_lib.APPEND_QUANT, pos[:stored])] + (
                [(_lib.APPEND_RING, pos[stored:])] if window else []))
            if window:
                continue
            out, want = torch.empty(n, G * H, D, device="cuda"), torch.empty(n, G * H, D, device="cuda")
            nb = _lib.kvq_prefill_workspace_size(caches[layer].desc, n, G * H)
            w = torch.zeros(max(nb, 16), dtype=torch.uint8, device="cuda")
            _lib.kvq_prefill_sinks(caches[layer].desc, q, G * H, _i([row] * n), _i(pos), pages.table, B, mb, sinks, span, out,
                                   workspace=w, workspace_bytes=nb, err_word=err)
            other = fresh()
            table = torch.arange(B * mb, device="cuda").int().view(B, mb)
            k, v = (torch.stack([t[x] for t in apart.rows[row][layer]]) for x in range(2))
            _lib.kvq_prefill_sinks(other.desc, q, G * H, _i([row] * n), _i(pos), table, B, mb, sinks, span, want, k_new=k,
                                   v_new=v, workspace=w, workspace_bytes=nb, err_word=err)
            assert torch.equal(out, want)
        pages.lens[row] = n

    admit(0, 100)
    admit(3, 37)
    for step in range(40):
        live = [b for b in range(B) if apart.rows[b][0]]
        parent = None
        if step % 5 == 3:   # rows fork, end and stay
            parent = np.array([rng.choice(live + [b]) if rng.random() < 0.6 else (b if rng.random() < 0.8 else -1)
                               for b in range(B)])
            parent[rng.integers(0, B)] = live[0]  # one at least lives on
            apart.rows = [[list(y) for y in apart.rows[p]] if p >= 0 else [[] for _ in range(LAYERS)] for p in parent]
        live = np.array([bool(apart.rows[b][0]) for b in range(B)])
        pages.update(parent=None if parent is None else _i(parent), room=_i(live), err_word=err)
        if step == 21:
            used = int((pages.refs > 0).sum())
            pages.compact(err_word=err)
            assert pages.counts[1].item() == used and bool((pages.refs[:used] > 0).all())
            assert not bool((pages.refs[used:] > 0).any()) and int(pages.table.max()) < used
        # every page is held as often as the table says
        held = torch.bincount(pages.table[pages.table >= 0].flatten(), minlength=blocks)
        assert torch.equal(held.int(), pages.refs)
        # the rows that go on get a token each
        seq = np.nonzero(live)[0]
        pos = np.array([len(apart.rows[b][0]) for b in seq])
        assert pages.lens.tolist() == [len(apart.rows[b][0]) for b in range(B)]
        for layer in range(LAYERS):
            q = write(layer, seq, pos, [(_lib.APPEND_STEP if window else _lib.APPEND_QUANT, np.arange(len(seq)))])
            full = torch.zeros(B, G * H, D, dtype=torch.bfloat16, device="cuda")
            full[torch.as_tensor(seq, device="cuda")] = q
            lens = pages.lens + _i(live)
            out, lse = torch.empty(B, G * H, D, device="cuda"), torch.empty(B, G * H, device="cuda")
            _lib.kvq_decode_sinks(caches[layer].desc, full, B, G * H, lens, pages.table, mb, sinks, span, out, lse=lse,
                                  workspace=ws.buf, workspace_bytes=ws.nbytes, err_word=err)
            want, want_lse = apart.decode(layer, full, sinks, span, fresh)
            assert torch.equal(out, want) and torch.equal(lse, want_lse), (step, layer)
        pages.lens += _i(live)
        if step in (10, 26) and not live.all():
            admit(int(np.nonzero(~live)[0][0]), 50 + step)
    assert err.item() == 0
    # a window of 70 tokens, and the sinks: no row holds more than 6 pages and the one it writes to
    assert int((pages.table >= 0).sum(1).max()) <= 8


def test_a_batch_without_pages_left_stays_as_it_is():
    """Too few pages for a fork: tables, lengths and rings as they were, the error reported, and the next step goes on."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache, Pages
    cache = KVCache(4, 1, 8, 8, window=16, window_batch=3)
    pages, err = Pages([cache], 3, 8), _i([0])
    pages.update(room=_i([40, 0, 0]), err_word=err)
    pages.lens[0] = 40      # 24 tokens in two pages, 16 in the ring
    rings = torch.randint(0, 256, cache.k_window.view(torch.uint8).shape, dtype=torch.uint8, device="cuda")
    cache.k_window.view(torch.uint8).copy_(rings)
    before = [t.clone() for t in (pages.table, pages.lens, pages.refs)]
    pages.update(parent=_i([0, 0, 0]), room=16, err_word=err)   # three last pages and their next ones: four more than there are
    assert err.item() == _lib.KVQ_DEVERR_NO_BLOCKS
    for t, b in zip((pages.table, pages.lens, pages.refs), before):
        assert torch.equal(t, b)
    assert torch.equal(cache.k_window.view(torch.uint8), rings) and pages.parents.tolist() == [0, 1, 2]
    err.zero_()
    pages.update(parent=_i([0, 0, -1]), room=8, err_word=err)
    assert err.item() == 0 and pages.lens.tolist() == [40, 40, 0] and pages.refs.tolist() == [2, 1, 1, 0]
    row = rings.view(3, -1)
    assert torch.equal(cache.k_window.view(torch.uint8).view(3, -1), torch.stack([row[0], row[0], row[2]]))
