"""The cache operators as a serving loop uses them: rotary write, decode over a shared prefix, attention mass, eviction.

The reference keeps every sequence's tokens in the order of its slots, in float64 from
what the cache gives back (kvq_dequant); rotated keys are checked against the formula.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

H, G, B, D, T = 2, 4, 5, 128, 16
PREFIX = 3                      # blocks shared by sequences 0..3; sequence 4 stands alone


def turned(x, pos, R=64, base=10000.0):
    """x [n, heads, 128] turned by pos [n], halves of the first R dims, float64."""
    f = base ** (-2.0 * np.arange(R // 2) / R)
    c, s = np.cos(pos[:, None] * f)[:, None], np.sin(pos[:, None] * f)[:, None]
    y = x.copy()
    y[..., :R // 2] = x[..., :R // 2] * c - x[..., R // 2:R] * s
    y[..., R // 2:R] = x[..., :R // 2] * s + x[..., R // 2:R] * c
    return y


@pytest.mark.parametrize("k_bits,v_bits,asym", [(8, 8, False), (4, 4, True), (4, 8, False)])
def test_serving_steps_with_eviction(k_bits, v_bits, asym):
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache, RopeTable, SharedWorkspace
    rng = np.random.default_rng(k_bits + 10 * v_bits)
    mbps, own = 9, [40, 1, 17, 33]
    stream = torch.cuda.Stream()
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    with torch.cuda.stream(stream):
        cache = KVCache(PREFIX + B * mbps, H, k_bits, v_bits, asym=asym)
        rope = RopeTable(4096, rotary_dim=64)
        ids = rng.permutation(PREFIX + B * mbps).astype(np.int32)
        table = ids[PREFIX:].reshape(B, mbps).copy()
        table[:4, :PREFIX] = ids[:PREFIX]
        table_t, err = i32(table), torch.zeros(1, dtype=torch.int32, device="cuda")
        keys, vals = [np.zeros((0, H, D))] * B, [np.zeros((0, H, D))] * B
        qmax = lambda bits: (2 ** bits - 1 if asym else 2 ** (bits - 1) - 1)

        def write(seq, slot, pos):
            """Rows of one fused projection through kvq_rope_append; the turned queries, stored keys and values."""
            n = len(seq)
            x = torch.from_numpy(rng.standard_normal((n, (G + 2) * H * D)).astype(np.float32)).bfloat16().cuda()
            q, k, v = x[:, :G * H * D], x[:, G * H * D:(G + 1) * H * D], x[:, (G + 1) * H * D:]
            q_out = torch.empty(n, G * H, D, dtype=torch.bfloat16, device="cuda")
            _lib.kvq_rope_append(cache.desc, rope.desc, q, G * H, q_out, k, v, i32(pos), i32(seq), i32(slot),
                                 _lib.APPEND_QUANT, table_t, B, mbps, err_word=err)
            where = i32(table[seq, np.asarray(slot) // T] * T + np.asarray(slot) % T)
            kr, vr = (torch.empty(n, H, D, device="cuda") for _ in range(2))
            _lib.kvq_dequant(cache.desc, where, kr, vr)
            want_q = turned(q.double().cpu().numpy().reshape(n, G * H, D), np.asarray(pos, float))
            want_k = turned(k.double().cpu().numpy().reshape(n, H, D), np.asarray(pos, float))
            # half a bf16 step of the value, and what the table's float32 entries add (2^-24 of each term)
            near = lambda y: 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * np.abs(y).max()
            assert np.all(np.abs(q_out.double().cpu().numpy() - want_q) <= near(want_q))
            # half a code step, on the range of the row, and the key's own rounding
            span = (want_k.max(-1) - want_k.min(-1) if asym else np.abs(want_k).max(-1))[..., None] * (1 + 2.0 ** -7)
            assert np.all(np.abs(kr.double().cpu().numpy() - want_k) <= 0.5 * span / qmax(k_bits) * (1 + 2.0 ** -20)
                          + near(want_k))
            return q_out, kr.double().cpu().numpy(), vr.double().cpu().numpy()

        # the shared prefix once, then every sequence's own prompt, in one call of 140 rows
        seq = [0] * (PREFIX * T) + sum([[b] * own[b] for b in range(4)], []) + [4] * 1
        slot = list(range(PREFIX * T)) + sum([list(range(PREFIX * T, PREFIX * T + n)) for n in own], []) + [0]
        _, kr, vr = write(np.array(seq), slot, slot)
        head = PREFIX * T
        for b in range(4):
            rows = list(range(head)) + [r for r in range(head, len(seq)) if seq[r] == b]
            keys[b], vals[b] = kr[rows], vr[rows]
        keys[4], vals[4] = kr[-1:], vr[-1:]
        pos_next = np.array([len(k) for k in keys])
        cap = mbps * T
        mass = torch.zeros(B, H, cap, device="cuda")
        ref_mass = np.zeros((B, H, cap))
        token_pos = i32(np.broadcast_to(np.arange(cap), (B, H, cap))).contiguous()
        ws = SharedWorkspace(cache, B, G * H, 1)
        evicted = False
        for step in range(6):
            lens = np.array([len(k) for k in keys])
            q, kr, vr = write(np.arange(B), lens, pos_next)     # the new token of every sequence, at its true position
            for b in range(B):
                keys[b], vals[b] = np.concatenate([keys[b], kr[b:b + 1]]), np.concatenate([vals[b], vr[b:b + 1]])
                token_pos[b, :, lens[b]] = int(pos_next[b])
                mass[b, :, lens[b]] = 0.0
                ref_mass[b, :, lens[b]] = 0.0
            lens, pos_next = lens + 1, pos_next + 1
            out = torch.empty(B, G * H, D, device="cuda")
            lse = torch.empty(B, G * H, device="cuda")
            _lib.kvq_decode_shared(cache.desc, q, B, G * H, i32(lens), table_t, mbps, 1, i32([0, 4]), i32([PREFIX]), out,
                                   lse=lse, workspace=ws.buf, workspace_bytes=ws.nbytes, err_word=err)
            _lib.kvq_attn_mass(cache.desc, q, B, G * H, lse, i32(lens), table_t, mbps, mass, decay=0.5, err_word=err)
            got, got_mass, qd = out.double().cpu().numpy(), mass.double().cpu().numpy(), q.double().cpu().numpy()
            for b in range(B):
                for h in range(H):
                    s = qd[b, h * G:(h + 1) * G] @ keys[b][:, h].T / np.sqrt(D)
                    p = np.exp(s - s.max(1, keepdims=True))
                    p /= p.sum(1, keepdims=True)
                    assert np.max(np.abs(got[b, h * G:(h + 1) * G] - p @ vals[b][:, h])) <= 2e-3
                    n = lens[b]
                    ref_mass[b, h, :n] = 0.5 * ref_mass[b, h, :n] + p.sum(0)
                    # the log-sum-exp is good to 2e-3: each weight to exp(2e-3) - 1
                    assert np.all(np.abs(got_mass[b, h, :n] - ref_mass[b, h, :n]) <= 2.1e-3 * ref_mass[b, h, :n] + 1e-9)
            if step != 2:
                continue
            # keep half of what lies behind the prefix; its tokens, the first of sequence 4 and the last three stay
            keep = head + (lens - head) // 2
            keep[4] = lens[4] - 1
            source, new = torch.zeros(B, H, cap, dtype=torch.int32, device="cuda"), i32(np.zeros(B))
            _lib.kvq_evict(cache.desc, mass, mass, i32(lens), i32(keep), table_t, B, mbps, source, new, protect_first=head,
                           protect_recent=3, token_pos=token_pos, token_pos_out=token_pos, next_pos=i32(pos_next),
                           err_word=err)
            new, source = new.cpu().numpy(), source.cpu().numpy()
            for b in range(B):
                assert new[b] == max(min(lens[b], keep[b]), 0)
                k2, v2 = np.empty((new[b], H, D)), np.empty((new[b], H, D))
                for h in range(H):
                    src = source[b, h, :new[b]]
                    evicted = evicted or not np.array_equal(src, np.arange(new[b]))
                    stay = min(head, new[b])
                    assert len(set(src)) == len(src) and np.array_equal(src[:stay], np.arange(stay))
                    k2[:, h], v2[:, h] = keys[b][src, h], vals[b][src, h]
                    ref_mass[b, h, :new[b]] = ref_mass[b, h, src]
                    np.testing.assert_array_equal(token_pos[b, h, :new[b]].cpu().numpy(), src)
                keys[b], vals[b] = k2, v2
                at = np.arange(new[b])
                kr, vr = (torch.empty(new[b], H, D, device="cuda") for _ in range(2))
                _lib.kvq_dequant(cache.desc, i32(table[b, at // T] * T + at % T), kr, vr)
                np.testing.assert_array_equal(kr.double().cpu().numpy(), k2)
                np.testing.assert_array_equal(vr.double().cpu().numpy(), v2)
        assert evicted and int(err) == 0


def test_two_streams_at_once():
    """Calls of two loops on two streams, with workspaces and caches of their own: the bits of the calls one by one."""
    from quantized_kv_cache_07_gb300 import _lib
    from quantized_kv_cache_07_gb300.cache import KVCache, RopeTable, SharedWorkspace
    batch, heads, group, mbps, prefix = 20, 2, 4, 24, 16
    rope = RopeTable(4096)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    def loop(seed, bits):
        g = torch.Generator(device="cuda").manual_seed(seed)
        cache = KVCache(batch * mbps, heads, bits, bits)
        ws = SharedWorkspace(cache, batch, heads * group, 1)
        table = torch.arange(batch * mbps, device="cuda").int().view(batch, mbps)
        table[:, :prefix] = table[0, :prefix]
        n = prefix * T + batch * 100
        seq = i32([0] * (prefix * T) + sum([[b] * 100 for b in range(batch)], []))
        slot = i32(list(range(prefix * T)) + list(range(prefix * T, prefix * T + 100)) * batch)
        k, v = (torch.randn(n, heads, D, generator=g, device="cuda").bfloat16() for _ in range(2))
        q = torch.randn(batch, heads * group, D, generator=g, device="cuda").bfloat16()
        lens = torch.randint(prefix * T + 20, prefix * T + 101, (batch,), generator=g, device="cuda").int()
        start, blocks, keep = i32([0, batch]), i32([prefix]), i32([prefix * T + 15] * batch)
        out = torch.zeros(batch, heads * group, D, device="cuda")
        lse = torch.zeros(batch, heads * group, device="cuda")
        mass = torch.zeros(batch, heads, mbps * T, device="cuda")
        source, new = torch.zeros(batch, heads, mbps * T, dtype=torch.int32, device="cuda"), torch.zeros_like(lens)

        def run():
            mass.zero_()
            _lib.kvq_rope_append(cache.desc, rope.desc, None, 0, None, k, v, None, seq, slot, _lib.APPEND_QUANT, table,
                                 batch, mbps)
            _lib.kvq_decode_shared(cache.desc, q, batch, heads * group, lens, table, mbps, 1, start, blocks, out, lse=lse,
                                   workspace=ws.buf, workspace_bytes=ws.nbytes)
            _lib.kvq_attn_mass(cache.desc, q, batch, heads * group, lse, lens, table, mbps, mass)
            _lib.kvq_evict(cache.desc, mass, mass, lens, keep, table, batch, mbps, source, new, protect_first=prefix * T)
        return run, lambda: [t.clone() for t in (out, lse, mass, source, new, cache.k_codes, cache.v_codes)]

    loops = [loop(1, 8), loop(2, 4)]
    want = []
    for run, read in loops:
        run()
        torch.cuda.synchronize()
        want.append(read())
    streams = [torch.cuda.Stream() for _ in loops]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (run, _) in zip(streams, loops):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for (_, read), w in zip(loops, want):
        for a, b in zip(read(), w):
            assert torch.equal(a, b)
