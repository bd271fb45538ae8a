"""Cases of the operators of sliding-window serving: normed rotary write, attention with sinks, and pages of a cache.

A case names its operator in "op":
  norm     norm each head of queries and keys, rotate them by their positions and write keys and values into the cache
           (kvq_norm_rope_append)
  decode   one decode step over a sliding window and the first tokens of each sequence (kvq_decode_sinks)
  prefill  the same for a chunk of new tokens (kvq_prefill_sinks)
  fork     give each row of a batch its parent's pages, with a page of its own to write to, in every layer
           (kvq_pages_update, kvq_copy_blocks, kvq_fork_windows)
  compact  move the pages in use to the front of their pools, in every layer (kvq_pages_compact, kvq_copy_blocks)

Head dimension 128 and 16-token blocks (pages), as everywhere in this package.  Caches are made in their stored byte
order (include/kvq.h), so both forms read the same bytes.
"""
import math

import torch

own = False

D, T = 128, 16


# ------------------------------------------------------------------ the cases

def listed():
    heads = dict(q_heads=32, kv_heads=8, k_bits=8, v_bits=8, asym=False, factor=False)
    norm = dict(heads, op="norm")
    decode = dict(heads, op="decode")
    prefill = dict(heads, op="prefill")
    fork = dict(heads, op="fork", window=0, sinks=0, span=0)
    compact = dict(heads, op="compact")
    return [
        # the new token of each of 64 running sequences, one weight for all heads
        dict(norm, name="norm step of 64", n=64, max_pos=32768, rotary=128, interleaved=False, per_head=False),
        # prompts of odd length into a 4-bit cache, half of each head rotated in neighbouring pairs, a weight for each head
        dict(norm, name="norm prompts of 4099, int4", n=4099, max_pos=8192, rotary=64, interleaved=True, per_head=True,
             k_bits=4, v_bits=4),
        # one short sequence, hardly longer than its window: latency
        dict(decode, name="sinks 1 of 700", batch=1, low=700, high=700, sinks=4, span=512, q_heads=4, kv_heads=4),
        # a batch of ragged contexts, 4-bit cache with a key factor, windows that end inside blocks
        dict(decode, name="sinks 33 of 1k-20k, int4", batch=33, low=1000, high=20000, sinks=5, span=1000, k_bits=4,
             v_bits=4, factor=True),
        # a full batch far into its contexts
        dict(decode, name="sinks 64 of 32768", batch=64, low=20000, high=32768, sinks=4, span=4096),
        # short prompts whole, windows much smaller than they are
        dict(prefill, name="sinks prompts of 700", seqs=3, n=700, start=0, sinks=3, span=200, asym=True),
        # a chunk of one long prompt
        dict(prefill, name="sinks chunk of 2048", seqs=1, n=2048, start=16384, sinks=4, span=4096),
        # the four beams of one request, few layers: latency
        dict(fork, name="fork 4 beams", layers=4, groups=1, beams=4, low=300, high=700, width=64),
        # beams of several requests behind a bf16 window, 4-bit cache, the pages behind the sliding window freed
        dict(fork, name="fork 12 x 4 beams, windows", layers=8, groups=12, beams=4, low=1000, high=4000, width=300,
             window=128, sinks=16, span=1024, k_bits=4, v_bits=4),
        # 64 answers to one prompt, every layer of a model
        dict(fork, name="fork 64 samples", layers=32, groups=1, beams=64, low=3001, high=3001, width=2048, fan=True),
        # one layer's small pool
        dict(compact, name="compact 300 pages", layers=1, blocks=300, used=0.5, batch=4, width=64),
        # pools that lost half of their sequences
        dict(compact, name="compact 4000 pages", layers=8, blocks=4000, used=0.6, batch=48, width=512),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "decode", "prefill", "fork", "compact"])
    q_heads, kv_heads = rng.choice([(32, 8), (64, 8), (16, 8), (8, 8), (8, 2), (4, 4), (24, 8), (10, 2)])
    k_bits, v_bits = rng.choice([(8, 8), (4, 4), (4, 8), (8, 4)])
    case = dict(op=op, q_heads=q_heads, kv_heads=kv_heads, k_bits=k_bits, v_bits=v_bits,
                asym=rng.random() < 0.3, factor=rng.random() < 0.3)
    if op == "norm":
        case.update(n=_log(rng, 1, 4096), max_pos=_log(rng, 5000, 131072), rotary=rng.choice([32, 64, 96, 128]),
                    interleaved=rng.random() < 0.5, per_head=rng.random() < 0.5)
    elif op == "decode":
        high = _log(rng, 100, 32768)
        case.update(batch=_log(rng, 1, 48), low=rng.randint(1, high), high=high, sinks=rng.randint(0, 40),
                    span=_log(rng, 16, 3000))
    elif op == "prefill":
        n = _log(rng, 17, 1500)
        case.update(seqs=rng.randint(1, min(4, n)), n=n, start=rng.choice([0, _log(rng, 1, 8000)]),
                    sinks=rng.randint(0, 40), span=_log(rng, 16, 2500))
    elif op == "fork":
        fan = rng.random() < 0.5
        high = _log(rng, 200, 3000)
        case.update(layers=_log(rng, 1, 10), groups=1 if fan else rng.randint(1, 8), beams=rng.randint(2, 16 if fan else 6),
                    low=rng.randint(100, high), high=high, width=rng.randint(250, 1500), fan=fan,
                    window=rng.choice([0, 0, 32, 128]), sinks=rng.randint(0, 30), span=rng.choice([0, 128, 600]))
    else:
        case.update(layers=_log(rng, 1, 6), blocks=_log(rng, 200, 3500), used=round(rng.uniform(0.1, 0.95), 3),
                    batch=rng.randint(1, 32), width=rng.randint(100, 600))
    return case


# ------------------------------------------------------------------ the stored form of a cache

def _cells(bits, is_key, device):
    """Where element (token, dim) of a block lies: the index of its byte or nibble, [16, 128]."""
    i = torch.arange(T, device=device)[:, None]
    d = torch.arange(D, device=device)[None, :]
    if is_key:
        g, hi, t, e = i & 7, i >> 3, d >> 5, d & 31
        lane = 4 * g + t
        if bits == 8:
            return (2 * hi + (e >> 4)) * 512 + lane * 16 + (e & 15)
        return 2 * (hi * 512 + lane * 16 + (e >> 3) * 4) + ((e & 7) >> 1) + 4 * (e & 1)
    m, r = d >> 4, d & 15
    g, hi, t, j = r & 7, r >> 3, (i & 7) >> 1, 2 * (i & 1) + (i >> 3)
    lane = 4 * g + t
    if bits == 8:
        return (m >> 1) * 512 + lane * 16 + (2 * (m & 1) + hi) * 4 + j
    return 2 * ((m >> 2) * 512 + lane * 16 + (m & 3) * 4) + 2 * hi + (j >> 1) + 4 * (j & 1)


def _quantize(x, bits, asym):
    """Stored code, scale and zero point of vectors along the last dimension, by the package's rule, in 64 bits."""
    x = x.double()
    if asym:
        low = x.amin(-1, keepdim=True)
        span = x.amax(-1, keepdim=True) - low
        s = torch.where(span == 0, torch.ones_like(span), span / (2 ** bits - 1)).float()
        u = torch.round((x - low) / s.double()).clamp(0, 2 ** bits - 1)
        return u.to(torch.uint8), s, low.float()
    top = 2 ** (bits - 1) - 1
    a = x.abs().amax(-1, keepdim=True)
    s = torch.where(a == 0, torch.ones_like(a), a / top).float()
    c = torch.round(x / s.double()).clamp(-top, top) + (top + 1)
    return c.to(torch.uint8), s, torch.zeros_like(s)


def _stand_for(u, s, z, bits, asym):
    """The values that stored codes stand for, in the type of s."""
    return u.to(s.dtype) * s + z if asym else (u.to(s.dtype) - 2 ** (bits - 1)) * s


def _random(shape, gen, spread=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * spread).bfloat16()


def _cache(case, blocks, gen, filled=True):
    """A cache of `blocks` blocks in its stored form: random keys with a few strong channels and random values, or zeros."""
    H, asym = case["kv_heads"], case["asym"]
    state = dict(blocks=blocks, factor=None)
    if case["factor"]:
        state["factor"] = (torch.rand(H, D, generator=gen, device="cuda") + 0.5).contiguous()
    meta = torch.zeros(H, blocks, 4 if asym else 2, T, device="cuda")
    for name, is_key, bits in (("k", True, case["k_bits"]), ("v", False, case["v_bits"])):
        pool = torch.zeros(H, blocks, T * D * bits // 8, dtype=torch.uint8, device="cuda")
        at, first = _cells(bits, is_key, "cuda").reshape(-1), 0 if is_key else meta.shape[2] // 2
        for h in range(H if filled else 0):
            x = torch.randn(blocks, T, D, generator=gen, device="cuda")
            if is_key:
                x[..., 5::37] *= 3.0
                if state["factor"] is not None:
                    x /= state["factor"][h]
            u, s, z = _quantize(x.bfloat16(), bits, asym)
            codes = torch.empty(blocks, T * D, dtype=torch.uint8, device="cuda")
            codes[:, at] = u.reshape(blocks, -1)
            pool[h] = codes if bits == 8 else codes[:, 0::2] | (codes[:, 1::2] << 4)
            meta[h, :, first] = s[..., 0]
            if asym:
                meta[h, :, first + 1] = z[..., 0]
        state[name] = pool.view(-1)
    state["meta"] = meta
    return state


def _block_bytes(case):
    """Bytes of one page of one head: codes of keys and of values, scales and zero points."""
    return T * D * case["k_bits"] // 8, T * D * case["v_bits"] // 8, T * 4 * (4 if case["asym"] else 2)


def _pools(case, blocks, gen):
    """All layers' pools with pages of any content: [layers, heads, blocks, bytes] of keys, values and scales."""
    k, v, m = _block_bytes(case)
    shape = case["layers"], case["kv_heads"], blocks
    codes = [torch.randint(0, 256, shape + (size,), dtype=torch.uint8, generator=gen, device="cuda") for size in (k, v)]
    return dict(k=codes[0], v=codes[1], meta=torch.rand(shape + (m // 4,), generator=gen, device="cuda"))


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 29)
    return {"norm": _prepare_norm, "decode": _prepare_decode, "prefill": _prepare_prefill, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, gen)


def _prepare_norm(case, gen):
    n, Hq, H, R = case["n"], case["q_heads"], case["kv_heads"], case["rotary"]
    # n rows of up to 8 sequences with consecutive positions each (one row each up to 64 rows)
    seqs = n if n <= 64 else 8
    lengths = torch.full((seqs,), n // seqs, device="cuda")
    lengths[: n % seqs] += 1
    seq = torch.repeat_interleave(torch.arange(seqs, device="cuda"), lengths)
    row = torch.arange(n, device="cuda") - torch.repeat_interleave(lengths.cumsum(0) - lengths, lengths)
    start = torch.randint(0, case["max_pos"] - int(lengths.max()) + 1, (seqs,), generator=gen, device="cuda")
    counts = (lengths + T - 1) // T
    width, blocks = int(counts.max()), int(counts.sum())
    table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None] < counts[:, None]] = torch.randperm(
        blocks, generator=gen, device="cuda").int()
    slot = row.int()
    state = _cache(case, blocks, gen, filled=False)
    # one row of a fused projection (its heads' sizes differ), queries, keys and values beside each other
    size = torch.rand(Hq + 2 * H, 1, generator=gen, device="cuda") * 4 + 0.25
    qkv = (torch.randn(n, Hq + 2 * H, D, generator=gen, device="cuda") * size).bfloat16().view(n, -1)
    weights = [torch.rand((h, D) if case["per_head"] else (D,), generator=gen, device="cuda") + 0.5 for h in (Hq, H)]
    j = torch.arange(R // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2 * j / R)
    state.update(case=case, qkv=qkv, table_cs=torch.stack((angle.cos(), angle.sin()), -1).float().contiguous(),
                 seq=seq.int(), slot=slot, pos=(start[seq] + row).int(), table=table, q_weight=weights[0],
                 k_weight=weights[1], eps=1e-6, where=(table[seq, row // T] * T + slot % T).int().contiguous(),
                 q_out=torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda"),
                 k_read=torch.empty(n, H, D, device="cuda"), v_read=torch.empty(n, H, D, device="cuda"))
    return state


def _seen_table(lengths, low, sinks, gen):
    """Tables that hold only the blocks of the first `sinks` tokens and those from token low[b] on, and their number."""
    count = (lengths + T - 1) // T
    width = int(count.max())
    col = torch.arange(width, device="cuda")[None]
    held = (col < count[:, None]) & ((col * T < sinks) | ((col + 1) * T > low[:, None]))
    blocks = int(held.sum())
    table = torch.full(held.shape, -1, dtype=torch.int32, device="cuda")
    table[held] = torch.randperm(blocks, generator=gen, device="cuda").int()
    return table, blocks


def _prepare_decode(case, gen):
    B, Hq = case["batch"], case["q_heads"]
    lengths = torch.randint(case["low"], case["high"] + 1, (B,), generator=gen, device="cuda")
    lengths[0] = case["high"]
    # pages behind the window have been freed
    table, blocks = _seen_table(lengths, lengths - case["span"], case["sinks"], gen)
    state = _cache(case, blocks, gen)
    state.update(case=case, q=_random((B, Hq, D), gen, 1.5), lengths=lengths.int(), table=table,
                 out=torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(B, Hq, device="cuda"))
    return state


def _prompts(case):
    """Lengths of the chunk's rows by sequence."""
    return [case["n"] * (i + 1) // case["seqs"] - case["n"] * i // case["seqs"] for i in range(case["seqs"])]


def _prepare_prefill(case, gen):
    n, Hq, start = case["n"], case["q_heads"], case["start"]
    rows = torch.tensor(_prompts(case), device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(rows), device="cuda"), rows)
    pos = start + torch.arange(n, device="cuda") - torch.repeat_interleave(rows.cumsum(0) - rows, rows)
    # the chunk is in the cache already; pages that its first row does not see have been freed
    first = torch.full((len(rows),), start + 1 - case["span"], device="cuda")
    table, blocks = _seen_table(start + rows, first, case["sinks"], gen)
    state = _cache(case, blocks, gen)
    state.update(case=case, q=_random((n, Hq, D), gen, 1.5), seq=seq.int(), pos=pos.int(), table=table,
                 out=torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(n, Hq, device="cuda"))
    return state


def _prepare_fork(case, gen):
    groups, beams, width, W = case["groups"], case["beams"], case["width"], case["window"]
    B = groups * beams
    lengths = torch.randint(case["low"], case["high"] + 1, (groups,), generator=gen, device="cuda")
    lengths[0] = case["high"]
    # beams of a request share the pages of its first half and hold the others themselves; answers to one prompt
    # are about to be forked from row 0, the only row in use
    table = torch.full((B, width), -1, dtype=torch.int32)
    lens, refs, at = [0] * B, [], 0
    for g, length in enumerate(lengths.tolist()):
        count = (max(length - W, 0) + T - 1) // T
        shared = count if case.get("fan") else count // 2
        for i in range(1 if case.get("fan") else beams):
            r = g * beams + i
            lens[r] = length
            if i == 0:
                first, at = at, at + shared
            table[r, :shared] = torch.arange(first, first + shared)
            table[r, shared:count] = torch.arange(at, at + count - shared)
            at += count - shared
        refs += [1 if case.get("fan") else beams] * shared + [1] * (at - len(refs) - shared)
    # room for the longest lengths, and a few pages
    most = (max(case["high"] - W, 0) + T - 1) // T
    blocks = (most if case.get("fan") else groups * (most // 2 + beams * (most - most // 2))) + 3 * B + 7
    ids = torch.randperm(blocks, generator=gen, device="cuda")
    table = table.cuda()
    table = torch.where(table >= 0, ids[table.clamp(min=0).long()].int(), -1).contiguous()
    counts = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    counts[ids[:at]] = torch.tensor(refs, dtype=torch.int32, device="cuda")
    if case.get("fan"):
        parent = torch.zeros(B, dtype=torch.long, device="cuda")
    else:
        parent = torch.randint(0, beams, (B,), generator=gen, device="cuda") + torch.arange(B, device="cuda") // beams * beams
    state = dict(case=case, pools=_pools(case, blocks, gen), blocks=blocks, refs=counts, table=table,
                 lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), parent=parent.int(),
                 refs_out=torch.zeros_like(counts), table_out=torch.zeros_like(table),
                 lens_out=torch.zeros(B, dtype=torch.int32, device="cuda"),
                 copies=torch.zeros(B, 2, dtype=torch.int32, device="cuda"),
                 num_copies=torch.zeros(1, dtype=torch.int32, device="cuda"))
    for name in ("k_window", "v_window") if W else ():
        state["pools"][name] = _random((case["layers"], B, case["kv_heads"] * W * D), gen)
    return state


def _prepare_compact(case, gen):
    blocks, B, width = case["blocks"], case["batch"], case["width"]
    used = max(1, int(blocks * case["used"]))
    ids = torch.randperm(blocks, generator=gen, device="cuda")[:used].int()
    # each row a stretch of the pages in use, some of them held by two rows; every page by one row at least
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    each = min(width, -(-used // B))
    at = (torch.arange(B, device="cuda")[:, None] * each + torch.arange(each, device="cuda")[None]) % used
    table[:, :each] = ids[at]
    held = table[table >= 0].long()
    refs = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    refs[ids.long()] = 1  # pages that no row holds are kept by their user
    refs.scatter_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    return dict(case=case, pools=_pools(case, blocks, gen), blocks=blocks, refs=refs, table=table,
                refs_out=torch.zeros_like(refs), table_out=torch.zeros_like(table),
                moves=torch.zeros(blocks // 2, 2, dtype=torch.int32, device="cuda"),
                counts=torch.zeros(2, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "decode": _plain_decode, "prefill": _plain_prefill, "fork": _plain_fork,
            "compact": _plain_compact}[state["case"]["op"]](state)


def _desc(lib, c, blocks, k, v, meta, factor=None, **more):
    return lib.CacheDesc(num_kv_heads=c["kv_heads"], head_dim=D, block_size=T, num_blocks=blocks, k_bits=c["k_bits"],
                         v_bits=c["v_bits"], k_codes=k.data_ptr(), v_codes=v.data_ptr(), meta=meta.data_ptr(),
                         asym=int(c["asym"]), k_channel_factor=None if factor is None else factor.data_ptr(), **more)


def _handle(state):
    """The descriptors and the workspace that a program keeps with its cache."""
    from quantized_kv_cache_07_gb300 import _lib as lib
    c = state["case"]
    if "desc" in state:
        return lib, state["desc"], c
    if "pools" in state:
        layers = [{name: pool[i] for name, pool in state["pools"].items()} for i in range(c["layers"])]
        state["desc"] = lib.CacheList([
            _desc(lib, c, state["blocks"], y["k"], y["v"], y["meta"],
                  **(dict(window=c["window"], window_batch=len(state["table"]), k_window=y["k_window"].data_ptr(),
                          v_window=y["v_window"].data_ptr()) if c.get("window") else {})) for y in layers])
        size = lib.kvq_pages_workspace_size(state["blocks"])
        state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        return lib, state["desc"], c
    state["desc"] = _desc(lib, c, state["blocks"], state["k"], state["v"], state["meta"], state["factor"])
    if c["op"] == "norm":
        state["rope"] = lib.RopeDesc(rotary_dim=c["rotary"], interleaved=int(c["interleaved"]), max_pos=c["max_pos"],
                                     table=state["table_cs"].data_ptr())
        state["norm"] = lib.NormDesc(eps=state["eps"], per_head=int(c["per_head"]),
                                     q_weight=state["q_weight"].data_ptr(), k_weight=state["k_weight"].data_ptr())
    else:
        size = (lib.kvq_prefill_workspace_size(state["desc"], c["n"], c["q_heads"]) if c["op"] == "prefill" else
                lib.kvq_decode_workspace_size(state["desc"], c["batch"], c["q_heads"]))
        state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        lib.kvq_workspace_init(state["workspace"], size)
    return lib, state["desc"], c


def _own(state):
    lib, desc, c = _handle(state)
    if c["op"] == "norm":
        Hq, H, qkv = c["q_heads"], c["kv_heads"], state["qkv"]
        q, k, v = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + H) * D], qkv[:, (Hq + H) * D:]
        lib.kvq_norm_rope_append(desc, state["rope"], state["norm"], q, Hq, state["q_out"], k, v, state["pos"],
                                 state["seq"], state["slot"], lib.APPEND_QUANT, state["table"], *state["table"].shape)
        lib.kvq_dequant(desc, state["where"], state["k_read"], state["v_read"])
        return state["q_out"], state["k_read"], state["v_read"]
    table = state["table"]
    if c["op"] == "decode":
        lib.kvq_decode_sinks(desc, state["q"], c["batch"], c["q_heads"], state["lengths"], table, table.shape[1],
                             c["sinks"], c["span"], state["out"], lse=state["lse"], workspace=state["workspace"],
                             workspace_bytes=state["workspace"].numel())
        return state["out"], state["lse"]
    if c["op"] == "prefill":
        lib.kvq_prefill_sinks(desc, state["q"], c["q_heads"], state["seq"], state["pos"], table, *table.shape,
                              c["sinks"], c["span"], state["out"], lse=state["lse"], workspace=state["workspace"],
                              workspace_bytes=state["workspace"].numel())
        return state["out"], state["lse"]
    if c["op"] == "fork":
        lib.kvq_pages_update(state["refs"], table, state["lens"], state["refs_out"], state["table_out"],
                             state["lens_out"], state["copies"], state["num_copies"], parent=state["parent"], room=T,
                             window=c["window"], sinks=c["sinks"], span=c["span"], workspace=state["workspace"])
        lib.kvq_copy_blocks(desc, state["copies"], state["num_copies"])
        if c["window"]:
            lib.kvq_fork_windows(desc, state["parent"], len(table))
        return _fork_result(state)
    lib.kvq_pages_compact(state["refs"], table, state["refs_out"], state["table_out"], state["moves"], state["counts"],
                          workspace=state["workspace"])
    lib.kvq_copy_blocks(desc, state["moves"], state["counts"])
    return _compact_result(state)


def _fork_result(state):
    return [state[x] for x in ("refs_out", "table_out", "lens_out", "copies", "num_copies")] + list(state["pools"].values())


def _compact_result(state):
    return [state[x] for x in ("refs_out", "table_out", "moves", "counts")] + list(state["pools"].values())


# ------------------------------------------------------------------ plain forms

def _values(state, is_key, ids):
    """What the blocks `ids` stand for, [kv_heads, *ids, 16, 128] float32."""
    c = state["case"]
    bits = c["k_bits"] if is_key else c["v_bits"]
    raw = state["k" if is_key else "v"].view(c["kv_heads"], state["blocks"], -1)[:, ids]
    if bits == 4:
        raw = torch.stack((raw & 15, raw >> 4), -1).flatten(-2)
    u = raw[..., _cells(bits, is_key, "cuda")]
    rec = state["meta"][:, ids]
    at = 0 if is_key else rec.shape[-2] // 2
    x = _stand_for(u, rec[..., at, :, None], rec[..., at + 1, :, None] if c["asym"] else 0.0, bits, c["asym"])
    if is_key and state["factor"] is not None:
        x = x * state["factor"].view(-1, *[1] * (x.dim() - 2), D)
    return x


def _normed(x, weight, eps):
    """Heads x [n, heads, 128] over the root of their mean square, times the weight; in 64 bits: 4-bit codes follow."""
    x = x.double()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight


def _plain_norm(state):
    c = state["case"]
    n, Hq, H = c["n"], c["q_heads"], c["kv_heads"]
    x = state["qkv"].view(n, Hq + 2 * H, D)
    y = torch.cat((_normed(x[:, :Hq], state["q_weight"], state["eps"]),
                   _normed(x[:, Hq:Hq + H], state["k_weight"], state["eps"])), 1)
    cs = state["table_cs"][state["pos"].long()]
    pairs = cs.shape[1]
    a = y[..., :2 * pairs]
    x0, x1 = (a[..., 0::2], a[..., 1::2]) if c["interleaved"] else (a[..., :pairs], a[..., pairs:])
    cos, sin = cs[:, None, :, 0].double(), cs[:, None, :, 1].double()
    y0, y1 = x0 * cos - x1 * sin, x0 * sin + x1 * cos
    a = torch.stack((y0, y1), -1).flatten(-2) if c["interleaved"] else torch.cat((y0, y1), -1)
    turned = torch.cat((a, y[..., 2 * pairs:]), -1).float().bfloat16()
    key = turned[:, Hq:].float()
    if state["factor"] is not None:
        key = key / state["factor"]
    read = []
    for value, bits in ((key, c["k_bits"]), (x[:, Hq + H:], c["v_bits"])):
        u, s, z = _quantize(value, bits, c["asym"])
        read.append(_stand_for(u, s.double(), z.double(), bits, c["asym"]).float())
    return turned[:, :Hq].contiguous(), read[0], read[1]


def _attend(q, k, v, seen):
    """Softmax attention of q [.., rows, 128] over k, v [.., tokens, 128] where `seen`: output and log-sum-exp."""
    score = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / total, (top + torch.log(total))[..., 0]


def _plain_decode(state):
    c, q, table = state["case"], state["q"], state["table"]
    B, Hq, H = c["batch"], c["q_heads"], c["kv_heads"]
    # the columns that a row of its window can need: the blocks of the first tokens, then those from the window's start
    front, width = -(-c["sinks"] // T), table.shape[1]
    length = state["lengths"].long()[:, None]
    first = (length - c["span"]).clamp(min=0) // T
    col = torch.arange(front + (c["span"] + T - 2) // T + 1, device="cuda")[None]
    col = torch.where(col < front, col.expand(B, -1), torch.maximum(first, torch.full_like(first, front)) + col - front)
    ids = table.long().gather(1, col.clamp(max=width - 1)).clamp(min=0)
    token = (col[..., None] * T + torch.arange(T, device="cuda")).flatten(1)
    seen = (token < length) & ((token < c["sinks"]) | (token >= length - c["span"]))
    k, v = (_values(state, is_key, ids).flatten(2, 3).transpose(0, 1) for is_key in (True, False))
    out, lse = _attend(q.float().view(B, H, -1, D), k, v, seen[:, None, None])
    return out.reshape(B, Hq, D).bfloat16(), lse.reshape(B, Hq)


def _plain_prefill(state):
    c, q = state["case"], state["q"]
    Hq, H = c["q_heads"], c["kv_heads"]
    out, lse, r0 = [], [], 0
    for b, rows in enumerate(_prompts(c)):
        width = (c["start"] + rows + T - 1) // T
        ids = state["table"][b, :width].long().clamp(min=0)
        k, v = (_values(state, is_key, ids).flatten(1, 2) for is_key in (True, False))
        pos = state["pos"][r0:r0 + rows].long()[:, None]
        token = torch.arange(width * T, device="cuda")[None]
        seen = (token <= pos) & ((token < c["sinks"]) | (token > pos - c["span"]))
        x = q[r0:r0 + rows].float().view(rows, H, -1, D).permute(1, 2, 0, 3)
        o, s = _attend(x, k[:, None], v[:, None], seen)
        out.append(o.permute(2, 0, 1, 3).reshape(rows, Hq, D))
        lse.append(s.permute(2, 0, 1).reshape(rows, Hq))
        r0 += rows
    return torch.cat(out).bfloat16(), torch.cat(lse)


def _copy_pages(state, source, target):
    for name in ("k", "v", "meta"):
        for layer in state["pools"][name]:
            layer[:, target] = layer[:, source]


def _plain_fork(state):
    c, table, lens = state["case"], state["table"].long(), state["lens"].long()
    B, width = table.shape
    W, blocks, refs = c["window"], state["blocks"], state["refs"].long()
    one = torch.ones(B, width, dtype=torch.long, device="cuda")
    row, col = torch.arange(B, device="cuda")[:, None], torch.arange(width, device="cuda")[None]
    parent = state["parent"].long()[:, None]
    length = torch.where(parent >= 0, lens[parent.clamp(min=0)], 0)
    stored = (length - W).clamp(min=0)
    count = (stored + T - 1) // T
    need = torch.where(parent >= 0, ((length + T - W).clamp(min=0) + T - 1) // T, 0)
    keep = (col < count) | ((parent == row) & (col < need))
    if c["span"]:
        keep &= (col < -(-c["sinks"] // T)) | ((col + 1) * T > length - c["span"])
    page = torch.where(keep & (parent >= 0), table[parent[:, 0].clamp(min=0)], -1)

    def held(pages):
        n = torch.zeros(blocks + 1, dtype=torch.long, device="cuda")
        return n.scatter_add_(0, torch.where(pages >= 0, pages, blocks).flatten(), one.flatten())[:blocks]

    refs = refs - held(table) + held(page)
    # a page kept for coming tokens that others hold is not one to write to
    spare = (col >= count) & (page >= 0) & (refs[page.clamp(min=0)] > 1)
    refs = refs - held(torch.where(spare, page, -1))
    page = torch.where(spare, -1, page)
    # the last page, if there is room left in it: the lowest of the rows that write to it keeps it, if no one else holds it
    last = page.gather(1, (count - 1).clamp(min=0))
    last = torch.where((stored % T != 0) & (last >= 0), last, -1)
    at = torch.where(last >= 0, last, blocks)[:, 0]
    writers = torch.zeros(blocks + 1, dtype=torch.long, device="cuda").scatter_add_(0, at, one[:, 0])
    first = torch.full((blocks + 1,), B, device="cuda").scatter_reduce_(0, at, row[:, 0], "amin")
    of = last.clamp(min=0)
    copy = (last >= 0) & ~((writers[of] == refs[of]) & (first[of] == row))
    wanted = (copy & (col == count - 1)) | ((col >= count) & (col < need) & (page < 0))
    # the lowest free pages, in the order of rows and columns
    free = torch.sort((refs != 0).int(), stable=True).indices
    rank = wanted.flatten().cumsum(0).view(B, width) - 1
    page = torch.where(wanted, free[rank.clamp(0, blocks - 1)], page)
    refs = refs - held(torch.where(copy, last, -1).expand(B, width) * (col == 0) - (col != 0).long()) + held(
        torch.where(wanted, page, -1))
    target = page.gather(1, (count - 1).clamp(min=0))
    state["refs_out"].copy_(refs)
    state["table_out"].copy_(page)
    state["lens_out"].copy_(length[:, 0])
    state["num_copies"].copy_(copy.sum())
    pairs = torch.cat((torch.cat((last, target), 1), torch.zeros(1, 2, dtype=torch.long, device="cuda")))
    order = torch.sort((~copy[:, 0]).int(), stable=True).indices
    state["copies"].copy_(torch.where(copy[order], pairs[order], state["copies"].long()))
    # rows without a copy repeat the first one (or page 0 onto itself)
    some = copy.any()
    lead = torch.where(some, pairs[order[0]], 0)
    _copy_pages(state, *torch.where(copy, pairs[:B], lead).T)
    for name in ("k_window", "v_window") if W else ():
        for layer in state["pools"][name]:
            layer.copy_(layer[torch.where(parent >= 0, parent, row)[:, 0]])
    return _fork_result(state)


def _plain_compact(state):
    refs, table, blocks = state["refs"].long(), state["table"].long(), state["blocks"]
    block = torch.arange(blocks, device="cuda")
    live = (refs > 0).sum()
    hole, tail = (refs == 0) & (block < live), (refs > 0) & (block >= live)
    moves = hole.sum()
    # the i-th hole takes the i-th page from behind
    holes = torch.sort((~hole).int(), stable=True).indices
    tails = torch.sort((~tail).int(), stable=True).indices
    moved = block < moves
    to = torch.where(tail, holes[(tail.cumsum(0) - 1).clamp(min=0)], block)
    state["table_out"].copy_(torch.where(table >= 0, to[table.clamp(min=0)], table))
    state["refs_out"].copy_(torch.where(hole, refs[tails[(hole.cumsum(0) - 1).clamp(min=0)]], torch.where(tail, 0, refs)))
    state["counts"].copy_(torch.stack((moves, live)))
    pairs = torch.stack((tails, holes), 1)[: len(state["moves"])]
    state["moves"].copy_(torch.where(moved[: len(pairs), None], pairs, state["moves"].long()))
    # places behind the last move: each page onto itself
    where = torch.where(hole, tails[(hole.cumsum(0) - 1).clamp(min=0)], block)
    _copy_pages(state, where, block)
    return _compact_result(state)


# ------------------------------------------------------------------ cost

def work(case):
    H, Hq, B = case["kv_heads"], case["q_heads"], case.get("batch", 0)
    per = 8 if case["asym"] else 4
    token = D * (case["k_bits"] + case["v_bits"]) / 8 + 2 * per
    if case["op"] == "norm":
        n = case["n"]
        # queries, keys and values in, queries and stored tokens out, the read-back of the stored values
        moved = n * ((2 * Hq + 2 * H) * D * 2 + 2 * H * token + 2 * H * D * 4 + 4 * case["rotary"] + 16)
        return {"bytes": moved, "flops": n * ((Hq + H) * (3 * case["rotary"] + 4 * D) + 2 * H * 3 * D)}
    if case["op"] == "decode":
        reach = case["sinks"] + case["span"]
        seen = sum(min((case["low"] * (2 * B - 1 - i) + case["high"] * (1 + i)) / (2 * B), reach) for i in range(B))
        return {"bytes": seen * H * token + 2 * B * Hq * D * 2 + 4 * B * Hq, "flops": 4 * D * Hq * seen}
    if case["op"] == "prefill":
        seen = held = 0
        for rows in _prompts(case):
            seen += sum(min(case["start"] + i + 1, case["sinks"] + case["span"]) for i in range(rows))
            held += min(case["start"] + rows, case["sinks"] + case["span"] + rows)
        return {"bytes": held * H * token + case["n"] * Hq * (4 * D + 4), "flops": 4 * D * Hq * seen}
    page = case["layers"] * H * sum(_block_bytes(case))
    if case["op"] == "fork":
        rows, beams = case["groups"] * case["beams"], case["beams"]
        # of `beams` choices so many parents are chosen on average; their first child keeps the last page
        copies = rows - (1 if case.get("fan") else case["groups"] * beams * (1 - (1 - 1 / beams) ** beams))
        rings = copies * case["layers"] * 2 * H * case["window"] * D * 2
        pages = (0.5 if not case.get("fan") else 1) * (case["low"] + case["high"]) / 2 / T * (
            1 if case.get("fan") else case["groups"] * (1 + beams))
        return {"bytes": 2 * copies * page * 15 / 16 + 2 * rings + 8 * rows * case["width"] + 8 * pages,
                "flops": rows * case["width"]}
    # as many pages move as there are free ones in the front part
    moved = case["blocks"] * case["used"] * (1 - case["used"])
    return {"bytes": 2 * moved * page + 8 * case["blocks"] + 8 * B * case["width"] + 8 * moved, "flops": case["blocks"]}


# ------------------------------------------------------------------ in 64 bits, one sequence and head at a time

def _whose(bits, is_key):
    """Token and dim of each code place of a block, found from the place: two lists of 2048."""
    token, dim = [], []
    for place in range(T * D):
        byte, half = (place, 0) if bits == 8 else divmod(place, 2)
        chunk, rest = divmod(byte, 512)
        lane, b = divmod(rest, 16)
        g, t = divmod(lane, 4)
        word, nib = b // 4, 2 * (b % 4) + half
        if is_key and bits == 8:
            token.append(g + 8 * (chunk // 2))
            dim.append(32 * t + 16 * (chunk % 2) + b)
        elif is_key:
            token.append(g + 8 * chunk)
            dim.append(32 * t + 8 * word + 2 * (nib % 4) + nib // 4)
        else:
            j = b % 4 if bits == 8 else 2 * (nib % 2) + nib // 4
            token.append(2 * t + j // 2 + 8 * (j % 2))
            dim.append((32 * chunk + 16 * (word // 2) + 8 * (word % 2) if bits == 8 else
                        64 * chunk + 16 * word + 8 * ((nib % 4) // 2)) + g)
    return torch.tensor(token, device="cuda"), torch.tensor(dim, device="cuda")


def _exact_rows(state, b, h, is_key, places, tokens):
    """Keys or values of the given tokens of sequence b, head h, in 64 bits, [tokens, 128]."""
    c = state["case"]
    bits = c["k_bits"] if is_key else c["v_bits"]
    blocks, back = torch.unique(tokens // T, return_inverse=True)
    ids = state["table"][b, blocks].long()
    raw = state["k" if is_key else "v"].view(c["kv_heads"], state["blocks"], -1)[h, ids].long()
    if bits == 4:
        raw = torch.stack((raw % 16, raw // 16), 2).reshape(len(ids), -1)
    x = torch.zeros(len(ids), T, D, dtype=torch.float64, device="cuda")
    x[:, places[0], places[1]] = raw.double()
    rec = state["meta"][h, ids].double()
    if c["asym"]:
        x = x * rec[:, 0 if is_key else 2][..., None] + rec[:, 1 if is_key else 3][..., None]
    else:
        x = (x - (128 if bits == 8 else 8)) * rec[:, 0 if is_key else 1][..., None]
    if is_key and state["factor"] is not None:
        x = x * state["factor"][h].double()
    return x[back, tokens % T]


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # they choose and move: nothing in them is computed
    state = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(state)
    Hq, H, sinks, span = case["q_heads"], case["kv_heads"], case["sinks"], case["span"]
    G = Hq // H
    places = _whose(case["k_bits"], True), _whose(case["v_bits"], False)
    q = state["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    if case["op"] == "decode":
        parts = [(b, slice(b, b + 1), torch.tensor([length - 1])) for b, length in enumerate(state["lengths"].tolist())]
    else:
        ends = torch.tensor(_prompts(case)).cumsum(0).tolist()
        parts = [(b, slice(begin, end), torch.arange(case["start"], case["start"] + end - begin))
                 for b, (begin, end) in enumerate(zip([0] + ends, ends))]
    for b, rows, pos in parts:
        token = torch.arange(int(pos[-1]) + 1)
        token = token[(token < sinks) | (token > int(pos[0]) - span)]
        see = (token[None] <= pos[:, None]) & ((token[None] < sinks) | (token[None] > pos[:, None] - span))
        token, hidden = token.cuda(), ~see.cuda()
        for h in range(H):
            k, v = (_exact_rows(state, b, h, is_key, places[not is_key], token) for is_key in (True, False))
            for g in range(h * G, (h + 1) * G):
                s = (q[rows, g] @ k.T * D ** -0.5).masked_fill_(hidden, -math.inf)
                out[rows, g] = torch.softmax(s, -1) @ v
                lse[rows, g] = torch.logsumexp(s, -1)
    return out, lse


def _exact_norm(state):
    """Queries in 64 bits; the stored values from the turned keys, which are bf16 by definition."""
    c = state["case"]
    Hq, H, R = c["q_heads"], c["kv_heads"], c["rotary"]
    x = state["qkv"].double().view(c["n"], -1, D)
    weight = torch.cat([w.double().expand(h, D) for w, h in ((state["q_weight"], Hq), (state["k_weight"], H))])
    y = x[:, :Hq + H] / (x[:, :Hq + H].square().sum(-1, keepdim=True) / D + state["eps"]).sqrt() * weight
    lead = torch.arange(0, R, 2, device="cuda") if c["interleaved"] else torch.arange(R // 2, device="cuda")
    mate = lead + (1 if c["interleaved"] else R // 2)
    angle = torch.view_as_complex(state["table_cs"].double().contiguous())[state["pos"].long()][:, None]
    turned = torch.complex(y[..., lead], y[..., mate]) * angle
    y[..., lead], y[..., mate] = turned.real, turned.imag
    k = y[:, Hq:].float().bfloat16().float()
    if state["factor"] is not None:
        k = k / state["factor"]
    stored = []
    for v, bits in ((k.double(), c["k_bits"]), (x[:, Hq + H:], c["v_bits"])):
        if c["asym"]:
            low, high = v.min(-1).values, v.max(-1).values
            step = ((high - low) / (2 ** bits - 1)).float().double()
            step[high == low] = 1.0
            stored.append(((v - low[..., None]) / step[..., None]).round().clamp(0, 2 ** bits - 1) * step[..., None]
                          + low[..., None])
        else:
            step = (v.abs().max(-1).values / (2 ** (bits - 1) - 1)).float().double()
            step[step == 0] = 1.0
            stored.append((v / step[..., None]).round() * step[..., None])
    return y[:, :Hq], stored[0], stored[1]
