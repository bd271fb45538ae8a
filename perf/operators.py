"""Cases of the cache operators beside decode: rotary write, shared-prefix decode, attention mass and eviction.

A case names its operator in "op":
  rope   rotate queries and keys by their positions and write keys and values into the cache (kvq_rope_append)
  shared one decode step of a batch whose sequences share a prefix (kvq_decode_shared)
  mass   add every cached token's attention weight of this step to its running sum (kvq_attn_mass)
  evict  keep each sequence's heaviest tokens, in place (kvq_evict)

Head dimension 128 and 16-token blocks, as everywhere in this package.  The cache is made in its stored byte order
(include/kvq.h) from random keys and values, so both forms read the same bytes.
"""
import math

import torch

own = False

D, T = 128, 16


# ------------------------------------------------------------------ the cases

def listed():
    rope = dict(op="rope", q_heads=32, kv_heads=8, k_bits=8, v_bits=8, asym=False, factor=False)
    shared = dict(op="shared", q_heads=32, kv_heads=8, k_bits=8, v_bits=8, asym=False, factor=False)
    mass = dict(op="mass", q_heads=32, kv_heads=8, k_bits=8, v_bits=8, asym=False, factor=False)
    evict = dict(op="evict", q_heads=32, kv_heads=8, k_bits=8, v_bits=8, asym=False, factor=False)
    return [
        # the new token of each of 64 running sequences, far into their contexts
        dict(rope, name="rope step of 64", n=64, max_pos=32768, rotary=128, interleaved=False),
        # a prompt of odd length into a 4-bit cache with a key factor, half of each head rotated in neighbouring pairs
        dict(rope, name="rope prompt of 1337, int4", n=1337, max_pos=8192, rotary=64, interleaved=True,
             k_bits=4, v_bits=4, factor=True),
        # a prefill chunk of several long prompts
        dict(rope, name="rope chunk of 8192", n=8192, max_pos=131072, rotary=128, interleaved=False),
        # four answers to one short prompt: latency
        dict(shared, name="shared 4 of 2048", batch=4, groups=1, prefix=2048, suffix=200),
        # a few dozen requests behind one system prompt, 4-bit cache with a key factor, odd lengths
        dict(shared, name="shared 33 of 8176, int4", batch=33, groups=1, prefix=8176, suffix=700, k_bits=4, v_bits=4,
             factor=True),
        # three documents asked about by a batch, eight query heads to a KV head, 4-bit keys with 8-bit values
        dict(shared, name="shared 3 documents, k4v8", batch=24, groups=3, prefix=16384, suffix=500, q_heads=64,
             k_bits=4, v_bits=8),
        # the largest: 64 requests on one long document
        dict(shared, name="shared 64 of 32768", batch=64, groups=1, prefix=32768, suffix=1000),
        # one short sequence: latency
        dict(mass, name="mass 1 of 256", batch=1, low=256, high=256, q_heads=4, kv_heads=4),
        # a batch of ragged contexts, 4-bit cache
        dict(mass, name="mass 32 of 1k-8k, int4", batch=32, low=1024, high=8192, k_bits=4, v_bits=4),
        # few very long contexts, eight query heads to a KV head
        dict(mass, name="mass 4 of 131072", batch=4, low=131072, high=131072, q_heads=64, k_bits=4, v_bits=8),
        # a batch that is cut back to half its tokens
        dict(evict, name="evict 8 of 4096", batch=8, low=4096, high=4096, share=0.5, first=4, recent=128),
        # few long contexts of odd lengths, cut back to a quarter
        dict(evict, name="evict 4 of 32768, asym", batch=4, low=30000, high=32768, share=0.25, first=16, recent=500,
             asym=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope", "shared", "mass", "evict"])
    q_heads, kv_heads = rng.choice([(32, 8), (64, 8), (16, 8), (8, 8), (8, 2), (4, 4), (24, 8), (10, 2)])
    k_bits, v_bits = rng.choice([(8, 8), (4, 4), (4, 8), (8, 4)])
    case = dict(op=op, q_heads=q_heads, kv_heads=kv_heads, k_bits=k_bits, v_bits=v_bits,
                asym=rng.random() < 0.3, factor=rng.random() < 0.3)
    if op == "rope":
        case.update(n=_log(rng, 1, 4096), max_pos=_log(rng, 5000, 131072), rotary=rng.choice([32, 64, 96, 128]),
                    interleaved=rng.random() < 0.5)
    elif op == "shared":
        groups = rng.choice([1, 1, 1, 2, 3])
        case.update(batch=_log(rng, 2, 48) + groups - 1, groups=groups, prefix=16 * _log(rng, 16, 1024),
                    suffix=_log(rng, 1, 1000))
    elif op == "mass":
        high = _log(rng, 100, 32768)
        case.update(batch=_log(rng, 1, 12), low=rng.randint(1, high), high=high)
    else:
        high = _log(rng, 300, 16384)
        case.update(batch=_log(rng, 1, 8), low=rng.randint(100, high), high=high,
                    share=round(rng.uniform(0.1, 0.9), 3), first=rng.randint(0, 20), recent=rng.randint(0, 100))
    return case


# ------------------------------------------------------------------ the stored form of a cache

def _cells(bits, is_key, device):
    """Where element (token, dim) of a block lies: the index of its byte, nibble or 16-bit word, [16, 128]."""
    i = torch.arange(T, device=device)[:, None]
    d = torch.arange(D, device=device)[None, :]
    if is_key:
        g, hi, t, e = i & 7, i >> 3, d >> 5, d & 31
        lane = 4 * g + t
        if bits == 8:
            return (2 * hi + (e >> 4)) * 512 + lane * 16 + (e & 15)
        nib = ((e & 7) >> 1) + 4 * (e & 1)
        return 2 * (hi * 512 + lane * 16 + (e >> 3) * 4) + nib
    m, r = d >> 4, d & 15
    g, hi, t, j = r & 7, r >> 3, (i & 7) >> 1, 2 * (i & 1) + (i >> 3)
    lane = 4 * g + t
    if bits == 8:
        return (m >> 1) * 512 + lane * 16 + (2 * (m & 1) + hi) * 4 + j
    nib = 2 * hi + (j >> 1) + 4 * (j & 1)
    return 2 * ((m >> 2) * 512 + lane * 16 + (m & 3) * 4) + nib


def _unpack(pool, bits, heads):
    """The pool's codes, one per place, [heads, blocks, 2048]."""
    if bits == 8:
        return pool.view(heads, -1, T * D)
    return torch.stack((pool & 15, pool >> 4), -1).view(heads, -1, T * D)


def _pack(codes, bits):
    if bits == 8:
        return codes.reshape(-1)
    codes = codes.reshape(-1, 2)
    return codes[:, 0] | (codes[:, 1] << 4)


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


def _fill(x, bits, asym, is_key):
    """The pool and the scales and zero points [heads, blocks, 16] of vectors x [heads, blocks, 16, 128]."""
    heads, blocks = x.shape[:2]
    codes = torch.empty(heads, blocks, T * D, dtype=torch.uint8, device=x.device)
    at = _cells(bits, is_key, x.device)
    s = torch.empty(heads, blocks, T, device=x.device)
    z = torch.empty_like(s)
    for h in range(heads):
        u, sh, zh = _quantize(x[h], bits, asym)
        codes[h][:, at.reshape(-1)] = u.reshape(blocks, -1)
        s[h], z[h] = sh[..., 0], zh[..., 0]
    return _pack(codes, bits).contiguous(), s, z


def _random(shape, gen, spread=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * spread).bfloat16()


def _cache(case, blocks, gen, keys=True, values=True):
    """A cache of `blocks` full blocks in its stored form: random keys with a few strong channels, random values."""
    H, asym = case["kv_heads"], case["asym"]
    state = dict(blocks=blocks)
    state["factor"] = None
    if case["factor"]:
        state["factor"] = (torch.rand(H, D, generator=gen, device="cuda") + 0.5).contiguous()
    meta = torch.zeros(H, blocks, 4 if asym else 2, T, device="cuda")
    for name, is_key, bits, wanted in (("k", True, case["k_bits"], keys), ("v", False, case["v_bits"], values)):
        if not wanted:
            state[name] = torch.zeros(H * blocks * T * D * bits // 8, dtype=torch.uint8, device="cuda")
            continue
        x = torch.randn(H, blocks, T, D, generator=gen, device="cuda")
        if is_key:
            x[..., 5::37] *= 3.0
            if state["factor"] is not None:
                x /= state["factor"][:, None, None]
        state[name], s, z = _fill(x.bfloat16(), bits, asym, is_key)
        at = 0 if is_key else meta.shape[2] // 2
        meta[:, :, at] = s
        if asym:
            meta[:, :, at + 1] = z
        del x
    state["meta"] = meta
    return state




def _lengths(case, gen):
    n = torch.randint(case["low"], case["high"] + 1, (case["batch"],), generator=gen, device="cuda")
    n[0] = case["high"]
    return n.int()


def _plain_table(case, lengths, gen):
    """Table of sequences that share nothing: [batch, blocks of the longest], -1 where unused, in a pool with room for all."""
    counts = (lengths + T - 1) // T
    width = (case["high"] + T - 1) // T
    total = case["batch"] * width
    ids = torch.randperm(total, generator=gen, device="cuda").int()
    used = torch.arange(width, device="cuda")[None] < counts[:, None]
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device="cuda")
    table[used] = ids[: int(counts.sum())]
    return table.contiguous(), total


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 13)
    return {"rope": _prepare_rope, "shared": _prepare_shared, "mass": _prepare_mass, "evict": _prepare_evict}[
        case["op"]](case, gen)


def _prepare_rope(case, gen):
    n, Hq, H, R = case["n"], case["q_heads"], case["kv_heads"], case["rotary"]
    # n rows of up to 8 sequences with consecutive positions each, ending at the longest context (one row each up to 64 rows)
    seqs = n if n <= 64 else 8
    lengths = torch.full((seqs,), n // seqs, device="cuda")
    lengths[: n % seqs] += 1
    seq = torch.repeat_interleave(torch.arange(seqs, device="cuda"), lengths)
    row = torch.arange(n, device="cuda") - torch.repeat_interleave(lengths.cumsum(0) - lengths, lengths)
    start = torch.randint(0, case["max_pos"] - int(lengths.max()) + 1, (seqs,), generator=gen, device="cuda")
    pos = (start[seq] + row).int()
    # the cache slots of these rows: the first of their sequences (a cache that holds fewer tokens than positions)
    counts = (lengths + T - 1) // T
    width, blocks = int(counts.max()), int(counts.sum())
    table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None] < counts[:, None]] = torch.randperm(
        blocks, generator=gen, device="cuda").int()
    slot = row.int()
    phys = table[seq, (row // T)]
    state = _cache(case, blocks, gen, keys=False, values=False)
    # one row of a fused projection: queries, keys and values beside each other
    qkv = _random((n, (Hq + 2 * H) * D), gen)
    j = torch.arange(R // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2 * j / R)
    state.update(case=case, qkv=qkv, table_cs=torch.stack((angle.cos(), angle.sin()), -1).float().contiguous(),
                 seq=seq.int(), slot=slot, pos=pos, table=table, where=(phys * T + slot % T).int().contiguous(),
                 q_out=torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda"),
                 k_read=torch.empty(n, H, D, device="cuda"), v_read=torch.empty(n, H, D, device="cuda"))
    return state


def _prepare_shared(case, gen):
    B, groups, Hq = case["batch"], case["groups"], case["q_heads"]
    # groups of nearly equal size; their prefixes differ by some blocks
    start = [g * B // groups for g in range(groups + 1)]
    prefix = [case["prefix"] // T - 5 * g for g in range(groups)]
    group = torch.zeros(B, dtype=torch.long, device="cuda")
    for g in range(groups):
        group[start[g]:start[g + 1]] = g
    per_row = torch.tensor(prefix, device="cuda")[group]
    own_tokens = torch.randint(1, case["suffix"] + 1, (B,), generator=gen, device="cuda")
    own_blocks = (own_tokens + T - 1) // T
    total = sum(prefix) + int(own_blocks.sum())
    width = int((per_row + own_blocks).max())
    ids = torch.randperm(total, generator=gen, device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(width, device="cuda")[None]
    first = torch.tensor([sum(prefix[:g]) for g in range(groups)], device="cuda")
    in_prefix = col < per_row[:, None]
    table[in_prefix] = ids[(first[group][:, None] + col)[in_prefix]]
    table[(col >= per_row[:, None]) & (col < (per_row + own_blocks)[:, None])] = ids[sum(prefix):]
    state = _cache(case, total, gen)
    state.update(case=case, q=_random((B, Hq, D), gen, 1.5), lengths=(per_row * T + own_tokens).int(), table=table,
                 group_start=torch.tensor(start, dtype=torch.int32, device="cuda"),
                 prefix_blocks=torch.tensor(prefix, dtype=torch.int32, device="cuda"),
                 out=torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(B, Hq, device="cuda"))
    return state


def _prepare_mass(case, gen):
    B, Hq, H = case["batch"], case["q_heads"], case["kv_heads"]
    lengths = _lengths(case, gen)
    table, blocks = _plain_table(case, lengths, gen)
    state = _cache(case, blocks, gen, values=False)
    state.update(case=case, q=_random((B, Hq, D), gen, 1.5), lengths=lengths, table=table)
    score, used = _pool_scores(state)
    score = torch.where(used[None, :, None], score, -math.inf)
    # the log-sum-exp that the decode step before this call gave: [batch, q_heads]
    state["lse"] = torch.logsumexp(score.double(), -1).float().permute(1, 0, 2).reshape(B, Hq).contiguous()
    state["mass"] = torch.rand(B, H, table.shape[1] * T, generator=gen, device="cuda")
    return state


def _prepare_evict(case, gen):
    B, H = case["batch"], case["kv_heads"]
    lengths = _lengths(case, gen)
    table, blocks = _plain_table(case, lengths, gen)
    state = _cache(case, blocks, gen)
    width = table.shape[1] * T
    # attention sums: most tokens light, a few heavy
    mass = torch.randn(B, H, width, generator=gen, device="cuda").mul(1.5).exp()
    state.update(case=case, lengths=lengths, table=table, mass=mass,
                 keep=(lengths * case["share"]).ceil().int(),
                 mass_out=torch.zeros_like(mass), source=torch.zeros(B, H, width, dtype=torch.int32, device="cuda"),
                 new_lengths=torch.zeros(B, dtype=torch.int32, device="cuda"))
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "shared": _plain_shared, "mass": _plain_mass, "evict": _plain_evict}[
        state["case"]["op"]](state)


def _handle(state):
    """The cache descriptor (and the workspace) that a program keeps with its cache."""
    from quantized_kv_cache_07_gb300 import _lib
    if "desc" not in state:
        c = state["case"]
        state["desc"] = _lib.CacheDesc(
            num_kv_heads=c["kv_heads"], head_dim=D, block_size=T, num_blocks=state["blocks"], k_bits=c["k_bits"],
            v_bits=c["v_bits"], k_codes=state["k"].data_ptr(), v_codes=state["v"].data_ptr(),
            meta=state["meta"].data_ptr(), asym=int(c["asym"]),
            k_channel_factor=None if state["factor"] is None else state["factor"].data_ptr())
        if c["op"] == "shared":
            size = _lib.kvq_decode_shared_workspace_size(state["desc"], c["batch"], c["q_heads"], c["groups"])
            state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
            _lib.kvq_workspace_init(state["workspace"], size)
        if c["op"] == "rope":
            state["rope"] = _lib.RopeDesc(rotary_dim=c["rotary"], interleaved=int(c["interleaved"]),
                                          max_pos=c["max_pos"], table=state["table_cs"].data_ptr())
    return _lib, state["desc"], state["case"]


def _own(state):
    lib, desc, c = _handle(state)
    if c["op"] == "rope":
        Hq, H, qkv = c["q_heads"], c["kv_heads"], state["qkv"]
        q, k, v = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + H) * D], qkv[:, (Hq + H) * D:]
        lib.kvq_rope_append(desc, state["rope"], q, Hq, state["q_out"], k, v, state["pos"], state["seq"],
                            state["slot"], lib.APPEND_QUANT, state["table"], *state["table"].shape)
        lib.kvq_dequant(desc, state["where"], state["k_read"], state["v_read"])
        return state["q_out"], state["k_read"], state["v_read"]
    B = c["batch"]
    if c["op"] == "shared":
        lib.kvq_decode_shared(desc, state["q"], B, c["q_heads"], state["lengths"], state["table"],
                              state["table"].shape[1], c["groups"], state["group_start"], state["prefix_blocks"],
                              state["out"], lse=state["lse"], workspace=state["workspace"],
                              workspace_bytes=state["workspace"].numel())
        return state["out"], state["lse"]
    if c["op"] == "mass":
        lib.kvq_attn_mass(desc, state["q"], B, c["q_heads"], state["lse"], state["lengths"], state["table"],
                          state["table"].shape[1], state["mass"], decay=0.9)
        return state["mass"]
    lib.kvq_evict(desc, state["mass"], state["mass_out"], state["lengths"], state["keep"], state["table"], B,
                  state["table"].shape[1], state["source"], state["new_lengths"], protect_first=c["first"],
                  protect_recent=c["recent"])
    return state["k"], state["v"], state["meta"], state["mass_out"], state["source"], state["new_lengths"]


# ------------------------------------------------------------------ plain forms

def _scales(state, is_key):
    meta, asym = state["meta"], state["case"]["asym"]
    at = 0 if is_key else meta.shape[2] // 2
    return meta[:, :, at, :, None], meta[:, :, at + 1, :, None] if asym else torch.zeros_like(meta[:, :, at, :, None])


def _pool_values(state, is_key):
    """What the pool's codes stand for, [kv_heads, blocks * 16, 128] float32."""
    c = state["case"]
    bits = c["k_bits"] if is_key else c["v_bits"]
    u = _unpack(state["k"] if is_key else state["v"], bits, c["kv_heads"])[..., _cells(bits, is_key, "cuda")]
    x = _stand_for(u, *_scales(state, is_key), bits, c["asym"]).reshape(c["kv_heads"], -1, D)
    return x * state["factor"][:, None] if is_key and state["factor"] is not None else x


def _pool_index(state):
    """The pool's token under each position of each sequence, [batch, positions], and which positions are held."""
    table = state["table"].long()
    at = (table[..., None] * T + torch.arange(T, device="cuda")).flatten(1)
    held = torch.arange(at.shape[1], device="cuda")[None] < state["lengths"][:, None]
    return torch.where(held, at, 0), held


def _pool_scores(state):
    """Scores of every query against every token of the pool, [kv_heads, batch, group, tokens], and which are its own."""
    c, q = state["case"], state["q"]
    B, H = q.shape[0], c["kv_heads"]
    x = q.float().view(B, H, -1, D).transpose(0, 1).reshape(H, -1, D)
    score = torch.matmul(x, _pool_values(state, True).transpose(1, 2)) / math.sqrt(D)
    at, held = _pool_index(state)
    used = torch.zeros(B, score.shape[-1] + 1, dtype=torch.bool, device="cuda")
    used.scatter_(1, torch.where(held, at, score.shape[-1]), True)
    return score.view(H, B, -1, score.shape[-1]), used[:, :-1]


def _rotate(x, cs, interleaved):
    """x [n, heads, 128] rotated by cs [n, pairs, 2], in 64 bits, rounded to float32 and then to bf16."""
    pairs = cs.shape[1]
    a, rest = x[..., :2 * pairs].double(), x[..., 2 * pairs:]
    if interleaved:
        x0, x1 = a[..., 0::2], a[..., 1::2]
    else:
        x0, x1 = a[..., :pairs], a[..., pairs:]
    c, s = cs.double()[:, None, :, 0], cs.double()[:, None, :, 1]
    y0, y1 = x0 * c - x1 * s, x0 * s + x1 * c
    y = torch.stack((y0, y1), -1).flatten(-2) if interleaved else torch.cat((y0, y1), -1)
    return torch.cat((y.float().bfloat16(), rest), -1)


def _plain_rope(state):
    c = state["case"]
    n, Hq, H = c["n"], c["q_heads"], c["kv_heads"]
    x = state["qkv"].view(n, Hq + 2 * H, D)
    cs = state["table_cs"][state["pos"].long()]
    turned = _rotate(x[:, :Hq + H], cs, c["interleaved"])
    key = turned[:, Hq:].float()
    if state["factor"] is not None:
        key = key / state["factor"]
    read = []
    for value, bits in ((key, c["k_bits"]), (x[:, Hq + H:], c["v_bits"])):
        u, s, z = _quantize(value, bits, c["asym"])
        # one rounding, as of a fused multiply-add
        read.append(_stand_for(u, s.double(), z.double(), bits, c["asym"]).float())
    return turned[:, :Hq].contiguous(), read[0], read[1]


def _plain_shared(state):
    score, used = _pool_scores(state)
    B, Hq = state["q"].shape[:2]
    score = torch.where(used[None, :, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    H = score.shape[0]
    out = torch.matmul(p.view(H, -1, p.shape[-1]), _pool_values(state, False)).view(H, B, -1, D) / total
    lse = (top + torch.log(total))[..., 0]
    return out.permute(1, 0, 2, 3).reshape(B, Hq, D).bfloat16(), lse.permute(1, 0, 2).reshape(B, Hq)


def _plain_mass(state):
    score, used = _pool_scores(state)
    H, B, G, tokens = score.shape
    lse = state["lse"].view(B, H, G).transpose(0, 1)
    weight = torch.exp(score - lse[..., None]).sum(2)
    at, held = _pool_index(state)
    weight = torch.gather(weight, 2, at[None].expand(H, -1, -1)).transpose(0, 1)
    mass = state["mass"]
    mass.copy_(torch.where(held[:, None], 0.9 * mass + weight, mass))
    return mass


def _plain_evict(state):
    c, mass = state["case"], state["mass"]
    B, H, width = mass.shape
    slot = torch.arange(width, device="cuda")
    length = state["lengths"].long()[:, None, None]
    keep = torch.minimum(length, state["keep"].long()[:, None, None])
    held = slot < length
    # kept: the first, the recent and then the heaviest; of equal ones the lowest slot
    rank_by = torch.where((slot < c["first"]) | (slot >= length - c["recent"]), math.inf, mass)
    order = torch.where(held, rank_by, -math.inf).sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order))
    kept = held & (rank < keep)
    hole, tail = (slot < keep) & ~kept, (slot >= keep) & kept
    # the i-th hole takes the i-th kept token behind the new length
    of_rank = torch.zeros(B, H, width + 1, dtype=torch.long, device="cuda")
    of_rank.scatter_(-1, torch.where(tail, tail.cumsum(-1) - 1, width), slot.expand(B, H, -1))
    source = torch.where(hole, of_rank.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), slot.expand(B, H, -1))
    now = (slot < keep).expand(B, H, -1)
    state["source"].copy_(torch.where(now, source, state["source"].long()))
    state["mass_out"].copy_(torch.where(now, mass.gather(-1, source), state["mass_out"]))
    state["new_lengths"].copy_(keep[:, 0, 0])
    # move the tokens: head h of physical block f, token t
    table = state["table"].long().clamp(min=0)
    row = torch.arange(B, device="cuda")[:, None, None]
    head = torch.arange(H, device="cuda")[None, :, None].expand(B, H, width)
    to = (head[now], table[row, slot // T].expand(B, H, -1)[now], (slot % T).expand(B, H, -1)[now])
    fr = (head[now], table[row, source // T][now], (source % T)[now])
    for name, is_key in (("k", True), ("v", False)):
        bits = c["k_bits"] if is_key else c["v_bits"]
        at = _cells(bits, is_key, "cuda")
        codes = _unpack(state[name], bits, H)
        new = codes.clone()
        new[to[0][:, None], to[1][:, None], at[to[2]]] = codes[fr[0][:, None], fr[1][:, None], at[fr[2]]]
        state[name].copy_(_pack(new, bits))
    meta = state["meta"].clone()
    meta[to[0], to[1], :, to[2]] = state["meta"][fr[0], fr[1], :, fr[2]]
    state["meta"].copy_(meta)
    # an eviction moves stored bytes and computes nothing on them: the pools come back as they are stored
    return state["k"], state["v"], state["meta"], state["mass_out"], state["source"], state["new_lengths"]


# ------------------------------------------------------------------ cost

def _token_bytes(case, keys=True, values=True):
    per = 8 if case["asym"] else 4
    return (D * case["k_bits"] / 8 + per if keys else 0) + (D * case["v_bits"] / 8 + per if values else 0)


def work(case):
    H, Hq = case["kv_heads"], case["q_heads"]
    if case["op"] == "rope":
        n = case["n"]
        # queries, keys and values in, rotated queries and stored tokens out, the read-back of the stored values
        moved = n * ((2 * Hq + 2 * H) * D * 2 + 2 * H * _token_bytes(case) + 2 * H * D * 4 + 4 * case["rotary"] + 16)
        return {"bytes": moved, "flops": n * ((Hq + H) * 3 * case["rotary"] + 2 * H * 3 * D)}
    B = case["batch"]
    if case["op"] == "shared":
        prefix = sum(case["prefix"] // T - 5 * g for g in range(case["groups"])) * T
        suffix = B * (case["suffix"] + 1) / 2
        attended = suffix + sum((case["prefix"] - 80 * g) * ((g + 1) * B // case["groups"] - g * B // case["groups"])
                                for g in range(case["groups"]))
        return {"bytes": (prefix + suffix) * H * _token_bytes(case) + 2 * B * Hq * D * 2 + 4 * B * Hq,
                "flops": 4 * D * Hq * attended}
    tokens = case["high"] + (B - 1) * (case["low"] + case["high"]) / 2
    if case["op"] == "mass":
        return {"bytes": tokens * H * (_token_bytes(case, values=False) + 8) + B * Hq * (2 * D + 4),
                "flops": 2 * D * Hq * tokens}
    # the sums in; the sums and sources out; the moved tokens read and written (of the kept ones, those behind the new length)
    kept = tokens * case["share"]
    return {"bytes": H * (4 * tokens + 8 * kept + 2 * kept * (1 - case["share"]) * _token_bytes(case)), "flops": tokens * H}


# ------------------------------------------------------------------ in 64 bits, one sequence and head at a time

def _whose(bits, is_key):
    """Token and dim of each code place of a block, found from the place: two lists of 2048."""
    token, dim = [], []
    for place in range(T * D):
        byte, half = (place, 0) if bits == 8 else divmod(place, 2)
        chunk, rest = divmod(byte, 512)
        lane, b = divmod(rest, 16)
        g, t = divmod(lane, 4)
        word = b // 4
        if is_key:
            if bits == 8:
                token.append(g + 8 * (chunk // 2))
                dim.append(32 * t + 16 * (chunk % 2) + b)
            else:
                nib = 2 * (b % 4) + half
                token.append(g + 8 * chunk)
                dim.append(32 * t + 8 * word + 2 * (nib % 4) + nib // 4)
        elif bits == 8:
            j = b % 4
            token.append(2 * t + j // 2 + 8 * (j % 2))
            dim.append(32 * chunk + 16 * (word // 2) + 8 * (word % 2) + g)
        else:
            nib = 2 * (b % 4) + half
            j = 2 * (nib % 2) + nib // 4
            token.append(2 * t + j // 2 + 8 * (j % 2))
            dim.append(64 * chunk + 16 * word + 8 * ((nib % 4) // 2) + g)
    return torch.tensor(token, device="cuda"), torch.tensor(dim, device="cuda")


def _exact_rows(state, b, h, is_key, places):
    """Keys or values of sequence b, head h in 64 bits, [tokens, 128]."""
    c = state["case"]
    bits = c["k_bits"] if is_key else c["v_bits"]
    length = int(state["lengths"][b])
    ids = state["table"][b, : (length + T - 1) // T].long()
    size = T * D * bits // 8
    raw = state["k" if is_key else "v"].view(c["kv_heads"], -1, size)[h, ids].long()
    if bits == 4:
        raw = torch.stack((raw % 16, raw // 16), 2).reshape(len(ids), -1)
    token, dim = places
    x = torch.zeros(len(ids), T, D, dtype=torch.float64, device="cuda")
    x[:, token, dim] = raw.double()
    rec = state["meta"][h, ids].double()
    if c["asym"]:
        x = x * rec[:, 0 if is_key else 2][..., None] + rec[:, 1 if is_key else 3][..., None]
    else:
        x = (x - (128 if bits == 8 else 8)) * rec[:, 0 if is_key else 1][..., None]
    if is_key and state["factor"] is not None:
        x = x * state["factor"][h].double()
    return x.reshape(-1, D)[:length]


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(state)
    if case["op"] == "evict":
        return None  # it chooses and moves: nothing in it is computed
    B, Hq, H = case["batch"], case["q_heads"], case["kv_heads"]
    G = Hq // H
    key_places, value_places = _whose(case["k_bits"], True), _whose(case["v_bits"], False)
    q = state["q"].double()
    if case["op"] == "mass":
        mass = state["mass"].double()
        for b in range(B):
            for h in range(H):
                k = _exact_rows(state, b, h, True, key_places)
                s = q[b, h * G:(h + 1) * G] @ k.T * D ** -0.5
                w = torch.exp(s - state["lse"][b, h * G:(h + 1) * G, None].double()).sum(0)
                mass[b, h, :len(w)] = mass[b, h, :len(w)] * 0.9 + w
        return mass
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, Hq, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(H):
            s = q[b, h * G:(h + 1) * G] @ _exact_rows(state, b, h, True, key_places).T * D ** -0.5
            out[b, h * G:(h + 1) * G] = torch.softmax(s, -1) @ _exact_rows(state, b, h, False, value_places)
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
    return out, lse


def _exact_rope(state):
    """Turned queries in 64 bits; the stored values from the rotated keys, which are bf16 by definition."""
    c = state["case"]
    Hq, H, R = c["q_heads"], c["kv_heads"], c["rotary"]
    x = state["qkv"].double().view(c["n"], -1, D)
    lead = torch.arange(0, R, 2, device="cuda") if c["interleaved"] else torch.arange(R // 2, device="cuda")
    mate = lead + (1 if c["interleaved"] else R // 2)
    angle = torch.view_as_complex(state["table_cs"].double().contiguous())[state["pos"].long()][:, None]
    turned = torch.complex(x[:, :Hq + H, lead], x[:, :Hq + H, mate]) * angle
    y = x[:, :Hq + H].clone()
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
