"""Measured cases of the operators around the paged KV cache.

  append   art_append_kv: rotate the new tokens' queries and keys to their
           positions and write keys and values into the cache's pages
  extend   dense_extend: attention of several new tokens of each sequence over
           its cached tokens (causal), or over an encoder's states (full)
  shared   dense_decode_shared: decode attention of a batch whose groups of
           sequences share a long prefix, read once for the group

A case is a dict of sizes; lengths that differ from sequence to sequence are
drawn from the case's own `spread` number, so they belong to the case and not to
the seed of the data.
"""
import math
import random

import torch

own = False


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _append(name, dtype, heads, page, batch, new, ctx, rot, interleaved, fused, spread):
    return {"name": name, "op": "append", "dtype": dtype, "hq": heads[0], "hkv": heads[1], "d": heads[2],
            "page": page, "batch": batch, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "rot": rot, "interleaved": interleaved, "fused": fused, "spread": spread}


def _extend(name, dtype, heads, page, batch, new, ctx, causal, spread):
    return {"name": name, "op": "extend", "dtype": dtype, "hq": heads[0], "hkv": heads[1], "d": heads[2],
            "page": page, "batch": batch, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "causal": causal, "spread": spread}


def _shared(name, dtype, heads, page, groups, members, prefix, tail, singles, spread):
    return {"name": name, "op": "shared", "dtype": dtype, "hq": heads[0], "hkv": heads[1], "d": heads[2],
            "page": page, "groups": groups, "members_lo": members[0], "members_hi": members[1],
            "prefix_lo": prefix[0], "prefix_hi": prefix[1], "tail_lo": tail[0], "tail_hi": tail[1],
            "singles": singles, "spread": spread}


def listed():
    return [
        # one user's next token: nothing but latency
        _append("append_step_b1", "bf16", (32, 8, 128), 16, 1, (1, 1), (900, 900), 128, False, False, 1),
        # a serving step of 128 sequences, queries, keys and values still side by side in the projection's rows
        _append("append_step_b128", "bf16", (32, 8, 128), 16, 128, (1, 1), (0, 8191), 128, False, True, 2),
        # a mixed step: short and long prompt chunks, neighbouring pairs rotated over half of the head
        _append("append_chunks", "bf16", (28, 4, 128), 64, 7, (1, 4001), (0, 120000), 64, True, False, 3),
        # whole prompts of a large prefill batch
        _append("append_prompts", "bf16", (32, 8, 128), 16, 8, (2048, 8192), (0, 0), 128, False, True, 4),
        # verification of five drafted tokens of each sequence
        _extend("extend_drafts_b16", "bf16", (32, 8, 128), 16, 16, (5, 5), (1000, 8192), True, 5),
        # prompt chunks behind contexts of all lengths
        _extend("extend_chunks", "bf16", (32, 8, 128), 16, 4, (1024, 2048), (0, 8192), True, 6),
        # a decoder's prompt over an encoder's states (no causal mask)
        _extend("extend_encoder", "bf16", (8, 8, 64), 64, 12, (1, 449), (333, 1500), False, 7),
        # a small model in fp32, as for reference runs
        _extend("extend_f32", "f32", (8, 2, 64), 32, 3, (1, 201), (100, 2000), True, 8),
        # a few samples of one prompt
        _shared("shared_samples_b4", "bf16", (32, 8, 128), 16, 1, (4, 4), (1001, 1001), (1, 64), 0, 9),
        # a batch behind one system prompt
        _shared("shared_prompt_b64", "bf16", (32, 8, 128), 16, 1, (64, 64), (8192, 8192), (1, 1024), 0, 10),
        # several prompts with few and many sequences each, and sequences that share nothing
        _shared("shared_mixed", "bf16", (28, 4, 128), 64, 6, (1, 24), (3001, 20000), (0, 2000), 5, 11),
        # a large batch behind a long document
        _shared("shared_document_b128", "bf16", (32, 8, 128), 16, 1, (128, 128), (32768, 32768), (64, 2047), 0, 12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _run(rng, lo, hi):
    a, b = sorted((_log(rng, lo, hi), _log(rng, lo, hi)))
    return a, b


def draw(rng):
    op = rng.choice(("append", "extend", "shared"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    heads = rng.choice(((32, 8, 128), (28, 4, 128), (8, 2, 64), (8, 8, 64), (8, 1, 128), (6, 3, 64), (8, 2, 128)))
    page = rng.choice((8, 16, 16, 32, 64, 256))
    spread = rng.randrange(1 << 20)
    if op == "append":
        batch = _log(rng, 1, 128)
        new = rng.choice(((1, 1), _run(rng, 1, max(2, min(4000, 20000 // batch)))))
        rot = rng.choice((heads[2], heads[2], heads[2] // 2, 0))
        c = _append("", dtype, heads, page, batch, new, _run(rng, 1, min(8192, 400000 // batch)), rot,
                    rng.random() < 0.4, rng.random() < 0.5, spread)
    elif op == "extend":
        causal = rng.random() < 0.7
        batch = _log(rng, 1, 16)
        top = (4096 if dtype == "bf16" else 1024) // batch
        c = _extend("", dtype, heads, page, batch, _run(rng, 1, max(2, top)),
                    _run(rng, 1, 4096), causal, spread)
    else:
        groups = _log(rng, 1, 5)
        c = _shared("", dtype, heads, page, groups, _run(rng, 1, max(1, (64 if dtype == "bf16" else 24) // groups)),
                    _run(rng, 100, 16384 if dtype == "bf16" else 4096), _run(rng, 1, 1024),
                    rng.choice((0, 0, 1, 3)), spread)
    del c["name"]
    return c


# ----------------------------------------------------------------------------
# lengths of a case (plain numbers)
# ----------------------------------------------------------------------------
def _lens(case):
    """append, extend: (new tokens, cached tokens after them) of each sequence.
    shared: (group of each sequence or -1, its length, prefix of each group)."""
    r = random.Random(case["spread"])
    if case["op"] == "shared":
        of, seq, prefix = [], [], []
        for j in range(case["groups"]):
            prefix.append(r.randint(case["prefix_lo"], case["prefix_hi"]))
            for _ in range(r.randint(case["members_lo"], case["members_hi"])):
                of.append(j)
                seq.append(prefix[-1] + r.randint(case["tail_lo"], case["tail_hi"]))
        for _ in range(case["singles"]):
            of.append(-1)
            seq.append(r.randint(1, case["prefix_hi"]))
        return of, seq, prefix
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    behind = case["op"] == "append" or case["causal"]  # an encoder's states do not hold the new tokens
    return new, [c + n if behind else c for n, c in zip(new, ctx)]


def _pages(n, page):
    return -(-n // page)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        new, seq = _lens(case)
        t = sum(new)
        turned = t * (hq + hkv) * case["rot"]
        return {"bytes": t * (hq + 2 * hkv) * d * e * 2 + 8 * len(new) + 4, "flops": 3 * turned}
    if case["op"] == "extend":
        new, seq = _lens(case)
        pairs = sum(n * s - (n * (n - 1) // 2 if case["causal"] else 0) for n, s in zip(new, seq))
        return {"bytes": (2 * sum(new) * hq + 2 * sum(seq) * hkv) * d * e, "flops": 4 * d * hq * pairs}
    of, seq, prefix = _lens(case)
    used = [p for j, p in enumerate(prefix) if j in of]
    keys = sum(used) + sum(s - (prefix[j] if j >= 0 else 0) for j, s in zip(of, seq))
    return {"bytes": (2 * len(seq) * hq + 2 * keys * hkv) * d * e, "flops": 4 * d * hq * sum(seq)}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]

    def normal(*size):
        return torch.randn(*size, generator=gen, device=dev, dtype=dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    st = {"case": case}
    if case["op"] == "shared":
        of, seq, prefix = _lens(case)
        batch, new = len(seq), [1] * len(seq)
    else:
        new, seq = _lens(case)
        batch = len(seq)
    cols = max(1, max(_pages(s, page) for s in seq))
    # the block table: pages handed out in random order; whole pages of a shared prefix are the leader's
    need = [_pages(s, page) for s in seq]
    lead, kept = list(range(batch)), [0] * batch
    if case["op"] == "shared":
        first = {}
        for b, j in enumerate(of):
            lead[b] = first.setdefault(j, b) if j >= 0 else b
            if lead[b] != b:
                kept[b] = prefix[j] // page
    rows = torch.arange(batch, device=dev)[:, None]
    col = torch.arange(cols, device=dev)[None, :]
    lead_t, kept_t, need_t = (torch.tensor(v, device=dev)[:, None] for v in (lead, kept, need))
    mine = (col >= kept_t) & (col < need_t)
    number = mine.reshape(-1).cumsum(0).reshape(batch, cols) - 1
    total = sum(n - k for n, k in zip(need, kept))
    pool = total + max(2, total // 16)
    perm = torch.randperm(pool, generator=gen, device=dev)
    table = torch.where(mine, perm[number.clamp(min=0)], torch.zeros_like(number))
    table = torch.where(col < kept_t, table[lead_t.expand(-1, cols), col.expand(batch, -1)], table)
    st["block_table"] = table.to(torch.int32).contiguous()
    st["seq_lens"] = ints(seq)
    st["k_cache"] = normal(pool, hkv, page, d)
    st["v_cache"] = normal(pool, hkv, page, d)
    st["sizes"] = {"batch": batch, "num_q_heads": hq, "num_kv_heads": hkv, "head_dim": d, "page_size": page,
                   "block_size": 64, "max_pages_per_seq": cols, "max_visit": 1, "num_probe": 1,
                   "num_pages_total": pool, "dtype": 0 if case["dtype"] == "bf16" else 1}
    if case["op"] == "shared":
        # a partly filled last page of the prefix is copied into each member's own page, as a server does
        for j, p in enumerate(prefix):
            m = [b for b in range(batch) if of[b] == j]
            if p % page and len(m) > 1:
                c = p // page
                src = st["block_table"][m[0], c].long()
                dst = st["block_table"][torch.tensor(m[1:], device=dev), c].long()
                for cache in (st["k_cache"], st["v_cache"]):
                    cache[dst, :, : p % page] = cache[src, :, : p % page]
        starts = [of.index(j) if j in of else 0 for j in range(len(prefix))]
        st["group_offsets"] = ints(starts + [sum(1 for j in of if j >= 0)])
        st["prefix_lens"] = ints(prefix)
        st["lead"], st["group"] = torch.tensor(lead, device=dev), torch.tensor(of, device=dev)
        st["q"] = normal(batch, hq, d)
        st["out"] = torch.empty_like(st["q"])
        return st
    tokens = sum(new)
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    st["q_offsets"] = ints(offsets)
    st["single"] = all(n == 1 for n in new)
    st["most_new"] = max(new)
    if case["op"] == "extend":
        st["q"] = normal(tokens, hq, d)
        st["out"] = torch.empty_like(st["q"])
        return st
    if case["fused"]:  # one projection's rows: queries, keys and values of a token side by side
        qkv = normal(tokens, hq + 2 * hkv, d)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        st["q"], st["k"], st["v"] = normal(tokens, hq, d), normal(tokens, hkv, d), normal(tokens, hkv, d)
    half = torch.arange(case["rot"] // 2, device=dev, dtype=torch.float64)
    st["inv_freq"] = torch.exp(half * (-2.0 * math.log(500000.0) / max(1, case["rot"]))).float()
    st["q_out"] = torch.empty(tokens, hq, d, dtype=dt, device=dev)
    return st


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------
def _token_places(st):
    """Sequence, place among the new tokens and position of every new token."""
    t = torch.arange(st["q"].shape[0], device=st["q"].device)
    off = st["q_offsets"].long()
    seq = torch.searchsorted(off[1:].contiguous(), t, right=True)
    i = t - off[seq]
    new = off[1:] - off[:-1]
    return seq, i, st["seq_lens"].long()[seq] - new[seq] + i


def _turn(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    x = x.float()
    y, rest = x[..., :rot], x[..., rot:]
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., : rot // 2], y[..., rot // 2:])
    c, s = cos[:, None], sin[:, None]
    a, b = a * c - b * s, b * c + a * s
    y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((y, rest), -1)


def _plain_append(st):
    case, page = st["case"], st["case"]["page"]
    seq, _, pos = _token_places(st)
    angle = pos.double()[:, None] * st["inv_freq"].double()[None, :]
    cos, sin = angle.cos().float(), angle.sin().float()
    dt = st["q"].dtype
    st["q_out"].copy_(_turn(st["q"], cos, sin, case["interleaved"]).to(dt))
    at = st["block_table"].long()[seq, pos // page], pos % page
    st["k_cache"][at[0], :, at[1]] = _turn(st["k"], cos, sin, case["interleaved"]).to(dt)
    st["v_cache"][at[0], :, at[1]] = st["v"]
    return st["q_out"], st["k_cache"], st["v_cache"]


def _attend(q, k, v, limit):
    """q [B, H, R, d], k and v [B, H, L, d], limit [B, 1, R]: keys below it are seen. fp32."""
    s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    hidden = torch.arange(k.shape[-2], device=q.device) >= limit[..., None]
    s = s.masked_fill(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)


def _rows(cache, table):
    """The cached rows behind a block table: [B, heads, columns * page, d] in fp32."""
    b, cols = table.shape
    x = cache[table.long()].permute(0, 2, 1, 3, 4)
    return x.reshape(b, cache.shape[1], cols * cache.shape[2], cache.shape[3]).float()


def _plain_extend(st):
    case = st["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    group = hq // hkv
    seq, i, _ = _token_places(st)
    off, lens = st["q_offsets"].long(), st["seq_lens"].long()
    batch, n = lens.shape[0], st["most_new"]
    new = off[1:] - off[:-1]
    at = torch.arange(n, device=off.device)[None, :]
    idx = (off[:-1, None] + at).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][idx].float().reshape(batch, n, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(batch, hkv, n * group, d)
    limit = lens[:, None] - new[:, None] + at + 1 if case["causal"] else lens[:, None].expand(-1, n)
    limit = limit[:, :, None].expand(-1, -1, group).reshape(batch, 1, n * group)
    o = _attend(q, _rows(st["k_cache"], st["block_table"]), _rows(st["v_cache"], st["block_table"]), limit)
    o = o.reshape(batch, hkv, n, group, d).permute(0, 2, 1, 3, 4).reshape(batch, n, hq, d)
    st["out"].copy_(o[seq, i].to(st["out"].dtype))
    return st["out"]


def _plain_shared(st):
    case = st["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    lens = st["seq_lens"].long()
    batch = lens.shape[0]
    # a page that lies wholly in the prefix is the leader's; the page that the prefix ends in is each member's copy
    whole = torch.where(st["group"] >= 0, st["prefix_lens"].long()[st["group"].clamp(min=0)] // page,
                        torch.zeros_like(st["group"]))
    table = st["block_table"]
    led = torch.arange(table.shape[1], device=table.device)[None, :] < whole[:, None]
    table = torch.where(led, table[st["lead"]], table)
    q = st["q"].float().reshape(batch, hkv, hq // hkv, d)
    limit = lens[:, None, None].expand(-1, 1, hq // hkv)
    o = _attend(q, _rows(st["k_cache"], table), _rows(st["v_cache"], table), limit)
    st["out"].copy_(o.reshape(batch, hq, d).to(st["out"].dtype))
    return st["out"]


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _kept(st):
    """The library, the shape and the workspace that a user's program keeps between calls."""
    if "kept" not in st:
        import kv_cache_early_gb300 as K
        shape = K.make_shape(**st["sizes"])
        if st["case"]["op"] == "append":
            n = K.art_append_workspace_bytes(shape)
        elif st["case"]["op"] == "extend":
            n = K.dense_extend_workspace_bytes(shape, st["q"].shape[0])
        else:
            n = K.dense_decode_shared_workspace_bytes(shape, st["prefix_lens"].shape[0])
        st["kept"] = K, shape, torch.empty(n, dtype=torch.uint8, device=st["q"].device)
    return st["kept"]


def run(state):
    st, case = state, state["case"]
    if not own:
        return {"append": _plain_append, "extend": _plain_extend, "shared": _plain_shared}[case["op"]](st)
    K, shape, workspace = _kept(st)
    if case["op"] == "append":
        # a step of one token for each sequence needs no offsets
        K.art_append_kv(st["q"], st["k"], st["v"], st["block_table"], st["seq_lens"],
                        None if st["single"] else st["q_offsets"], st["inv_freq"], st["q_out"], st["k_cache"],
                        st["v_cache"], shape, workspace, rot_dim=case["rot"], interleaved=case["interleaved"])
        return st["q_out"], st["k_cache"], st["v_cache"]
    if case["op"] == "extend":
        K.dense_extend(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["seq_lens"], st["q_offsets"],
                       st["out"], shape, workspace, causal=case["causal"])
        return st["out"]
    K.dense_decode_shared(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["seq_lens"],
                          st["group_offsets"], st["prefix_lens"], st["out"], shape, workspace)
    return st["out"]


# ----------------------------------------------------------------------------
# the definitions in 64 bits, one sequence (and head) at a time
# ----------------------------------------------------------------------------
def _cached(cache, table, b, lo, hi, page):
    """Rows lo..hi-1 of sequence b, token by token through the table: [heads, hi - lo, d] in fp64."""
    t = torch.arange(lo, hi, device=cache.device)
    return cache[table[b].long()[t // page], :, t % page].double().transpose(0, 1)


def _softmax_mean(q, k, v, seen):
    """One head: q [R, d], k, v [L, d], seen [R, L]."""
    s = (q @ k.t()) * (q.shape[-1] ** -0.5)
    s[~seen] = -math.inf
    return torch.softmax(s, -1) @ v


def exact(case, seed):
    st = prepare(case, seed)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    g = hq // hkv
    dev = st["q"].device
    if case["op"] == "append":
        new, seq = _lens(case)
        rot = case["rot"]
        q_out = st["q"].double().clone()
        k_new = st["k"].double().clone()
        k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
        if case["interleaved"]:
            first = torch.arange(0, rot, 2, device=dev)
            second = first + 1
        else:
            first = torch.arange(rot // 2, device=dev)
            second = first + rot // 2
        t0 = 0
        for b, (n, s) in enumerate(zip(new, seq)):
            pos = torch.arange(s - n, s, device=dev)
            turn = torch.polar(torch.ones(1, dtype=torch.float64, device=dev),
                               pos.double()[:, None, None] * st["inv_freq"].double())
            for x in (q_out, k_new):
                z = torch.complex(x[t0:t0 + n, :, first], x[t0:t0 + n, :, second]) * turn
                x[t0:t0 + n, :, first], x[t0:t0 + n, :, second] = z.real.clone(), z.imag.clone()
            where = st["block_table"][b].long()[pos // page]
            k_cache[where, :, pos % page] = k_new[t0:t0 + n]
            v_cache[where, :, pos % page] = st["v"][t0:t0 + n].double()
            t0 += n
        return q_out, k_cache, v_cache
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=dev)
    if case["op"] == "extend":
        new, seq = _lens(case)
        t0 = 0
        for b, (n, s) in enumerate(zip(new, seq)):
            keys = torch.arange(s, device=dev)
            last = torch.arange(s - n, s, device=dev) if case["causal"] else torch.full((n,), s - 1, device=dev)
            seen = (keys[None, :] <= last[:, None])
            k, v = (_cached(st[x], st["block_table"], b, 0, s, page) for x in ("k_cache", "v_cache"))
            for h in range(hq):
                out[t0:t0 + n, h] = _softmax_mean(st["q"][t0:t0 + n, h].double(), k[h // g], v[h // g], seen)
            t0 += n
        return out
    of, seq, prefix = _lens(case)
    shared = {}
    for b, (j, s) in enumerate(zip(of, seq)):
        p = prefix[j] if j >= 0 else 0
        if j >= 0 and j not in shared:
            shared = {j: [_cached(st[x], st["block_table"], b, 0, p, page) for x in ("k_cache", "v_cache")]}
        k, v = (_cached(st[x], st["block_table"], b, p, s, page) for x in ("k_cache", "v_cache"))
        if j >= 0:
            k, v = (torch.cat((a, c), 1) for a, c in zip(shared[j], (k, v)))
        for h in range(hkv):
            rows = slice(h * g, (h + 1) * g)
            out[b, rows] = _softmax_mean(st["q"][b, rows].double(), k[h], v[h],
                                         torch.ones(g, s, dtype=torch.bool, device=dev))
    return out
