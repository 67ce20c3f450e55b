"""Measured cases of the operators of a paged KV cache that is held in 4 bits.

  append   art_append_kv4: rotate the new tokens' queries and keys to their positions,
           quantise keys and values and write them into the cache's pages; then
           art_read_kv4 of these tokens, so that a pass gives what the cache now stands for
  read     art_read_kv4: the cached values, into the pages of a plain cache or into rows
  attend   dense_extend_kv4: attention over the cached tokens, of one new token of each
           sequence (decode) or of several (drafted tokens, prompt chunks)

The cache, bytes [pages][KV heads][page * (d + 8 d / group)]: the tokens of a page come in slabs
of S = min(page, 64), and a slab has, one after the other,
  the keys' codes    [S / 8][d / 32][8 tokens][16 bytes], two columns a byte, the lower one in the lower bits
  the values' codes  as the keys'
  the keys' scales   [S / 8][d / group][8 tokens] pairs of bf16: step, lowest
  the values' scales as the keys'
A column's value is lowest + step * code. Of the values x of a token's group of columns, lowest is the
largest bf16 that is no larger than min(x), step the bf16 nearest to (max(x) - lowest) / 15 and the code
the whole number nearest to (x - lowest) / step (ties to even), 15 at most.

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
def _case(name, op, dtype, heads, page, group, batch, new, ctx, spread, **more):
    return {"name": name, "op": op, "dtype": dtype, "hq": heads[0], "hkv": heads[1], "d": heads[2], "page": page,
            "group": group, "batch": batch, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "spread": spread, **more}


def _append(name, dtype, heads, page, group, batch, new, ctx, rot, interleaved, fused, spread):
    return _case(name, "append", dtype, heads, page, group, batch, new, ctx, spread, rot=rot, interleaved=interleaved,
                 fused=fused)


def _read(name, dtype, heads, page, group, batch, ctx, paged, spread):
    """paged: every token, to a plain cache's pages; else the last new_lo .. new_hi ones, to rows"""
    return _case(name, "read", dtype, heads, page, group, batch, (0, 0) if paged else (1, ctx[1]), ctx, spread, paged=paged)


def _attend(name, dtype, heads, page, group, batch, new, ctx, causal, spread):
    return _case(name, "attend", dtype, heads, page, group, batch, new, ctx, spread, causal=causal)


def listed():
    return [
        # one user's next token: nothing but latency
        _append("append_step_b1", "bf16", (32, 8, 128), 16, 64, 1, (1, 1), (900, 900), 128, False, False, 1),
        # a serving step of 128 sequences, queries, keys and values still side by side in the projection's rows
        _append("append_step_b128", "bf16", (32, 8, 128), 16, 128, 128, (1, 1), (0, 8191), 128, False, True, 2),
        # a mixed step: short and long prompt chunks, neighbouring pairs rotated over half of the head
        _append("append_chunks", "bf16", (28, 4, 128), 64, 32, 7, (1, 4001), (0, 60000), 64, True, False, 3),
        # whole prompts of a large prefill batch
        _append("append_prompts", "bf16", (32, 8, 128), 16, 64, 8, (2048, 8192), (0, 0), 128, False, True, 4),
        # contexts of several sequences handed to an operator that reads a plain cache
        _read("read_pages", "bf16", (32, 8, 128), 16, 64, 8, (2048, 16384), True, 5),
        # the newest tokens of a few sequences of a small model in fp32, for a look at what was kept
        _read("read_rows_f32", "f32", (8, 2, 64), 32, 32, 5, (100, 4000), False, 6),
        # one user's decode step
        _attend("decode_b1", "bf16", (32, 8, 128), 16, 64, 1, (1, 1), (4000, 4000), True, 7),
        # a serving step of a batch of ordinary lengths
        _attend("decode_b64", "bf16", (32, 8, 128), 16, 64, 64, (1, 1), (0, 8191), True, 8),
        # a few long documents
        _attend("decode_long", "bf16", (28, 4, 128), 64, 128, 8, (1, 1), (30000, 131071), True, 9),
        # a small model in fp32, as for reference runs
        _attend("decode_f32", "f32", (8, 2, 64), 32, 32, 5, (1, 1), (100, 4000), True, 10),
        # verification of five drafted tokens of each sequence
        _attend("drafts_b16", "bf16", (32, 8, 128), 16, 32, 16, (5, 5), (1000, 8192), True, 11),
        # prompt chunks behind contexts of all lengths
        _attend("prompt_chunks", "bf16", (32, 8, 128), 16, 64, 4, (1024, 2048), (0, 8192), True, 12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _run(rng, lo, hi):
    a, b = sorted((_log(rng, lo, hi), _log(rng, lo, hi)))
    return a, b


def draw(rng):
    op = rng.choice(("append", "read", "attend", "attend"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    heads = rng.choice(((32, 8, 128), (28, 4, 128), (8, 2, 64), (8, 8, 64), (8, 1, 128), (6, 3, 64), (8, 2, 128)))
    page = rng.choice((8, 16, 16, 32, 64, 256))
    group = rng.choice((32, 64, heads[2]))
    spread = rng.randrange(1 << 20)
    if op == "append":
        batch = _log(rng, 1, 128)
        new = rng.choice(((1, 1), _run(rng, 1, max(2, min(4000, 20000 // batch)))))
        rot = rng.choice((heads[2], heads[2], heads[2] // 2, 0))
        c = _append("", dtype, heads, page, group, batch, new, _run(rng, 1, min(8192, 400000 // batch)), rot,
                    rng.random() < 0.4, rng.random() < 0.5, spread)
    elif op == "read":
        batch = _log(rng, 1, 32)
        c = _read("", dtype, heads, page, group, batch, _run(rng, 1, min(16384, 100000 // batch)), rng.random() < 0.5, spread)
    elif rng.random() < 0.6:
        batch = _log(rng, 1, 64)
        most = (400000 if dtype == "bf16" else 60000) // batch
        c = _attend("", dtype, heads, page, group, batch, (1, 1), _run(rng, 1, min(131072, most)), True, spread)
    else:
        batch = _log(rng, 1, 16)
        top = (4096 if dtype == "bf16" else 512) // batch
        c = _attend("", dtype, heads, page, group, batch, _run(rng, 1, max(2, top)), _run(rng, 1, 4096),
                    rng.random() < 0.8, spread)
    del c["name"]
    return c


# ----------------------------------------------------------------------------
# lengths of a case (plain numbers)
# ----------------------------------------------------------------------------
def _lens(case):
    """(new tokens, cached tokens) of each sequence; the new ones are among the cached ones,
    but where rows of no causal order attend."""
    r = random.Random(case["spread"])
    if case["op"] == "read":
        seq = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
        return [s if case["paged"] else r.randint(1, s) for s in seq], seq
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    behind = case["op"] == "append" or case["causal"]
    return new, [c + n if behind else max(c, 1) for n, c in zip(new, ctx)]


def _page_bytes(case):
    return case["page"] * (case["d"] + 8 * (case["d"] // case["group"]))


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    held = hkv * (d + 8 * (d // case["group"]))  # bytes of a token in the cache
    new, seq = _lens(case)
    t = sum(new)
    if case["op"] == "append":  # rows in, queries out, the cache written; then its values
        return {"bytes": t * (2 * hq * d * e + 2 * hkv * d * e + held) + t * 2 * hkv * d * e,
                "flops": t * (3 * (hq + hkv) * case["rot"] + 10 * hkv * d)}
    if case["op"] == "read":
        return {"bytes": t * (held + 2 * hkv * d * e), "flops": 4 * t * hkv * d}
    pairs = sum(n * s - (n * (n - 1) // 2 if case["causal"] else 0) for n, s in zip(new, seq))
    return {"bytes": 2 * t * hq * d * e + sum(seq) * held, "flops": 4 * d * hq * pairs}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    hq, hkv, d, page, group = case["hq"], case["hkv"], case["d"], case["page"], case["group"]

    def normal(*size, dtype=dt):
        return torch.randn(*size, generator=gen, device=dev, dtype=dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    st = {"case": case}
    new, seq = _lens(case)
    batch = len(seq)
    # the block table: pages handed out in random order
    need = [-(-s // page) for s in seq]
    cols = max(1, max(need))
    col = torch.arange(cols, device=dev)[None, :]
    mine = col < torch.tensor(need, device=dev)[:, None]
    number = (mine.reshape(-1).cumsum(0).reshape(batch, cols) - 1).clamp(min=0)
    total = sum(need)
    pool = total + max(2, total // 16)

    def table():
        perm = torch.randperm(pool, generator=gen, device=dev)
        return torch.where(mine, perm[number], torch.zeros_like(number)).to(torch.int32).contiguous()

    st["block_table"] = table()
    st["seq_lens"] = ints(seq)
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    st["q_offsets"] = ints(offsets)
    st["single"] = all(n == 1 for n in new)
    st["most_new"] = max(new)
    tokens = offsets[-1]
    st["sizes"] = {"batch": batch, "num_q_heads": hq, "num_kv_heads": hkv, "head_dim": d, "page_size": page,
                   "block_size": 64, "max_pages_per_seq": cols, "max_visit": 1, "num_probe": 1,
                   "num_pages_total": pool, "dtype": 0 if case["dtype"] == "bf16" else 1}
    # a filled cache: codes as those of normal values, steps and lowest values of all sizes around theirs
    st["cache"] = torch.empty(pool, hkv, _page_bytes(case), dtype=torch.uint8, device=dev)
    for keys in (True, False):
        codes, scales = _parts(st["cache"], case, keys)

        def nibbles():
            return normal(codes.shape, dtype=torch.float16).mul_(3.0).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)

        codes.copy_(nibbles() | nibbles() << 4)
        step = torch.exp(0.3 * normal(scales.shape[:-1], dtype=torch.float32)) * 0.3
        scales[..., 0] = step
        scales[..., 1] = step * (normal(scales.shape[:-1], dtype=torch.float32) - 7.5)
    if case["op"] == "read":
        rows = (pool, hkv, page, d) if case["paged"] else (tokens, hkv, d)
        st["k_out"], st["v_out"] = (torch.zeros(rows, dtype=dt, device=dev) for _ in range(2))
        st["out_table"] = table() if case["paged"] else None
        return st
    if case["op"] == "attend":
        st["q"] = normal(tokens, hq, d)
        st["out"] = torch.empty_like(st["q"])
        return st
    # keys have columns of larger and smaller values
    wide = torch.exp(0.5 * normal(hkv, d, dtype=torch.float32)).to(dt)
    qkv = normal(tokens, hq + 2 * hkv, d)
    qkv[:, hq:hq + hkv] *= wide
    if case["fused"]:  # one projection's rows: queries, keys and values of a token side by side
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        st["q"], st["k"], st["v"] = (x.contiguous() for x in (qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]))
    half = torch.arange(case["rot"] // 2, device=dev, dtype=torch.float64)
    st["inv_freq"] = torch.exp(half * (-2.0 * math.log(500000.0) / max(1, case["rot"]))).float()
    st["q_out"] = torch.empty(tokens, hq, d, dtype=dt, device=dev)
    st["k_out"], st["v_out"] = (torch.empty(tokens, hkv, d, dtype=dt, device=dev) for _ in range(2))
    return st


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------
def _parts(cache, case, keys):
    """Codes [pages, heads, slabs, octets, d / 32, 8, 16] and scales [pages, heads, slabs, octets, groups, 8, 2]
    of the keys or of the values: views of the cache."""
    d, n = case["d"], case["d"] // case["group"]
    slab = min(case["page"], 64)
    x = cache.unflatten(-1, (case["page"] // slab, slab * (d + 8 * n)))
    c0 = 0 if keys else slab * d // 2
    s0 = slab * d + (0 if keys else slab * 4 * n)
    codes = x[..., c0:c0 + slab * d // 2].unflatten(-1, (slab // 8, d // 32, 8, 16))
    return codes, x[..., s0:s0 + slab * 4 * n].view(torch.bfloat16).unflatten(-1, (slab // 8, n, 8, 2))


def _place(case, place):
    """A place inside a page as slab, octet and token of the octet."""
    slab = min(case["page"], 64)
    at = place % case["page"]
    return at // slab, at % slab // 8, at % 8


def _values(codes, scales):
    """codes [..., d / 2] bytes, scales [..., groups, 2]: the values, in fp32."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    s = scales.float()
    c = c.unflatten(-1, (s.shape[-2], -1))
    return (s[..., 1:2] + s[..., 0:1] * c).flatten(-2)


def _token_places(st):
    """Sequence, place among the new tokens and cache place of every new token."""
    off = st["q_offsets"].long()
    t = torch.arange(st["k_out"].shape[0] if "k_out" in st else st["q"].shape[0], device=off.device)
    seq = torch.searchsorted(off[1:].contiguous(), t, right=True)
    i = t - off[seq]
    new = off[1:] - off[:-1]
    return seq, i, st["seq_lens"].long()[seq] - new[seq] + i


def _at(st, seq, pos):
    slab, octet, i = _place(st["case"], pos)
    return st["block_table"].long()[seq, pos // st["case"]["page"]], slab, octet, i


def _get(st, seq, pos, keys):
    """The values of one token each: [tokens, heads, d] in fp32."""
    codes, scales = _parts(st["cache"], st["case"], keys)
    page, slab, octet, i = _at(st, seq, pos)
    return _values(codes[page, :, slab, octet, :, i].flatten(-2), scales[page, :, slab, octet, :, i])


def _turn(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    x = x.to(cos.dtype)
    y, rest = x[..., :rot], x[..., rot:]
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., : rot // 2], y[..., rot // 2:])
    c, s = cos[:, None], sin[:, None]
    a, b = a * c - b * s, b * c + a * s
    y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((y, rest), -1)


def _to_bf16(x):
    """fp64 values rounded once to bf16's, ties to even (a cast goes by way of fp32)."""
    u = x.contiguous().view(torch.int64)
    return ((u + ((1 << 44) - 1) + (u >> 45 & 1)) >> 45 << 45).view(torch.float64)


def _floor_bf16(x):
    """The largest bf16 values that are no larger than fp32 values x."""
    u = x.contiguous().view(torch.int32)
    up = (u < 0) & ((u & 0xFFFF) != 0)
    return ((u >> 16) + up.int() << 16).view(torch.float32)


def _quantised(x, group):
    """x [tokens, heads, d] in 64 bits, values of the cache's type: codes [.., d / 2] and (step, lowest) [.., groups, 2].
    In 64 bits, since values stand next to the borders between codes."""
    x = x.unflatten(-1, (-1, group))
    low = _floor_bf16(x.amin(-1).float()).double()
    step = _to_bf16((x.amax(-1) - low) / 15.0)
    step = torch.where(step < 2.0 ** -100, torch.zeros_like(step), step)
    per = torch.where(step == 0, torch.ones_like(step), step)
    c = torch.round((x - low[..., None]) / per[..., None]).clamp(0, 15).flatten(-2).to(torch.uint8)
    return c[..., 0::2] | c[..., 1::2] << 4, torch.stack((step, low), -1).to(torch.bfloat16)


def _plain_append(st):
    case = st["case"]
    seq, _, pos = _token_places(st)
    dt = st["q"].dtype
    angle = pos.double()[:, None] * st["inv_freq"].double()[None, :]
    cos, sin = angle.cos(), angle.sin()
    st["q_out"].copy_(_turn(st["q"], cos.float(), sin.float(), case["interleaved"]).to(dt))
    k = _turn(st["k"], cos, sin, case["interleaved"])
    k = _to_bf16(k) if dt == torch.bfloat16 else k.float().double()
    page, slab, octet, i = _at(st, seq, pos)

    def put(x, keys):
        codes, scales = _parts(st["cache"], case, keys)
        c, s = _quantised(x, case["group"])
        codes[page, :, slab, octet, :, i] = c.unflatten(-1, (-1, 16))
        scales[page, :, slab, octet, :, i] = s

    put(k, True)
    put(st["v"].double(), False)
    st["k_out"].copy_(_get(st, seq, pos, True))
    st["v_out"].copy_(_get(st, seq, pos, False))
    return st["q_out"], st["k_out"], st["v_out"]


def _whole(st, keys):
    """The cached values behind the block table: [B, heads, columns * page, d] in fp32."""
    codes, scales = (x[st["block_table"].long()] for x in _parts(st["cache"], st["case"], keys))
    # [B, columns, heads, slabs, octets, chunks, 8, 16] -> [B, heads, columns, slabs, octets, 8, chunks * 16]
    x = _values(codes.permute(0, 2, 1, 3, 4, 6, 5, 7).flatten(-2), scales.permute(0, 2, 1, 3, 4, 6, 5, 7))
    return x.flatten(2, 5)


def _plain_read(st):
    case = st["case"]
    dt = st["k_out"].dtype
    if not case["paged"]:
        seq, _, pos = _token_places(st)
        st["k_out"].copy_(_get(st, seq, pos, True).to(dt))
        st["v_out"].copy_(_get(st, seq, pos, False).to(dt))
        return st["k_out"], st["v_out"]
    page = case["page"]
    lens, cols = st["seq_lens"].long(), st["block_table"].shape[1]
    here = torch.arange(cols * page, device=lens.device)[None, :] < lens[:, None]
    seq, pos = here.nonzero(as_tuple=True)
    to = st["out_table"].long()[seq, pos // page]
    st["k_out"][to, :, pos % page] = _whole(st, True).transpose(1, 2)[seq, pos].to(dt)
    st["v_out"][to, :, pos % page] = _whole(st, False).transpose(1, 2)[seq, pos].to(dt)
    return st["k_out"], st["v_out"]


def _softmax_rows(q, k, v, limit):
    """q [B, H, R, d], k and v [B, H, L, d], limit [B, 1, R]: keys below it are seen. fp32."""
    s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    hidden = torch.arange(k.shape[-2], device=q.device) >= limit[..., None]
    s = s.masked_fill(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)


def _plain_attend(st):
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
    o = _softmax_rows(q, _whole(st, True), _whole(st, False), limit)
    o = o.reshape(batch, hkv, n, group, d).permute(0, 2, 1, 3, 4).reshape(batch, n, hq, d)
    st["out"].copy_(o[seq, i].to(st["out"].dtype))
    return st["out"]


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _kept(st):
    """The library, the shape and the workspaces that a user's program keeps between calls."""
    if "kept" not in st:
        import kv_cache_early_gb300 as K
        shape = K.make_shape(**st["sizes"])
        if st["case"]["op"] == "attend":
            need = [K.dense_extend_kv4_workspace_bytes(shape, st["q"].shape[0], st["case"]["group"])]
        else:
            need = [K.art_append_kv4_workspace_bytes(shape), K.art_read_kv4_workspace_bytes(shape)]
        st["kept"] = K, shape, [torch.empty(n, dtype=torch.uint8, device=st["cache"].device) for n in need]
    return st["kept"]


def run(state):
    st, case = state, state["case"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attend": _plain_attend}[case["op"]](st)
    K, shape, workspaces = _kept(st)
    group = case["group"]
    # a step of one token for each sequence needs no offsets
    offsets = None if st["single"] else st["q_offsets"]
    if case["op"] == "append":
        K.art_append_kv4(st["q"], st["k"], st["v"], st["block_table"], st["seq_lens"], offsets, st["inv_freq"],
                         st["q_out"], st["cache"], shape, workspaces[0], group=group, rot_dim=case["rot"],
                         interleaved=case["interleaved"])
        K.art_read_kv4(st["cache"], st["block_table"], st["seq_lens"], offsets, st["k_out"], st["v_out"], shape,
                       workspaces[1], group=group)
        return st["q_out"], st["k_out"], st["v_out"]
    if case["op"] == "read":
        if case["paged"]:
            K.art_read_kv4(st["cache"], st["block_table"], st["seq_lens"], None, st["k_out"], st["v_out"], shape,
                           workspaces[1], group=group, out_table=st["out_table"])
        else:
            K.art_read_kv4(st["cache"], st["block_table"], st["seq_lens"], offsets, st["k_out"], st["v_out"], shape,
                           workspaces[1], group=group)
        return st["k_out"], st["v_out"]
    K.dense_extend_kv4(st["q"], st["cache"], st["block_table"], st["seq_lens"], offsets, st["out"], shape,
                       workspaces[0], group=group, causal=case["causal"])
    return st["out"]


# ----------------------------------------------------------------------------
# the definitions in 64 bits, from byte addresses, one sequence (and head) at a time
# ----------------------------------------------------------------------------
def _held(st, b, lo, hi, keys):
    """Tokens lo..hi-1 of sequence b as the cache holds them: [hi - lo, heads, d] in fp64."""
    case = st["case"]
    hkv, d, page, group = case["hkv"], case["d"], case["page"], case["group"]
    dev = st["cache"].device
    flat = st["cache"].reshape(-1)
    slab, size = min(page, 64), _page_bytes(case)
    t = torch.arange(lo, hi, device=dev)[:, None, None]
    g = torch.arange(hkv, device=dev)[None, :, None]
    e = torch.arange(d, device=dev)[None, None, :]
    page_id = st["block_table"][b].long()[t // page]
    in_page = t % page
    base = (page_id * hkv + g) * size + in_page // slab * (size // (page // slab))
    u = in_page % slab
    code = base + (0 if keys else slab * d // 2) + ((u // 8 * (d // 32) + e // 32) * 8 + u % 8) * 16 + e % 32 // 2
    code = flat[code].int() >> 4 * (e % 2) & 15
    n = d // group
    pair = base + slab * d + (0 if keys else 4 * slab * n) + ((u // 8 * n + e // group) * 8 + u % 8) * 4
    step, low = ((flat[pair + o].int() + 256 * flat[pair + o + 1].int()).to(torch.int16).view(torch.bfloat16).double()
                 for o in (0, 2))
    return low + step * code


def _near(x, bits):
    """fp64 values rounded to so many bits."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 2.0 ** bits) / 2.0 ** bits, e)


def _stood_for(x, group):
    """What the cache stands for after x [tokens, heads, d] was written: lowest + step * code."""
    y = x.reshape(*x.shape[:-1], -1, group)
    top, bottom = y.max(-1).values, y.min(-1).values
    m, e = torch.frexp(bottom)
    low = torch.ldexp(torch.floor(m * 256.0) / 256.0, e)
    step = _near((top - low) / 15.0, 8)
    step = step * (step >= 2.0 ** -100)
    code = torch.where(step[..., None] > 0, (y - low[..., None]) / step[..., None], torch.zeros_like(y))
    return (low[..., None] + step[..., None] * code.round().clamp(max=15.0)).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    dev = st["cache"].device
    new, seq = _lens(case)
    if case["op"] == "append":
        rot = case["rot"]
        q_out, k_new = st["q"].double().clone(), st["k"].double().clone()
        first = torch.arange(0, rot, 2, device=dev) if case["interleaved"] else torch.arange(rot // 2, device=dev)
        second = first + (1 if case["interleaved"] else rot // 2)
        t0 = 0
        for n, s in zip(new, seq):
            pos = torch.arange(s - n, s, device=dev)
            turn = torch.polar(torch.ones(1, dtype=torch.float64, device=dev),
                               pos.double()[:, None, None] * st["inv_freq"].double())
            for x in (q_out, k_new):
                z = torch.complex(x[t0:t0 + n, :, first], x[t0:t0 + n, :, second]) * turn
                x[t0:t0 + n, :, first], x[t0:t0 + n, :, second] = z.real.clone(), z.imag.clone()
            t0 += n
        k_new = _near(k_new, 8 if case["dtype"] == "bf16" else 24)  # a key is rounded to the cache's type first
        return q_out, _stood_for(k_new, case["group"]), _stood_for(st["v"].double(), case["group"])
    if case["op"] == "read":
        outs = []
        for x, keys in ((st["k_out"], True), (st["v_out"], False)):
            x = x.double()
            t0 = 0
            for b, (n, s) in enumerate(zip(new, seq)):
                for lo in range(s - n, s, 4096):
                    hi = min(lo + 4096, s)
                    rows = _held(st, b, lo, hi, keys)
                    if case["paged"]:
                        t = torch.arange(lo, hi, device=dev)
                        x[st["out_table"][b].long()[t // case["page"]], :, t % case["page"]] = rows
                    else:
                        x[t0 + lo - (s - n):t0 + hi - (s - n)] = rows
                t0 += n
            outs.append(x)
        return tuple(outs)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=dev)
    t0 = 0
    for b, (n, s) in enumerate(zip(new, seq)):
        keys = torch.arange(s, device=dev)
        last = torch.arange(s - n, s, device=dev) if case["causal"] else torch.full((n,), s - 1, device=dev)
        seen = keys[None, :] <= last[:, None]
        k, v = (torch.cat([_held(st, b, lo, min(lo + 4096, s), x) for lo in range(0, s, 4096)]) for x in (True, False))
        for h in range(hkv):
            rows = st["q"][t0:t0 + n, h * g:(h + 1) * g].double()
            a = torch.einsum("ngd,ld->ngl", rows, k[:, h]) * d ** -0.5
            a.masked_fill_(~seen[:, None, :], -math.inf)
            out[t0:t0 + n, h * g:(h + 1) * g] = torch.einsum("ngl,ld->ngd", torch.softmax(a, -1), v[:, h])
        t0 += n
    return out
