"""Cases and plain forms of what surrounds the 4-bit cache in a server that shares prompts.

  norm_rope   queries and keys of new tokens: each head's RMS norm and the
              rotation by the token's position (of one axis, or of several as
              images and video have them), before they are cached and attended
  shared      attention of requests that begin with the same long prefix, over
              the 4-bit cache: the prefix's keys are read once for all of them
  copy        pages of every cache of a model copied to other pages
  step        samples of cached prompts started anew: their pages given back
              (free), the prompts' pages shared with a copy of the last, partly
              filled one (fork), and slots for the next tokens (grow)
  compact     pages in use moved to the front of the caches, tables rewritten

``run`` computes them in elementary torch operations in 32 bits (angles in 64),
or, where ``own`` is true, calls the framework.

Rotation: of a head's first 2 n values, pair i (values i and i + n, or 2 i and
2 i + 1 where pairs are neighbours) turns by position[axis of i] * inv_freq[i].
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases

def _rope(name, tokens, q_heads, k_heads, d, rotary, axes, neighbours, dtype):
    return {"name": name, "op": "rope", "tokens": tokens, "q_heads": q_heads, "k_heads": k_heads, "d": d,
            "rotary": rotary, "axes": axes, "neighbours": neighbours, "dtype": dtype}


def _shared(name, groups, requests, query, prefix_lo, prefix_hi, tail, q_heads, kv_heads, d, block_size, dtype):
    return {"name": name, "op": "shared", "groups": groups, "requests": requests, "query": query,
            "prefix_lo": prefix_lo, "prefix_hi": prefix_hi, "tail": tail, "q_heads": q_heads, "kv_heads": kv_heads,
            "d": d, "block_size": block_size, "dtype": dtype}


def _pages(name, op, blocks, layers, kv_heads, d, block_size, **more):
    return {"name": name, "op": op, "blocks": blocks, "layers": layers, "kv_heads": kv_heads, "d": d,
            "block_size": block_size, **more}


def listed():
    return [
        # the decode workload's step: 32 new tokens, 64 query heads and 8 keys a token
        _rope("rope_decode", 32, 64, 8, 128, 128, 1, False, "f16"),
        # a long prompt's chunk at the end of 131072 positions
        _rope("rope_prompt", 16384, 64, 8, 128, 128, 1, False, "bf16"),
        # patches of a clip: time, height and width, an odd number of them, a small head
        _rope("rope_axes", 4001, 16, 16, 80, 80, 3, False, "f16"),
        # 64 samples of one prompt, each with some tokens of its own
        _shared("shared_decode", 1, 64, 1, 16384, 16384, 2048, 64, 8, 128, 64, "f16"),
        # a decode batch over one document of the longest context
        _shared("shared_long", 1, 32, 1, 131072, 131072, 512, 64, 8, 128, 64, "bf16"),
        # five system prompts of odd lengths, four speculative tokens a request, small heads and pages
        _shared("shared_groups", 5, 23, 4, 300, 5000, 400, 16, 2, 64, 16, "f16"),
        # three partly filled pages copied before they are written to: one layer
        _pages("copy_few", "copy", 256, 1, 8, 128, 64, pairs=3),
        # a quarter of the pages of four layers to other places
        _pages("copy_many", "copy", 2048, 4, 8, 128, 64, pairs=512),
        # four samples of one short prompt
        _pages("step_few", "step", 400, 1, 8, 128, 16, parents=1, children=4, lo=1000, hi=1000, new=1),
        # 64 samples of four long prompts, with four speculative tokens each
        _pages("step_many", "step", 2560, 4, 8, 128, 64, parents=4, children=64, lo=30000, hi=32768, new=4),
        # a small pool after some requests ended
        _pages("compact_few", "compact", 200, 1, 2, 64, 16, live=0.5, rows=6),
        # a large pool of two layers with two of five pages in use
        _pages("compact_many", "compact", 4096, 2, 8, 128, 64, live=0.4, rows=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges the listed ones stand for."""
    op = rng.choice(["rope", "rope", "shared", "shared", "copy", "step", "compact"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "rope":
        d = rng.choice([32, 64, 72, 80, 96, 128, 192, 256])
        rotary = rng.choice([d, d, d // 2 // 8 * 8, 16])
        heads = rng.choice([1, 2, 4, 8, 16])
        c = _rope("", _log(rng, 1, 8000), heads * rng.choice([1, 2, 4]), heads, d, rotary, rng.choice([1, 1, 2, 3, 4]),
                  rng.choice([False, True]), dtype)
    elif op == "shared":
        groups = rng.choice([1, 1, 2, 3, 5])
        kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 7, 8, 16])
        hi = _log(rng, 40, 16384)
        query = rng.choice([1, 1, 1, 2, 4, _log(rng, 5, 64)])
        requests = _log(rng, groups, 64 if query == 1 else 24 if query <= 4 else max(groups, 6))
        c = _shared("", groups, requests, query, _log(rng, 20, hi) if hi > 20 else hi, hi, _log(rng, query, 1024),
                    kv * group, kv, rng.choice([64, 96, 128, 192, 256]), rng.choice([16, 32, 64, 100]), dtype)
    else:
        bs = rng.choice([16, 32, 64, 100])
        kv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 256])
        layers = rng.choice([1, 2, 3])
        if op == "copy":
            blocks = _log(rng, 20, 800)
            c = _pages("", "copy", blocks, layers, kv, d, bs, pairs=_log(rng, 1, blocks // 2))
        elif op == "step":
            parents, children = rng.choice([1, 2, 3, 5]), _log(rng, 1, 48)
            hi = _log(rng, 20, 8000)
            lo = _log(rng, 10, hi)
            new = rng.choice([1, 1, 4, _log(rng, 2, 200)])
            blocks = parents * -(-hi // bs) + 2 * children * (2 + -(-new // bs)) + rng.randrange(1, 50)
            c = _pages("", "step", blocks, layers, kv, d, bs, parents=parents, children=children, lo=lo, hi=hi, new=new)
        else:
            c = _pages("", "compact", _log(rng, 10, 1000), layers, kv, d, bs, live=rng.choice([0.1, 0.4, 0.7, 0.95]),
                       rows=_log(rng, 1, 64))
    return {k: v for k, v in c.items() if k != "name"}


def _page_bytes(case):
    """Bytes of one page in all caches: K and V in 4 bits with their scales, and the indexer's 16-bit keys."""
    bs, kv, d = case["block_size"], case["kv_heads"], case["d"]
    return case["layers"] * bs * (2 * kv * (d // 2 + d // 32) + 2 * d)


def work(case):
    """Inputs read once, outputs written once, two operations per product and sum."""
    if case["op"] == "rope":
        values = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["d"]
        return {"bytes": 4 * values + 8 * case["tokens"] * case["axes"], "flops": 8.0 * values}
    bs = case["block_size"]
    if case["op"] == "shared":
        row = case["kv_heads"] * (case["d"] // 2 + case["d"] // 32)
        rows = case["requests"] * case["query"]
        prefix = 0.5 * (case["prefix_lo"] + case["prefix_hi"])
        tail = 0.5 * (case["query"] + case["tail"])
        keys = case["groups"] * prefix + case["requests"] * tail
        seen = prefix + tail - 0.5 * (case["query"] - 1)
        return {"bytes": keys * 2 * row + rows * case["q_heads"] * (case["d"] * 4 + 4) + 4 * keys / bs,
                "flops": 4.0 * rows * seen * case["q_heads"] * case["d"]}
    page = _page_bytes(case)
    if case["op"] == "copy":
        return {"bytes": case["pairs"] * (2 * page + 16), "flops": 0}
    if case["op"] == "step":
        pages = 0.5 * (case["lo"] + case["hi"]) / bs
        partial = case["children"] * (bs - 1) / bs   # a length that is a multiple of the page leaves none to copy
        # the tables' rows read, written as none and then anew, the counts read and written, the slots
        return {"bytes": partial * 2 * page + case["children"] * (12 * pages + 8 * case["new"]) + 8 * case["blocks"],
                "flops": 0}
    live = case["live"] * case["blocks"]
    moved = live * (1.0 - case["live"])
    return {"bytes": moved * 2 * page + 12 * case["blocks"] + 8 * live, "flops": 0}


# ------------------------------------------------------- the plain forms

def _plain_rope(s):
    pos = s["positions"].double()
    n = s["inv_freq"].numel()
    if pos.dim() == 1:
        angle = pos[:, None] * s["inv_freq"].double()
    else:
        angle = pos[s["axis_index"]].t() * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s[name + "_weight"]
        if s["neighbours"]:
            a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = x[..., :n], x[..., n:2 * n]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        out[name] = torch.cat((turned, x[..., 2 * n:]), -1).to(s[name].dtype)
    return out


def _dequantise(data, scale):
    """The f32 values of packed bytes [..., d/2] under scale bytes [..., d/32]."""
    code = torch.stack((data & 15, data >> 4), -1).flatten(-2)
    m = (code & 7).float()
    a = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, 2 * m - 8))
    a = torch.where(code >= 8, -a, a).unflatten(-1, (-1, 32))
    s = scale.int() - 127
    return torch.ldexp(torch.ldexp(a, (s // 2)[..., None]), (s - s // 2)[..., None]).flatten(-2)


def _plain_shared(s):
    rows, H, d = s["q"].shape
    Q, bs, kv = s["query"], s["block_size"], s["kv_heads"]
    g = H // kv
    out, lse = torch.empty_like(s["q"]), torch.empty((rows, H), device=DEV)
    vis = (s["seq_lens"].long()[:, None] - Q + 1 + torch.arange(Q, device=DEV)).view(-1)
    for f, to, prefix in s["host_groups"]:
        c = to - f
        table = s["block_table"][f:to].long()
        seen = vis[f * Q:to * Q].view(c, 1, Q, 1, 1)
        q = s["q"][f * Q:to * Q].float().view(c, Q, kv, g, d)
        at = torch.arange(prefix, device=DEV)
        slots = table[0, at // bs] * bs + at % bs
        # the prefix: [kv, c * Q * g, prefix]
        k = _dequantise(s["k_data"].flatten(0, 1)[slots], s["k_scale"].flatten(0, 1)[slots]).permute(1, 2, 0)
        first = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(kv, c * Q * g, d), k.contiguous())
        first = first.view(kv, c, Q, g, prefix).transpose(0, 1).masked_fill(at >= seen, -math.inf)
        # each request's own keys: [c, kv, Q * g, tail]
        at = prefix + torch.arange(s["max_seq_len"] - prefix, device=DEV)
        page = table.gather(1, (at // bs).expand(c, -1)).clamp(min=0)
        slots = page * bs + at % bs
        k = _dequantise(s["k_data"].flatten(0, 1)[slots], s["k_scale"].flatten(0, 1)[slots]).permute(0, 2, 3, 1)
        own_scores = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(c, kv, Q * g, d), k.contiguous())
        own_scores = own_scores.view(c, kv, Q, g, -1).masked_fill(at >= seen, -math.inf)
        z = torch.cat((first, own_scores), -1) * s["sm_scale"]
        del first, own_scores, k
        top = z.amax(-1, keepdim=True)
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        p = torch.exp(z - top)
        total = p.sum(-1, keepdim=True)
        del z
        v = _dequantise(s["v_data"].flatten(0, 1)[slots], s["v_scale"].flatten(0, 1)[slots]).transpose(1, 2)
        r = torch.matmul(p[..., prefix:].reshape(c, kv, Q * g, -1), v.contiguous()).view(c, kv, Q, g, d)
        at = torch.arange(prefix, device=DEV)
        slots = table[0, at // bs] * bs + at % bs
        v = _dequantise(s["v_data"].flatten(0, 1)[slots], s["v_scale"].flatten(0, 1)[slots]).transpose(0, 1)
        r = r + torch.matmul(p[..., :prefix].transpose(0, 1).reshape(kv, c * Q * g, prefix),
                             v.contiguous()).view(kv, c, Q, g, d).transpose(0, 1)
        r = r / torch.where(total > 0, total, torch.ones_like(total))
        out[f * Q:to * Q] = r.transpose(1, 2).reshape(c * Q, H, d).to(out.dtype)
        lse[f * Q:to * Q] = (torch.log(total) + top).squeeze(-1).transpose(1, 2).reshape(c * Q, H)
    return {"out": out, "lse": lse}


def _free_order(refs):
    """The pages nobody holds, lowest first (the others behind them), and how many there are."""
    used = refs > 0
    return torch.argsort(used.int(), stable=True), (~used).sum()


def _plain_step(s):
    table, lens, refs, bs = s["block_table"], s["seq_lens"], s["refs"], s["block_size"]
    parents, children = s["parents"].long(), s["children"].long()
    cols = torch.arange(table.shape[1], device=DEV)
    # free
    held = table[children].long()
    refs.index_add_(0, held.clamp(min=0).flatten(), -(held >= 0).int().flatten())
    # fork
    order, n_free = _free_order(refs)
    length = lens[parents].long()
    full, partial = length // bs, length % bs > 0
    rank = partial.cumsum(0) - 1
    ok = ~partial | (rank < n_free)
    page = order[rank.clamp(0, refs.numel() - 1)]
    fresh = torch.where(partial, torch.where(ok, page, torch.full_like(page, -2)), torch.full_like(page, -1))
    theirs = table[parents].long()
    row = torch.where((cols < full[:, None]) & ok[:, None], theirs, torch.full_like(theirs, -1))
    refs.index_add_(0, row.clamp(min=0).flatten(), (row >= 0).int().flatten())
    took = fresh >= 0
    refs.index_add_(0, fresh.clamp(min=0), took.int())
    row = torch.where((cols == full[:, None]) & took[:, None], fresh[:, None], row)
    table[children] = row.int()
    grown = torch.where(ok, length, torch.zeros_like(length))
    last = theirs.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    source = torch.where(took, last, theirs[:, 0])      # a page onto itself where there is none to copy
    target = torch.where(took, fresh, theirs[:, 0])
    for t in s["caches"]:
        t[target] = t[source]
    # grow
    new = s["new"]
    order, n_free = _free_order(refs)
    have, want = -(-grown // bs), -(-(grown + new) // bs)
    fits = want <= table.shape[1]
    need = torch.where(fits, want - have, torch.zeros_like(want))
    upto = need.cumsum(0)
    fits = fits & ((need == 0) | (upto <= n_free))
    k = cols[None, :] - have[:, None]
    mine = (k >= 0) & (k < need[:, None]) & fits[:, None]
    page = order[(upto[:, None] - need[:, None] + k).clamp(0, refs.numel() - 1)]
    row = torch.where(mine, page, table[children].long())
    refs.index_add_(0, page.flatten(), mine.int().flatten())
    table[children] = row.int()
    at = grown[:, None] + torch.arange(new, device=DEV)
    slots = row.gather(1, (at // bs).clamp(max=table.shape[1] - 1)) * bs + at % bs
    slots = torch.where(fits[:, None], slots, torch.full_like(slots, -1))
    lens[children] = (grown + torch.where(fits, new, 0)).int()
    return {"block_table": table, "seq_lens": lens, "refs": refs, "fresh": fresh.int(), "slots": slots,
            "caches": s["caches"]}


def _plain_compact(s):
    refs, n = s["refs"], s["refs"].numel()
    at = torch.arange(n, device=DEV)
    live = refs > 0
    count = live.sum()
    holes, late = ~live & (at < count), live & (at >= count)
    most = n // 2
    moves = torch.arange(most, device=DEV)
    # the i-th hole takes the i-th late page; beyond them the last page stays where it is
    hole_order, late_order = torch.argsort((~holes).int(), stable=True), torch.argsort((~late).int(), stable=True)
    valid = moves < late.sum()
    target = torch.where(valid, hole_order[:most], torch.full_like(moves, n - 1))
    source = torch.where(valid, late_order[:most], torch.full_like(moves, n - 1))
    place = torch.where(live, at, torch.full_like(at, -1))
    place = torch.where(late, hole_order[(late.cumsum(0) - 1).clamp(min=0)], place)
    for t in s["caches"]:
        t[target] = t[source]
    taken = holes & (holes.cumsum(0) <= late.sum())
    counts = torch.where(live & (at < count), refs, torch.zeros_like(refs))
    counts = torch.where(taken, refs[late_order[(holes.cumsum(0) - 1).clamp(min=0)]], counts)
    table = s["block_table"].long()
    table = torch.where(table >= 0, place[table.clamp(min=0)], torch.full_like(table, -1))
    return {"block_table": table.int(), "refs": counts, "place": place.int(), "live": count.view(1).int(),
            "caches": s["caches"]}


def _plain(s):
    if s["op"] == "rope":
        return _plain_rope(s)
    if s["op"] == "shared":
        return _plain_shared(s)
    if s["op"] == "copy":
        for t in s["caches"]:
            t[s["to"].long()] = t[s["from"].long()]
        return {"caches": s["caches"]}
    return _plain_step(s) if s["op"] == "step" else _plain_compact(s)


# --------------------------------------------------------------- the calls

def _call(s):
    import sparse_attention_lightning_indexer_amd as li
    if s["op"] == "rope":
        q, k = li.norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"], eps=s["eps"],
                            axes=s["axis_of"], interleaved=s["neighbours"])
        return {"q": q, "k": k}
    if s["op"] == "shared":
        out, lse = li.mx4_attend_shared(s["q"], s["k_data"], s["k_scale"], s["v_data"], s["v_scale"], s["block_table"],
                                        s["seq_lens"], s["query"], s["max_seq_len"], s["sm_scale"], s["prefix_lens"],
                                        s["max_prefix_len"], s["group_starts"], s["max_group"])
        return {"out": out, "lse": lse}
    if s["op"] == "copy":
        li.pages_copy(s["pages"], s["from"], s["to"])
        return {"caches": s["caches"]}
    if s["op"] == "step":
        li.pages_free(s["refs"], s["block_table"], s["seq_lens"], s["children"])
        fresh = li.pages_fork(s["pages"], s["refs"], s["block_table"], s["seq_lens"], s["parents"], s["children"],
                              s["block_size"])
        slots = li.pages_grow(s["refs"], s["block_table"], s["seq_lens"], s["children"], s["new"], s["block_size"])
        return {"block_table": s["block_table"], "seq_lens": s["seq_lens"], "refs": s["refs"], "fresh": fresh,
                "slots": slots, "caches": s["caches"]}
    refs, table = s["refs"].clone(), s["block_table"].clone()
    place, live = li.pages_compact(s["pages"], refs, table)
    return {"block_table": table, "refs": refs, "place": place, "live": live, "caches": s["caches"]}


def run(state):
    return _call(state) if own else _plain(state)


# -------------------------------------------------------------- the inputs

def _normal(gen, shape, dtype):
    """Unit-normal rows whose channels have spread magnitudes (a few large ones), as projected rows do."""
    gain = torch.exp(0.5 * torch.randn(shape[-1], generator=gen, device=DEV))
    x = torch.empty(shape, dtype=TYPES[dtype], device=DEV)
    for part in x.view(-1, shape[-1]).split(1 << 20):   # bounded scratch
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV) * gain)
    return x


def _bytes(gen, shape, lo=0, hi=256):
    return torch.randint(lo, hi, shape, generator=gen, device=DEV, dtype=torch.uint8)


def _cache(gen, case, blocks):
    """One of K and V in 4 bits: codes as unit-normal rows leave them, scales around 2^-2."""
    shape = (blocks, case["block_size"], case["kv_heads"])
    d = case["d"]
    # magnitudes of normal values under their block's scale: the middle codes most
    pair = torch.tensor([0, 1, 1, 2, 2, 3, 3, 4, 4, 5, 5, 6, 8, 9, 9, 10, 10, 11, 11, 12, 12, 13, 13, 14, 7, 15],
                        dtype=torch.uint8, device=DEV)
    data = torch.empty(shape + (d // 2,), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (case["block_size"] * case["kv_heads"] * d))
    for a in range(0, blocks, step):
        part = data[a:a + step]
        code = pair[torch.randint(0, pair.numel(), part.shape + (2,), generator=gen, device=DEV)]
        part.copy_(code[..., 0] + 16 * code[..., 1])
    return data, _bytes(gen, shape + (d // 32,), 124, 127)


def _prepare_rope(s, gen, case):
    n, d, axes = case["tokens"], case["d"], case["axes"]
    for name in ("q", "k"):
        s[name] = _normal(gen, (n, case[name + "_heads"], d), case["dtype"])
        s[name + "_weight"] = 1.0 + 0.2 * torch.randn(d, generator=gen, device=DEV)
    s["eps"] = 1e-6
    half = case["rotary"] // 2
    s["axis_of"], s["axis_index"] = None, None
    if axes == 1:
        at = torch.arange(n, device=DEV)
        last = torch.randint(1024, 131072, (1,), generator=gen, device=DEV)
        s["positions"] = at + last if n > 64 else torch.randint(1023, 8192, (n,), generator=gen, device=DEV)
        s["inv_freq"] = torch.pow(10000.0, -torch.arange(half, device=DEV).double() / half).float()
    else:
        # a grid of patches, its innermost axes 40 wide, after some tokens of text
        at = torch.arange(n, device=DEV)
        place = [at // 1600, at // 40 % 40, at % 40, at % 7][:axes]
        start = torch.randint(0, 4000, (1,), generator=gen, device=DEV)
        s["positions"] = torch.stack([p + start for p in place]).contiguous()
        s["axis_of"] = tuple(i * axes // half for i in range(half))
        s["axis_index"] = torch.tensor(s["axis_of"], device=DEV)
        s["inv_freq"] = torch.pow(10000.0, -torch.arange(half, device=DEV).double() / half).float()


def _prepare_shared(s, gen, case):
    R, G, Q, bs = case["requests"], case["groups"], case["query"], case["block_size"]
    d = case["d"]
    # sizes are the program's own knowledge: drawn on the host, by the device generator's state alone
    cut = torch.rand(R - 1, generator=gen, device=DEV).argsort()[:G - 1].sort().values + 1 if R > 1 else None
    starts = [0] + (cut.tolist() if cut is not None else []) + [R]
    prefix = torch.randint(case["prefix_lo"], case["prefix_hi"] + 1, (G,), generator=gen, device=DEV).tolist()
    tails = torch.randint(Q, max(Q, case["tail"]) + 1, (R,), generator=gen, device=DEV).tolist()
    lens = [prefix[g] + tails[r] for g in range(G) for r in range(starts[g], starts[g + 1])]
    s["host_groups"] = [(starts[g], starts[g + 1], prefix[g]) for g in range(G)]
    s["max_group"] = max(to - f for f, to, _ in s["host_groups"])
    s["max_prefix_len"], s["max_seq_len"] = max(prefix), max(lens)
    cols = -(-max(lens) // bs)
    blocks = sum(-(-p // bs) for p in prefix) + sum(2 + -(-t // bs) for t in tails) + 3
    order = torch.randperm(blocks, generator=gen, device=DEV).tolist()
    table = torch.full((R, cols), -1, dtype=torch.int32)
    for f, to, p in s["host_groups"]:
        full, pages = p // bs, [order.pop() for _ in range(p // bs)]
        for r in range(f, to):      # whole pages of the prefix are shared, the rest is each request's own
            have = pages + [order.pop() for _ in range(-(-lens[r] // bs) - full)]
            table[r, :len(have)] = torch.tensor(have, dtype=torch.int32)
    s["block_table"] = table.to(DEV)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32, device=DEV)
    s["group_starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["k_data"], s["k_scale"] = _cache(gen, case, blocks)
    s["v_data"], s["v_scale"] = _cache(gen, case, blocks)
    for f, to, p in s["host_groups"]:                 # the prefix's end lies in a page of each request: copies of one
        if p % bs:
            own_pages = s["block_table"][f:to, p // bs].long()
            for name in ("k_data", "k_scale", "v_data", "v_scale"):
                s[name][own_pages, :p % bs] = s[name][own_pages[:1], :p % bs]
    s["q"] = torch.randn((R * Q, case["q_heads"], d), generator=gen, device=DEV).to(TYPES[case["dtype"]])
    s["sm_scale"] = 1.0 / math.sqrt(d)


def _prepare_pages(s, gen, case):
    n, bs = case["blocks"], case["block_size"]
    caches = []
    for _ in range(case["layers"]):
        for _ in ("k", "v"):
            shape = (n, bs, case["kv_heads"])
            caches += [_bytes(gen, shape + (case["d"] // 2,)), _bytes(gen, shape + (case["d"] // 32,), 110, 130)]
        caches.append(torch.randn((n, bs, case["d"]), generator=gen, device=DEV, dtype=torch.float16))
    s["caches"] = s["pages"] = caches
    order = torch.randperm(n, generator=gen, device=DEV)
    if case["op"] == "copy":
        s["from"], s["to"] = order[:case["pairs"]].int(), order[case["pairs"]:2 * case["pairs"]].int()
    elif case["op"] == "step":
        parents, children = case["parents"], case["children"]
        rows = parents + children
        lens = torch.randint(case["lo"], case["hi"] + 1, (rows,), generator=gen, device=DEV).tolist()
        cols = -(-(case["hi"] + case["new"]) // bs)
        table = torch.full((rows, cols), -1, dtype=torch.int32)
        spare = order.tolist()
        for r in range(parents):
            have = [spare.pop() for _ in range(-(-lens[r] // bs))]
            table[r, :len(have)] = torch.tensor(have, dtype=torch.int32)
        for c in range(children):           # what ended: samples that shared a prompt and had some pages of their own
            r, p = parents + c, c % parents
            full = lens[p] // bs
            table[r, :full] = table[p, :full]
            extra = min(cols - full, 1 + c % 2)
            table[r, full:full + extra] = torch.tensor([spare.pop() for _ in range(extra)], dtype=torch.int32)
            lens[r] = min(lens[p] + c % bs, (full + extra) * bs)
        s["refs"] = torch.bincount(table[table >= 0].long(), minlength=n).int().to(DEV)
        s["block_table"] = table.to(DEV)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        # the new samples: of the prompts in any order
        pick = torch.randint(0, parents, (children,), generator=gen, device=DEV)
        s["parents"] = pick.int()
        s["children"] = (parents + torch.randperm(children, generator=gen, device=DEV)).int()
    else:
        live = max(1, int(case["live"] * n))
        rows = case["rows"]
        pages = order[:live]
        # the pages in use, shared out to the rows, the first ones held by all of them
        common = pages[:min(live, 3)]
        per = -(-(live - common.numel()) // rows)
        table = torch.full((rows, common.numel() + per + 2), -1, dtype=torch.int32, device=DEV)
        table[:, :common.numel()] = common.int()
        for r in range(rows):
            mine = pages[common.numel() + r * per:common.numel() + (r + 1) * per]
            table[r, common.numel():common.numel() + mine.numel()] = mine.int()
        s["block_table"] = table
        s["refs"] = torch.bincount(table[table >= 0].long(), minlength=n).int()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "rope":
        _prepare_rope(s, gen, case)
    elif case["op"] == "shared":
        _prepare_shared(s, gen, case)
    else:
        _prepare_pages(s, gen, case)
        if own:     # a server checks and lists a model's caches once
            import sparse_attention_lightning_indexer_amd as li
            s["pages"] = li.PageSet(s["caches"])
    return s


# ----------------------------------- the definitions in 64 bits, or one by one

_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_rows(data, scale):
    """f64 values of cache rows [n, heads, d/2], by table."""
    table = torch.tensor([v for v in _MAGNITUDES] + [-v for v in _MAGNITUDES], dtype=torch.float64, device=data.device)
    pair = torch.stack([table[(data % 16).long()], table[torch.div(data, 16, rounding_mode="floor").long()]], -1)
    factor = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=data.device), scale.double() - 127)
    return (pair.reshape(data.shape[:-1] + (-1, 32)) * factor[..., None]).reshape(data.shape[:-1] + (-1,))


def _exact_rope(s):
    """As complex numbers: a pair times e^(i angle)."""
    n = s["inv_freq"].numel()
    out = {}
    for name in ("q", "k"):
        x, weight = s[name], s[name + "_weight"].double()
        to = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        for a in range(0, x.shape[0], 2048):
            v = x[a:a + 2048].double()
            v = v * weight / torch.sqrt(torch.sum(v ** 2, -1, keepdim=True) / x.shape[-1] + s["eps"])
            angle = torch.zeros((v.shape[0], n), dtype=torch.float64, device=x.device)
            for i in range(n):
                p = s["positions"] if s["axis_of"] is None else s["positions"][s["axis_of"][i]]
                angle[:, i] = p[a:a + 2048].double() * s["inv_freq"][i].double()
            turn = torch.polar(torch.ones_like(angle), angle)[:, None]
            first = torch.arange(n, device=x.device) * 2 if s["neighbours"] else torch.arange(n, device=x.device)
            second = first + (1 if s["neighbours"] else n)
            z = torch.complex(v[..., first].contiguous(), v[..., second].contiguous()) * turn
            v[..., first], v[..., second] = z.real, z.imag
            to[a:a + 2048] = v
        out[name] = to
    return out


def _exact_shared(s):
    rows, H, d = s["q"].shape
    kv, Q, bs = s["kv_heads"], s["query"], s["block_size"]
    out = torch.zeros((rows, H, d), dtype=torch.float64, device=DEV)
    lse = torch.full((rows, H), -math.inf, dtype=torch.float64, device=DEV)
    lens, tables = s["seq_lens"].tolist(), s["block_table"].long()

    def keys(name, row, lo, hi):
        at = torch.arange(lo, hi, device=DEV)
        slots = tables[row, at // bs] * bs + at % bs
        return _exact_rows(s[name + "_data"].flatten(0, 1)[slots], s[name + "_scale"].flatten(0, 1)[slots])

    for f, to, prefix in s["host_groups"]:
        before = {n: keys(n, f, 0, prefix) for n in ("k", "v")}
        for r in range(f, to):
            k, v = (torch.cat([before[n], keys(n, r, prefix, lens[r])]).transpose(0, 1).contiguous()
                    for n in ("k", "v"))
            for j in range(Q):
                t, seen = r * Q + j, lens[r] - Q + 1 + j
                z = torch.matmul(k[:, :seen], s["q"][t].double().view(kv, H // kv, d).transpose(1, 2).contiguous())
                z = z.transpose(1, 2) * s["sm_scale"]
                lse[t] = torch.logsumexp(z, -1).view(H)
                out[t] = torch.matmul(torch.exp(z - lse[t].view(kv, -1, 1)), v[:, :seen]).view(H, d)
    return {"out": out, "lse": lse}


def _exact_step(s):
    """One row after the other, on lists."""
    bs, n = s["block_size"], s["blocks"]
    table, lens, refs = s["block_table"].tolist(), s["seq_lens"].tolist(), s["refs"].tolist()
    children = s["children"].tolist()
    for c in children:
        for p in table[c]:
            if p >= 0:
                refs[p] -= 1
        table[c], lens[c] = [-1] * len(table[c]), 0
    fresh, copies, spare = [], [], [p for p in range(n) if refs[p] <= 0]
    for c, parent in zip(children, s["parents"].tolist()):
        full, rest = divmod(lens[parent], bs)
        if rest and not spare:
            fresh.append(-2)
            continue
        table[c][:full] = table[parent][:full]
        for p in table[c][:full]:
            refs[p] += 1
        lens[c] = lens[parent]
        if rest:
            p = spare.pop(0)
            refs[p] = 1
            table[c][full] = p
            copies.append((table[parent][full], p))
        fresh.append(p if rest else -1)
    slots, spare = [], [p for p in range(n) if refs[p] <= 0]
    for c in children:
        have, want = -(-lens[c] // bs), -(-(lens[c] + s["new"]) // bs)
        if want > len(table[c]) or want - have > len(spare):
            slots.append([-1] * s["new"])
            spare = spare[:0] if want <= len(table[c]) else spare    # later rows find no page either
            continue
        for i in range(have, want):
            table[c][i] = spare.pop(0)
            refs[table[c][i]] = 1
        slots.append([table[c][p // bs] * bs + p % bs for p in range(lens[c], lens[c] + s["new"])])
        lens[c] += s["new"]
    caches = [t.clone() for t in s["caches"]]
    for a, b in copies:
        for t in caches:
            t[b].copy_(t[a])
    return {"block_table": torch.tensor(table, dtype=torch.int32), "seq_lens": torch.tensor(lens, dtype=torch.int32),
            "refs": torch.tensor(refs, dtype=torch.int32), "fresh": torch.tensor(fresh, dtype=torch.int32),
            "slots": torch.tensor(slots, dtype=torch.int64), "caches": caches}


def _exact_compact(s):
    refs, n = s["refs"].tolist(), s["blocks"]
    count = sum(r > 0 for r in refs)
    holes = [p for p in range(count) if refs[p] <= 0]
    late = [p for p in range(count, n) if refs[p] > 0]
    place = [p if refs[p] > 0 else -1 for p in range(n)]
    caches, counts = [t.clone() for t in s["caches"]], [r if p < count else 0 for p, r in enumerate(refs)]
    for a, b in zip(late, holes):
        place[a], counts[b] = b, refs[a]
        for t in caches:
            t[b].copy_(t[a])
    table = [[place[p] if p >= 0 else -1 for p in row] for row in s["block_table"].tolist()]
    return {"block_table": torch.tensor(table, dtype=torch.int32), "refs": torch.tensor(counts, dtype=torch.int32),
            "place": torch.tensor(place, dtype=torch.int32), "live": torch.tensor([count], dtype=torch.int32),
            "caches": caches}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if case["op"] == "shared":
        return _exact_shared(s)
    if case["op"] == "copy":
        caches = [t.clone() for t in s["caches"]]
        for a, b in zip(s["from"].tolist(), s["to"].tolist()):
            for t in caches:
                t[b].copy_(t[a])
        return {"caches": caches}
    return _exact_step(s) if case["op"] == "step" else _exact_compact(s)
