"""Cases and plain forms of the 4-bit (MXFP4) key/value cache and the attention over it.

The operators are what a server does around the indexer's selection: write a
step's or a prompt's keys and values into the paged cache in 4 bits, read rows
back, and attend either to the keys the top-k selected or to a sliding window
with a few first tokens.  ``run`` computes them in elementary torch operations
in 32 bits, or, where ``own`` is true, calls the framework.

Cache format: blocks of 32 values along the head dimension share a byte s
(a factor 2^(s - 127)) and hold a 4-bit float each (sign, magnitude one of 0,
.5, 1, 1.5, 2, 3, 4, 6; the even dimension in the low half of a byte).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
# the scale exponents a source type uses: those whose every 4-bit value the type holds
RANGE = {"f16": (-23, 13), "bf16": (-126, 125)}


# ------------------------------------------------------------------- cases

def _write(name, tokens, heads, d, block_size, dtype):
    return {"name": name, "op": "write", "tokens": tokens, "kv_heads": heads, "d": d, "block_size": block_size,
            "dtype": dtype}


def _read(name, rows, cached, heads, d, block_size, dtype):
    return {"name": name, "op": "read", "rows": rows, "cached": cached, "kv_heads": heads, "d": d,
            "block_size": block_size, "dtype": dtype}


def _selected(name, requests, query, lo, hi, k, pool, q_heads, kv_heads, d, block_size, dtype):
    return {"name": name, "op": "selected", "requests": requests, "query": query, "len_lo": lo, "len_hi": hi, "k": k,
            "pool": pool, "q_heads": q_heads, "kv_heads": kv_heads, "d": d, "block_size": block_size, "dtype": dtype}


def _window(name, requests, query, lo, hi, window, sinks, q_heads, kv_heads, d, block_size, dtype):
    return {"name": name, "op": "window", "requests": requests, "query": query, "len_lo": lo, "len_hi": hi,
            "window": window, "sinks": sinks, "q_heads": q_heads, "kv_heads": kv_heads, "d": d,
            "block_size": block_size, "dtype": dtype}


def listed():
    return [
        # a decode step's new tokens: one per request, written and read back
        _write("write_step", 32, 8, 128, 64, "f16"),
        # the prompt of the long-context workload, all of it
        _write("write_prompt", 131072, 8, 128, 64, "bf16"),
        # a reused prefix of odd length read back for another consumer
        _read("read_prefix", 777, 8192, 2, 64, 16, "f16"),
        # one request's whole cache of a speculative-decode length, read back
        _read("read_cache", 131072, 131072, 8, 128, 64, "bf16"),
        # the decode workload: 32 requests, one token each, its top-512
        _selected("selected_decode", 32, 1, 1024, 8192, 512, 1, 64, 8, 128, 64, "f16"),
        # the speculative workload: four tokens a request over 16384 keys, top-2048
        _selected("selected_spec", 32, 4, 16384, 16384, 2048, 1, 64, 8, 128, 64, "bf16"),
        # the long-context chunk: 1024 prompt tokens, each with its own 2048 of up to 131072 keys
        _selected("selected_chunk", 1, 1024, 131072, 131072, 2048, 1, 64, 8, 128, 64, "f16"),
        # pooled keys: each selected entry stands for 32 raw keys; one shared K/V head, short odd lengths
        _selected("selected_blocks", 7, 1, 97, 5001, 48, 32, 16, 1, 256, 16, "bf16"),
        # one request decoding at the longest context with everything visible
        _window("full_decode", 1, 1, 131072, 131072, 0, 0, 64, 8, 128, 64, "bf16"),
        # the decode batch with a window and four first tokens
        _window("window_decode", 32, 1, 1024, 8192, 1024, 4, 64, 8, 128, 64, "f16"),
        # a chunk of prompt under a window with first tokens, odd lengths
        _window("window_chunk", 1, 1000, 16321, 16321, 4096, 64, 64, 8, 128, 64, "bf16"),
        # a chunk of prompt with everything visible
        _window("full_chunk", 1, 1024, 16384, 16384, 0, 0, 64, 8, 128, 64, "f16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges the listed ones stand for."""
    op = rng.choice(["write", "read", "selected", "selected", "window", "window"])
    d = rng.choice([64, 96, 128, 192, 256])
    kv = rng.choice([1, 2, 4, 8])
    bs = rng.choice([16, 32, 64, 100])
    dtype = rng.choice(["f16", "bf16"])
    if op == "write":
        return {k: v for k, v in _write("", _log(rng, 1, 60000), kv, d, bs, dtype).items() if k != "name"}
    if op == "read":
        cached = _log(rng, 64, 60000)
        return {k: v for k, v in _read("", _log(rng, 1, cached), cached, kv, d, bs, dtype).items() if k != "name"}
    group = rng.choice([1, 3, 4, 7, 8, 16])
    hi = _log(rng, 40, 16384)
    lo = _log(rng, 20, hi) if hi > 20 else hi
    requests = _log(rng, 1, 32)
    query = rng.choice([1, 1, 2, 4, _log(rng, 5, 100)])
    if query > 4:
        requests = min(requests, 2)
    if op == "selected":
        pool = rng.choice([1, 1, 1, 16, 32])
        k = _log(rng, 1, 2048) if pool == 1 else _log(rng, 1, 2048 // pool)
        c = _selected("", requests, query, lo, hi, k, pool, kv * group, kv, d, bs, dtype)
    else:
        window, sinks = rng.choice([(0, 0), (_log(rng, 16, 4096), rng.choice([0, 1, 4, 64]))])
        c = _window("", requests, query, lo, hi, window, sinks, kv * group, kv, d, bs, dtype)
    return {k: v for k, v in c.items() if k != "name"}


def _mean_visible(case):
    """Keys a row attends to, on average over the lengths a case draws."""
    mean = 0.5 * (case["len_lo"] + case["len_hi"]) - 0.5 * (case["query"] - 1)
    if case["op"] == "selected":
        return min(mean, case["k"] * case["pool"])
    if case["window"]:
        return min(mean, case["window"] + case["sinks"])
    return mean


def work(case):
    """Inputs read once, outputs written once, two operations per product and sum."""
    row = case["kv_heads"] * (case["d"] // 2 + case["d"] // 32)      # bytes of one token in one cache
    elem = case["kv_heads"] * case["d"] * 2
    if case["op"] == "write":  # both tensors in, both caches written, both read back
        n = case["tokens"]
        return {"bytes": n * (2 * elem + 2 * row + 2 * elem + 8), "flops": 0}
    if case["op"] == "read":
        return {"bytes": case["rows"] * (row + elem + 8), "flops": 0}
    rows = case["requests"] * case["query"]
    vis = _mean_visible(case)
    length = 0.5 * (case["len_lo"] + case["len_hi"])
    if case["op"] == "selected":
        keys = case["requests"] * min(length, case["query"] * vis)
        extra = 4 * rows * case["k"]
    else:
        keys = case["requests"] * (min(length, vis + case["query"] - 1) if case["window"] else length)
        extra = 0
    pages = 4 * case["requests"] * math.ceil(length / case["block_size"])
    return {"bytes": keys * 2 * row + rows * case["q_heads"] * (case["d"] * 4 + 4) + extra + pages,
            "flops": 4.0 * rows * vis * case["q_heads"] * case["d"]}


# ------------------------------------------------------- the plain forms

def _scale_exponent(amax, dtype):
    """The least e with amax < 7 * 2^e, inside the type's range: amax = m * 2^E with m in [.5, 1)."""
    m, E = torch.frexp(amax)
    lo, hi = RANGE[dtype]
    e = E - 3 + (m >= 0.875).to(E.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, lo)).clamp(lo, hi)


def _quantise(x, dtype):
    """[..., d] -> packed bytes [..., d/2] and scale bytes [..., d/32]."""
    b = x.float().unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    e = _scale_exponent(b.abs().amax(-1), dtype)
    y = torch.ldexp(b, -e[..., None])
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + 8 * torch.signbit(y).to(torch.uint8)
    code = torch.where(bad[..., None], torch.zeros_like(code), code).flatten(-2)
    packed = code[..., 0::2] + 16 * code[..., 1::2]
    scale = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return packed, scale


def _dequantise(data, scale):
    """The f32 values of packed bytes [..., d/2] under scale bytes [..., d/32]."""
    code = torch.stack((data & 15, data >> 4), -1).flatten(-2)
    m = (code & 7).float()
    a = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, 2 * m - 8))
    a = torch.where(code >= 8, -a, a).unflatten(-1, (-1, 32))
    # two factors: 2^(s - 127) itself may lie below the normal range
    s = scale.int() - 127
    v = torch.ldexp(torch.ldexp(a, (s // 2)[..., None]), (s - s // 2)[..., None])
    return torch.where((scale == 255)[..., None], torch.full_like(v, math.nan), v).flatten(-2)


def _slots_of(s, positions):
    """Cache slots of key positions [R, ...] of each request."""
    bs = s["block_size"]
    flat = positions.flatten(1).long()
    return (s["block_table"].gather(1, flat // bs).long() * bs + flat % bs).view(positions.shape)


def _gathered(s, name, slots):
    """f32 rows of the cache `name` at `slots` (any shape): of the fewer of the two, the rows read or the rows held."""
    data, scale = s[name + "_data"].flatten(0, 1), s[name + "_scale"].flatten(0, 1)
    if slots.numel() < data.shape[0]:
        return _dequantise(data[slots], scale[slots])
    return _dequantise(data, scale)[slots]


def _plain_selected(s):
    q, pool, Q = s["q"].float(), s["pool"], s["query"]
    R = s["seq_lens"].numel()
    vis = (s["seq_lens"].long()[:, None] - Q + 1 + torch.arange(Q, device=q.device)).view(-1, 1)
    idx = s["idx"].long()
    pos = (idx[:, :, None] * pool + torch.arange(pool, device=q.device)).flatten(1)
    seen = (idx >= 0).repeat_interleave(pool, 1) & (pos < vis)
    pos = torch.where(seen, pos, torch.zeros_like(pos))
    slots = _slots_of(s, pos.view(R, -1)).view(pos.shape)
    kv = s["k_data"].shape[2]
    rows, H, d = q.shape
    k = _gathered(s, "k", slots).transpose(1, 2)                                         # [rows, kv, n, d]
    score = torch.matmul(q.view(rows, kv, H // kv, d), k.transpose(2, 3)) * s["sm_scale"]
    del k
    seen = seen[:, None, None, :]
    v = _gathered(s, "v", slots).transpose(1, 2)
    return _softmax_product(score, seen, v, rows, H, d, s)


def _softmax_product(score, seen, v, rows, H, d, s):
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return {"out": out.reshape(rows, H, d).to(s["q"].dtype), "lse": (torch.log(total) + top).reshape(rows, H)}


def _plain_window(s):
    q, Q = s["q"].float(), s["query"]
    rows, H, d = q.shape
    R, L = s["seq_lens"].numel(), s["max_seq_len"]
    kv = s["k_data"].shape[2]
    at = torch.arange(L, device=q.device)
    vis = s["seq_lens"].long()[:, None] - Q + 1 + torch.arange(Q, device=q.device)           # [R, Q]
    seen = at < vis[..., None]
    if s["window"]:
        seen = seen & ((at >= vis[..., None] - s["window"]) | (at < s["sinks"]))
    owned = at[None, :] < s["seq_lens"].long()[:, None]
    slots = _slots_of(s, torch.where(owned, at[None, :], torch.zeros_like(at[None, :])))     # [R, L]
    k = _gathered(s, "k", slots).permute(0, 2, 3, 1)                                         # [R, kv, d, L]
    g = H // kv
    qs = q.view(R, Q, kv, g, d).permute(0, 2, 1, 3, 4).reshape(R, kv, Q * g, d)
    score = torch.matmul(qs, k) * s["sm_scale"]
    del k
    v = _gathered(s, "v", slots).transpose(1, 2)                                             # [R, kv, L, d]
    seen = seen[:, None, :, None, :].expand(R, 1, Q, g, L).reshape(R, 1, Q * g, L)
    r = _softmax_product(score, seen, v, R * kv * Q * g, 1, d, s)
    return {"out": r["out"].view(R, kv, Q, g, d).transpose(1, 2).reshape(rows, H, d),
            "lse": r["lse"].view(R, kv, Q, g).transpose(1, 2).reshape(rows, H)}


def _plain(s):
    if s["op"] == "write":
        for x, data, scale in ((s["k"], s["k_data"], s["k_scale"]), (s["v"], s["v_data"], s["v_scale"])):
            packed, byte = _quantise(x, s["dtype"])
            data.flatten(0, 1)[s["slots"]] = packed
            scale.flatten(0, 1)[s["slots"]] = byte
        return {n: _gathered(s, n, s["slots"]).to(s[n].dtype) for n in ("k", "v")}
    if s["op"] == "read":
        return _gathered(s, "k", s["slots"]).to(TYPES[s["dtype"]])
    return _plain_selected(s) if s["op"] == "selected" else _plain_window(s)


# --------------------------------------------------------------- the calls

def _call(s):
    import sparse_attention_lightning_indexer_amd as li
    if s["op"] == "write":
        li.mx4_cache_write(s["k"], s["slots"], s["k_data"], s["k_scale"], s["v"], s["v_data"], s["v_scale"])
        return {n: li.mx4_cache_read(s[n + "_data"], s[n + "_scale"], s["slots"], s[n].dtype) for n in ("k", "v")}
    if s["op"] == "read":
        return li.mx4_cache_read(s["k_data"], s["k_scale"], s["slots"], TYPES[s["dtype"]])
    cache = (s["k_data"], s["k_scale"], s["v_data"], s["v_scale"], s["block_table"], s["seq_lens"])
    if s["op"] == "selected":
        out, lse = li.mx4_attend_selected(s["q"], *cache, s["query"], s["idx"], s["sm_scale"], pool_size=s["pool"])
    else:
        out, lse = li.mx4_attend_window(s["q"], *cache, s["query"], s["max_seq_len"], s["sm_scale"],
                                        window=s["window"], sinks=s["sinks"])
    return {"out": out, "lse": lse}


def run(state):
    return _call(state) if own else _plain(state)


# -------------------------------------------------------------- the inputs

def _normal(gen, shape, dtype):
    """Unit-normal rows whose channels have spread magnitudes (a few large ones), as projected keys do."""
    gain = torch.exp(0.5 * torch.randn(shape[-1], generator=gen, device=DEV))
    x = torch.empty(shape, dtype=TYPES[dtype], device=DEV)
    for part in x.view(-1, shape[-1]).split(1 << 20):   # bounded scratch
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV) * gain)
    return x


def _filled(gen, n_blocks, bs, heads, d, dtype):
    """A cache of quantised rows."""
    data = torch.empty((n_blocks, bs, heads, d // 2), dtype=torch.uint8, device=DEV)
    scale = torch.empty((n_blocks, bs, heads, d // 32), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 25) // (bs * heads * d))
    for a in range(0, n_blocks, step):
        n = min(step, n_blocks - a)
        data[a:a + n], scale[a:a + n] = _quantise(_normal(gen, (n, bs, heads, d), dtype), dtype)
    return data, scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case)
    heads, d, bs, dtype = case["kv_heads"], case["d"], case["block_size"], case["dtype"]
    if case["op"] in ("write", "read"):
        n = case["tokens"] if case["op"] == "write" else case["cached"]
        blocks = -(-n // bs) + 3
        order = torch.randperm(blocks, generator=gen, device=DEV)
        at = torch.arange(n, device=DEV)
        slots = order[at // bs] * bs + at % bs                     # consecutive tokens, pages in any order
        if case["op"] == "write":
            for name in ("k", "v"):
                s[name] = _normal(gen, (n, heads, d), dtype)
                s[name + "_data"] = torch.zeros((blocks, bs, heads, d // 2), dtype=torch.uint8, device=DEV)
                s[name + "_scale"] = torch.full((blocks, bs, heads, d // 32), 127, dtype=torch.uint8, device=DEV)
        else:
            s["k_data"], s["k_scale"] = _filled(gen, blocks, bs, heads, d, dtype)
            slots = slots[:case["rows"]]
        s["slots"] = slots.contiguous()
        return s
    R, Q = case["requests"], case["query"]
    lens = torch.randint(case["len_lo"], case["len_hi"] + 1, (R,), generator=gen, device=DEV)
    s["max_seq_len"] = case["len_hi"]
    per = -(-case["len_hi"] // bs)
    blocks = R * per + 3
    s["block_table"] = torch.randperm(blocks, generator=gen, device=DEV)[: R * per].view(R, per).int().contiguous()
    s["seq_lens"] = lens.int()
    s["k_data"], s["k_scale"] = _filled(gen, blocks, bs, heads, d, dtype)
    s["v_data"], s["v_scale"] = _filled(gen, blocks, bs, heads, d, dtype)
    s["q"] = torch.randn((R * Q, case["q_heads"], d), generator=gen, device=DEV).to(TYPES[dtype])
    s["sm_scale"] = 1.0 / math.sqrt(d)
    if case["op"] == "selected":
        # as the top-k gives them: distinct entries in order of a score, -1 behind a short row's last
        units = -(-case["len_hi"] // case["pool"])
        k = case["k"]
        idx = torch.full((R * Q, k), -1, dtype=torch.int32, device=DEV)
        vis = (lens[:, None] - Q + 1 + torch.arange(Q, device=DEV)).view(-1)
        have = (vis + case["pool"] - 1).clamp(min=0) // case["pool"]
        for a in range(0, R * Q, 128):
            r = torch.rand((min(128, R * Q - a), units), generator=gen, device=DEV)
            r = r.masked_fill(torch.arange(units, device=DEV) >= have[a:a + 128, None], -1.0)
            top, at = r.topk(min(k, units), 1)
            idx[a:a + 128, : top.shape[1]] = torch.where(top >= 0, at, -torch.ones_like(at)).int()
        s["idx"] = idx
    return s


# --------------------------------------- the definition in 64 bits, row by row

_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_rows(data, scale):
    """f64 values of cache rows [n, heads, d/2], by table."""
    table = torch.tensor([v for v in _MAGNITUDES] + [-v for v in _MAGNITUDES], dtype=torch.float64, device=data.device)
    pair = torch.stack([table[(data % 16).long()], table[torch.div(data, 16, rounding_mode="floor").long()]], -1)
    values = pair.reshape(data.shape[:-1] + (-1, 32))
    factor = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=data.device), scale.double() - 127)
    factor = torch.where(scale == 255, torch.full_like(factor, math.nan), factor)
    return (values * factor[..., None]).reshape(data.shape[:-1] + (-1,))


def _exact_quantised(x, dtype):
    """The value each element of x is held as: the nearest of its block's grid, ties to the even code."""
    lo, hi = RANGE[dtype]
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    limit = torch.tensor([7.0 * 2.0 ** e for e in range(lo, hi)], dtype=torch.float64, device=x.device)
    flat, to = x.reshape(-1, 32), out.view(-1, 32)
    for a in range(0, flat.shape[0], 1 << 20):
        b = flat[a:a + (1 << 20)].double()
        e = lo + torch.searchsorted(limit, b.abs().amax(1), right=True)
        unit = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=x.device), e.double())[:, None]
        r = b.abs() / unit
        held = torch.zeros_like(r)
        for i in range(1, 8):  # above the middle of two neighbours, or on it where the upper code is even
            middle = 0.5 * (_MAGNITUDES[i - 1] + _MAGNITUDES[i])
            held = torch.where((r > middle) | ((r == middle) & (i % 2 == 0)), _MAGNITUDES[i], held)
        to[a:a + (1 << 20)] = torch.copysign(held * unit, b)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        return {n: _exact_quantised(s[n], case["dtype"]) for n in ("k", "v")}
    bs = case["block_size"]
    if case["op"] == "read":
        return _exact_rows(s["k_data"].flatten(0, 1)[s["slots"]], s["k_scale"].flatten(0, 1)[s["slots"]])
    rows, H, d = s["q"].shape
    kv, Q = case["kv_heads"], case["query"]
    out = torch.zeros((rows, H, d), dtype=torch.float64, device=DEV)
    lse = torch.full((rows, H), -math.inf, dtype=torch.float64, device=DEV)
    lens, tables = s["seq_lens"].tolist(), s["block_table"].long()
    for r, length in enumerate(lens):
        at = torch.arange(length, device=DEV)
        slots = tables[r, at // bs] * bs + at % bs
        k, v = (_exact_rows(s[n + "_data"].flatten(0, 1)[slots], s[n + "_scale"].flatten(0, 1)[slots]).transpose(0, 1)
                .contiguous() for n in ("k", "v"))                                # [kv, length, d]
        for j in range(Q):
            t, vis = r * Q + j, length - Q + 1 + j
            if vis <= 0:
                continue
            if case["op"] == "selected":
                first = s["idx"][t][s["idx"][t] >= 0].long() * case["pool"]
                pos = (first[:, None] + torch.arange(case["pool"], device=DEV)).flatten()
                pos = pos[pos < vis]
            elif case["window"]:
                start = max(0, vis - case["window"])
                pos = torch.cat([at[: min(case["sinks"], start)], at[start:vis]])
            else:
                pos = at[:vis]
            if not pos.numel():
                continue
            keys, values = (k[:, :vis], v[:, :vis]) if pos.numel() == vis and case["op"] == "window" else (
                k[:, pos], v[:, pos])
            z = torch.matmul(s["q"][t].double().view(kv, H // kv, d), keys.transpose(1, 2).contiguous()) * s["sm_scale"]
            lse[t] = torch.logsumexp(z, -1).view(H)
            out[t] = torch.matmul(torch.exp(z - lse[t].view(kv, -1, 1)), values).view(H, d)
    return {"out": out, "lse": lse}
