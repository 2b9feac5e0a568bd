"""The operators of the 4-bit paged key/value cache, as they are measured: cases, inputs, plain forms, exact values.

Three operators, used one after the other in a serving step:
  page   block tables, slots and the free list advanced by one step from the requests' lengths
  write  new keys and values quantised to 4 bits and written at their slots
  attn   attention of one or more query tokens per sequence over the 4-bit cache
"""
import math

import numpy as np
import torch

own = False

UNIT = 16  # tokens of one cache unit
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step over long contexts: the attention workload of this repository's benchmark
        {"name": "attn_long", "op": "attn", "B": 16, "hq": 32, "hkv": 4, "d": 64, "group": 32, "page": 64,
         "len_lo": 32768, "len_hi": 32768, "q_max": 1, "window": 0, "dtype": "fp16"},
        # a continuous batch in the middle of its requests: every length from a few tokens to 8K
        {"name": "attn_ragged", "op": "attn", "B": 64, "hq": 32, "hkv": 8, "d": 128, "group": 32, "page": 16,
         "len_lo": 1, "len_hi": 8191, "q_max": 1, "window": 0, "dtype": "bf16"},
        # a single user's next token after a short prompt: latency
        {"name": "attn_one", "op": "attn", "B": 1, "hq": 32, "hkv": 8, "d": 128, "group": 64, "page": 16,
         "len_lo": 517, "len_hi": 517, "q_max": 1, "window": 0, "dtype": "bf16"},
        # drafted tokens checked together (1 to 6 a sequence), seven query heads a kv head, sliding window
        {"name": "attn_verify", "op": "attn", "B": 24, "hq": 28, "hkv": 4, "d": 128, "group": 128, "page": 32,
         "len_lo": 3, "len_hi": 12001, "q_max": 6, "window": 4096, "dtype": "bf16"},
        # chunked prefill: up to 1024 query tokens a sequence over the cached prefix and themselves
        {"name": "attn_chunk", "op": "attn", "B": 3, "hq": 32, "hkv": 8, "d": 128, "group": 32, "page": 64,
         "len_lo": 1024, "len_hi": 8192, "q_max": 1024, "window": 0, "dtype": "fp16"},
        # a small model with one kv head per query head (12 heads of 64, contexts up to 1024)
        {"name": "attn_mha", "op": "attn", "B": 8, "hq": 12, "hkv": 12, "d": 64, "group": 32, "page": 16,
         "len_lo": 17, "len_hi": 1024, "q_max": 1, "window": 0, "dtype": "fp16"},
        # the writes of one decode step: one token of each request
        {"name": "write_step", "op": "write", "n": 96, "hkv": 4, "d": 64, "group": 32, "page": 16,
         "run_len": 1, "skip": 0, "fused": 6, "dtype": "fp16"},
        # the writes of a large prefill batch, from a fused projection's output
        {"name": "write_prefill", "op": "write", "n": 65536, "hkv": 8, "d": 128, "group": 32, "page": 64,
         "run_len": 4096, "skip": 0, "fused": 6, "dtype": "bf16"},
        # a ragged batch padded to a captured size, in 32 bits: every 7th token has no slot
        {"name": "write_odd", "op": "write", "n": 5003, "hkv": 3, "d": 64, "group": 64, "page": 32,
         "run_len": 37, "skip": 7, "fused": 1, "dtype": "fp32"},
        # a decode step of a busy server: one token for each of 256 requests
        {"name": "page_decode", "op": "page", "B": 256, "page": 16, "max_blocks": 512, "len_hi": 8000, "n_slots": 256,
         "prefill_every": 0, "prefill": 0, "release_every": 0},
        # a large mixed step: decodes, prefills of 1500 tokens and finished requests together
        {"name": "page_mixed", "op": "page", "B": 2048, "page": 64, "max_blocks": 256, "len_hi": 12000, "n_slots": 262144,
         "prefill_every": 13, "prefill": 1500, "release_every": 17},
        # a handful of requests of one user, a captured batch larger than what is in it
        {"name": "page_few", "op": "page", "B": 5, "page": 32, "max_blocks": 64, "len_hi": 900, "n_slots": 64,
         "prefill_every": 3, "prefill": 20, "release_every": 4},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "write", "page"])
    if op == "attn":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 3, 4, 8, 12])
        hq = hkv * rng.choice([1, 2, 3, 4, 6, 7, 8, 8, 12, 16])
        q_max = rng.choice([1, 1, 1, _log_int(rng, 2, 16), _log_int(rng, 16, 512)])
        hi = max(q_max, _log_int(rng, 2, 32768))
        most = (1 << 27) // (hi * hkv * d)
        if q_max > 1:
            most = min(most, (1 << 32) // (hi * q_max * hq * 2))
        if most < 1:
            hi = max(q_max, 2048)
            most = 1 + (1 << 24) // (hi * hkv * d)
        case = {"op": "attn", "B": _log_int(rng, 1, max(1, min(256, most))), "hq": hq, "hkv": hkv, "d": d,
                "group": rng.choice([32, 64, d]), "page": rng.choice([16, 32, 64, 128]), "len_lo": rng.choice([0, 1, hi]),
                "len_hi": hi, "q_max": q_max, "window": rng.choice([0, 0, _log_int(rng, 1, 8192)]),
                "dtype": rng.choice(["fp16", "bf16"])}
        while work(case)["flops"] > 1.2e11:
            case["q_max"] = 1 + case["q_max"] // 2
        return case
    if op == "write":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 3, 4, 8])
        return {"op": "write", "n": _log_int(rng, 1, 65536 * 8 * 128 // (2 * hkv * d) if hkv * d > 512 else 32768),
                "hkv": hkv, "d": d, "group": rng.choice([32, 64, d]), "page": rng.choice([16, 32, 64, 128]),
                "run_len": _log_int(rng, 1, 5000), "skip": rng.choice([0, 0, 5]), "fused": rng.choice([1, 2, 6]),
                "dtype": rng.choice(["fp16", "bf16", "bf16", "fp32"])}
    B = _log_int(rng, 1, 2048)
    page = rng.choice([16, 32, 64, 128])
    pre = _log_int(rng, 1, 1500)
    every = rng.choice([0, 3, 13])
    tokens = B + (0 if not every else (B // every + 1) * pre)
    hi = _log_int(rng, 1, 12000)
    return {"op": "page", "B": B, "page": page, "max_blocks": (hi + pre) // page + rng.choice([1, 2, 100]), "len_hi": hi,
            "n_slots": min(262144, max(1, tokens + rng.choice([0, 0, 31, -tokens // 2]))), "prefill_every": every,
            "prefill": pre, "release_every": rng.choice([0, 5, 17])}


def work(case):
    if case["op"] == "attn":
        lens, qlens = _lens(case), _qlens(case)
        rec = case["d"] + 8 * (case["d"] // case["group"])  # bytes of a token of one kv head, key and value
        read, flops = 0, 0
        for n, m in zip(lens.tolist(), qlens.tolist()):
            first = max(0, n - m + 1 - case["window"]) if case["window"] else 0
            read += max(0, n - first) if m else 0
            for i in range(m):
                end = n - m + i + 1
                seen = max(0, min(end, case["window"]) if case["window"] else end)
                flops += 4 * seen * case["hq"] * case["d"]
        nq = int(qlens.sum())
        return {"bytes": read * case["hkv"] * rec + 2 * 2 * nq * case["hq"] * case["d"] + 4 * read // case["page"] + 8 * case["B"],
                "flops": flops}
    if case["op"] == "write":
        size = 4 if case["dtype"] == "fp32" else 2
        rec = case["d"] + 8 * (case["d"] // case["group"])
        return {"bytes": case["n"] * (case["hkv"] * (2 * 2 * case["d"] * size + rec) + 4), "flops": 10 * 2 * case["n"] * case["hkv"] * case["d"]}
    _, new = _page_lens(case)
    pages = int(sum(-(-int(x) // case["page"]) for x in new.tolist() if x > 0))
    return {"bytes": 4 * (4 * case["B"] + case["n_slots"] + 2 * pages), "flops": 0}


def _lens(case):
    """Cached tokens of each sequence, evenly spread over the case's range, in a fixed mixed-up order."""
    B = case["B"]
    x = case["len_lo"] + (case["len_hi"] - case["len_lo"]) * (np.arange(B) + 0.5) / B
    x = np.round(x).astype(np.int64)
    x[B // 2] = case["len_hi"]
    return np.random.RandomState(B).permutation(x)


def _qlens(case):
    B, m = case["B"], case["q_max"]
    x = 1 + (np.arange(B) * 7 + 3) % m
    x[0] = m
    return x.astype(np.int64)


def _page_lens(case):
    B = case["B"]
    lens = np.round(case["len_hi"] * (np.arange(B) + 0.5) / B).astype(np.int64)
    lens = np.random.RandomState(B).permutation(lens)
    new = np.ones(B, dtype=np.int64)
    if case["prefill_every"]:
        at = np.arange(1, B, case["prefill_every"])
        new[at] = case["prefill"]
        lens[at] = 0
    if case["release_every"]:
        new[2::case["release_every"]] = -1
    return lens, new


# ------------------------------------------------------------------------------------ the cache's layout

def _unit_bytes(d, group):
    return UNIT * d + 128 * (d // group)


def _layout(d, dev):
    """Positions of the values of one unit: key nibbles and value nibbles [16, d], and the row of a token in the key part."""
    tok = torch.arange(UNIT, device=dev)
    i = torch.arange(d, device=dev)
    row = 2 * (tok & 3) + ((tok >> 2) & 1) + (tok & 8)
    word = ((i % 32) // 8) * (d // 32) + i // 32
    key = row[:, None] * d + word * 8 + i % 8
    half = (((tok >> 1) & 1) * (d // 16 if d == 128 else 0))[:, None]
    value = tok[:, None] * d + ((i // 8) ^ half) * 8 + i % 8
    return key, value, row


def _quantise(x, group):
    """Codes, steps and zeros of x [..., d] in fp32: z = fp16(min), s = fp16((max - z) * fp32(1/15)), c = round((x - z) * fp32(1/s))."""
    x = x.float()
    g = x.unflatten(-1, (-1, group))
    z = g.amin(-1).clamp(-65504, 65504).half()
    s = ((g.amax(-1) - z.float()) * (1.0 / 15.0)).clamp(0, 65504).half()
    inv = torch.where(s > 0, 1.0 / s.float(), torch.zeros_like(s, dtype=torch.float32))
    c = ((g - z.float()[..., None]) * inv[..., None]).round().clamp(0, 15)
    return c, s, z


def _values(c, s, z):
    return (c * s.float()[..., None] + z.float()[..., None]).flatten(-2)


def _pack_bytes(nib):
    return nib[..., 0::2] | (nib[..., 1::2] << 4)


def _write_units(units, k, v, group):
    """Whole units [..., UB] from k and v [..., 16, d] (token order)."""
    d, ng = k.shape[-1], k.shape[-1] // group
    key, value, row = _layout(d, k.device)
    c, s, z = _quantise(k, group)
    sc = torch.empty(s.shape[:-1] + (2 * ng,), dtype=torch.float16, device=k.device)
    sc[..., row, :] = torch.cat([s, z], -1)
    _put_unit(units, c, key, sc, 0, UNIT * d)
    c, s, z = _quantise(v, group)
    _put_unit(units, c, value, torch.stack([s, z], -1).flatten(-2), UNIT * d // 2, UNIT * d + 64 * ng)


def _put_unit(units, c, place, sc, at, sc_at):
    d = place.shape[1]
    nib = torch.empty(c.shape[:-3] + (UNIT * d,), dtype=torch.uint8, device=c.device)
    nib[..., place.reshape(-1)] = c.flatten(-3).to(torch.uint8)
    units[..., at:at + UNIT * d // 2] = _pack_bytes(nib)
    sc = sc.flatten(-2).contiguous().view(torch.uint8)
    units[..., sc_at:sc_at + sc.shape[-1]] = sc


# ------------------------------------------------------------------------------------ inputs

def _channels(shape, gen, dev):
    """Per-(head, channel) scales of a cache: log-normal with one channel in a head ten times as large."""
    s = torch.exp(0.5 * torch.randn(shape, generator=gen, device=dev))
    s[..., 3] *= 10 if shape[-1] > 3 else 1
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 2 + 1)
    state = dict(case)
    if case["op"] == "attn":
        B, hkv, d, page = case["B"], case["hkv"], case["d"], case["page"]
        lens, qlens = _lens(case), _qlens(case)
        max_blocks = max(1, -(-int(lens.max()) // page))
        n_blocks = max(1, int(sum(-(-int(n) // page) for n in lens.tolist())))
        ids = torch.randperm(n_blocks, generator=gen, device=dev).to(torch.int32)
        table = np.full((B, max_blocks), -1, dtype=np.int64)
        at = 0
        for b, n in enumerate(lens.tolist()):
            m = -(-n // page)
            table[b, :m] = np.arange(at, at + m)
            at += m
        pos = torch.from_numpy(table).to(dev)
        tables = torch.where(pos >= 0, ids[pos.clamp(min=0)], torch.full_like(ids[:1], -1)).to(torch.int32)
        cache = torch.empty((n_blocks, hkv, page // UNIT, _unit_bytes(d, case["group"])), dtype=torch.uint8, device=dev)
        sk, sv = _channels((hkv, d), gen, dev), _channels((hkv, d), gen, dev)
        step = max(1, (1 << 25) // (hkv * page * d))
        for a in range(0, n_blocks, step):  # in pieces: the inputs of a large cache are four times its size
            m = min(step, n_blocks - a)
            shape = (m, hkv, page // UNIT, UNIT, d)
            k = torch.randn(shape, generator=gen, device=dev) * sk[:, None, None, :]
            v = torch.randn(shape, generator=gen, device=dev) * sv[:, None, None, :]
            _write_units(cache[a:a + m], k, v, case["group"])
        nq = int(qlens.sum())
        q = torch.randn((nq, case["hq"], d), generator=gen, device=dev) / sk.repeat_interleave(case["hq"] // hkv, 0).sqrt()
        cu = np.concatenate([[0], np.cumsum(qlens)])
        state.update(q=(1.5 * q).to(DTYPES[case["dtype"]]), cache=cache, tables=tables,
                     kv_lens=torch.from_numpy(lens).to(dev, torch.int32), cu_q=torch.from_numpy(cu).to(dev, torch.int32),
                     scale=1.0 / math.sqrt(d))
    elif case["op"] == "write":
        n, hkv, d, page = case["n"], case["hkv"], case["d"], case["page"]
        f = case["fused"]
        width = (f + 2) * hkv * d if f > 1 else 2 * hkv * d
        rows = torch.randn((n, width), generator=gen, device=dev).to(DTYPES[case["dtype"]])
        sc = _channels((hkv, d), gen, dev)
        rows[:, -2 * hkv * d:] *= torch.cat([sc.reshape(-1), sc.reshape(-1)]).to(rows.dtype)
        runs = -(-n // case["run_len"])
        blocks = -(-case["run_len"] // page) + 1
        n_blocks = runs * blocks
        ids = torch.randperm(n_blocks, generator=gen, device=dev).view(runs, blocks)
        i = torch.arange(n, device=dev)
        start = torch.randint(0, page, (runs,), generator=gen, device=dev)
        pos = start[i // case["run_len"]] + i % case["run_len"]
        slots = ids[i // case["run_len"], pos // page] * page + pos % page
        if case["skip"]:
            slots[::case["skip"]] = -1
        cache = torch.randint(0, 256, (n_blocks, hkv, page // UNIT, _unit_bytes(d, case["group"])), generator=gen, device=dev, dtype=torch.uint8)
        state.update(k=rows[:, -2 * hkv * d:-hkv * d].unflatten(1, (hkv, d)), v=rows[:, -hkv * d:].unflatten(1, (hkv, d)),
                     slots=slots.to(torch.int32), cache=cache)
    else:
        B, page, mb = case["B"], case["page"], case["max_blocks"]
        lens, new = _page_lens(case)
        held = -(-lens // page)
        need = int(sum(max(0, -(-(n + m) // page) - h) for n, m, h in zip(lens.tolist(), new.tolist(), held.tolist()) if m > 0))
        n_blocks = int(held.sum()) + need + 3
        ids = torch.randperm(n_blocks, generator=gen, device=dev).to(torch.int32)
        first = torch.from_numpy(np.cumsum(held) - held).to(dev)
        h = torch.from_numpy(held).to(dev)
        j = torch.arange(mb, device=dev)
        tables = torch.where(j < h[:, None], ids[(first[:, None] + j).clamp(max=n_blocks - 1)], torch.full_like(ids[:1], -1))
        free = torch.zeros(n_blocks, dtype=torch.int32, device=dev)
        n_free = n_blocks - int(held.sum())
        free[:n_free] = ids[int(held.sum()):]
        state.update(lens=torch.from_numpy(lens).to(dev, torch.int32), new_lens=torch.from_numpy(new).to(dev, torch.int32),
                     tables=tables.to(torch.int32).contiguous(), free_list=free,
                     free_count=torch.tensor([n_free], dtype=torch.int32, device=dev),
                     free_count_out=torch.zeros(1, dtype=torch.int32, device=dev))
    return state


# ------------------------------------------------------------------------------------ one pass

def run(state):
    return {"attn": _run_attn, "write": _run_write, "page": _run_page}[state["op"]](state)


def _run_attn(s):
    if own:
        import random_access_kv_fq_b200 as fq
        return fq.fq_kv4_attn(s["q"], s["cache"], s["tables"], s["kv_lens"], s["group"],
                              cu_q=s["cu_q"] if s["q_max"] > 1 else None, max_q=s["q_max"], window=s["window"], scale=s["scale"])
    q, cache, tables, page, d, group = s["q"], s["cache"], s["tables"], s["page"], s["d"], s["group"]
    B, hkv, hq, m = tables.shape[0], s["hkv"], s["hq"], s["q_max"]
    L, ng = tables.shape[1] * page, d // group
    key, value, row = _layout(d, q.device)
    units = cache[tables.long().clamp(0, cache.shape[0] - 1)]                 # [B, blocks, hkv, units, UB]
    units = units.permute(0, 2, 1, 3, 4).flatten(2, 3)                        # [B, hkv, L / 16, UB]
    nib = units[..., :UNIT * d]
    nib = torch.stack([nib & 15, nib >> 4], -1).flatten(-2)                   # [B, hkv, L / 16, 2 * 16 * d]
    sc = units[..., UNIT * d:].contiguous().view(torch.float16).float()
    ks = sc[..., :32 * ng].unflatten(-1, (UNIT, 2, ng))[..., row, :, :]       # [.., 16, 2, ng]
    vs = sc[..., 32 * ng:].unflatten(-1, (UNIT, ng, 2))
    kc = nib[..., key.reshape(-1)].unflatten(-1, (UNIT, ng, group)).float()
    k = (kc * ks[..., 0, :, None] + ks[..., 1, :, None]).flatten(-2).flatten(2, 3)
    vc = nib[..., UNIT * d + value.reshape(-1)].unflatten(-1, (UNIT, ng, group)).float()
    v = (vc * vs[..., 0, None] + vs[..., 1, None]).flatten(-2).flatten(2, 3)  # [B, hkv, L, d]
    cu, kv_lens = s["cu_q"].long(), s["kv_lens"].long().clamp(0, L)
    qn = cu[1:] - cu[:-1]
    i = torch.arange(m, device=q.device)
    rows = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)                      # [B, m]
    qp = q[rows].float().unflatten(2, (hkv, hq // hkv))                       # [B, m, hkv, g, d]
    sco = torch.einsum("bmhgd,bhld->bhgml", qp, k) * s["scale"]
    pos = torch.arange(L, device=q.device)
    end = (kv_lens - qn)[:, None] + i + 1                                     # [B, m]
    seen = pos < end[..., None]
    if s["window"]:
        seen &= pos >= end[..., None] - s["window"]
    seen &= ((tables >= 0) & (tables < cache.shape[0])).repeat_interleave(page, 1)[:, None]
    seen = seen[:, None, None]
    sco = sco.masked_fill(~seen, -math.inf)
    top = sco.amax(-1, keepdim=True)
    p = torch.exp(sco - torch.where(top == -math.inf, torch.zeros_like(top), top))
    den = p.sum(-1)[..., None]
    o = torch.einsum("bhgml,bhld->bhgmd", p, v) / torch.where(den > 0, den, torch.ones_like(den))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, m, hq, d).to(q.dtype)
    of = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(cu, of, right=True) - 1
    return o[b, of - cu[b]]


def _run_write(s):
    if own:
        import random_access_kv_fq_b200 as fq
        kv, vv = fq.fq_kv4_write(s["k"], s["v"], s["slots"], s["cache"], s["group"], values=True)
        return {"cache": s["cache"], "k": kv, "v": vv}
    cache, d, group, page = s["cache"], s["d"], s["group"], s["page"]
    slots = s["slots"].long()
    # with skipped tokens (slot -1) the others are picked out
    ok = (slots >= 0) & (slots < cache.shape[0] * page) if s["skip"] else slice(None)
    slots = slots[ok]
    unit = (slots // page)[:, None] * s["hkv"] + torch.arange(s["hkv"], device=cache.device)
    unit = unit * (page // UNIT) + ((slots % page) // UNIT)[:, None]
    tok, ng = slots % UNIT, d // group
    key, value, row = _layout(d, cache.device)
    c, st, z = _quantise(s["k"], group)
    k = _values(c, st, z).to(s["k"].dtype)
    _put_tokens(cache, unit, row[tok], c[ok], torch.argsort(key, 1)[tok], torch.cat([st[ok], z[ok]], -1), 0, UNIT * d)
    c, st, z = _quantise(s["v"], group)
    v = _values(c, st, z).to(s["v"].dtype)
    _put_tokens(cache, unit, tok, c[ok], torch.argsort(value, 1)[tok], torch.stack([st[ok], z[ok]], -1).flatten(-2), UNIT * d // 2, UNIT * d + 64 * ng)
    return {"cache": cache, "k": k, "v": v}


def _put_tokens(cache, unit, row, c, order, sc, at, sc_at):
    """Codes c [n, hkv, ng, group] and steps and zeros sc [n, hkv, 2 ng] into row `row` [n] of the units `unit` [n, hkv]."""
    flat = cache.view(-1, cache.shape[-1])
    nib = torch.gather(c.flatten(-2).to(torch.uint8), 2, order[:, None].expand(-1, unit.shape[1], -1))
    codes, sc = _pack_bytes(nib), sc.contiguous().view(torch.uint8)
    lane = torch.arange(codes.shape[-1], device=cache.device)
    flat[unit[..., None], (at + row * codes.shape[-1])[:, None, None] + lane] = codes
    lane = torch.arange(sc.shape[-1], device=cache.device)
    flat[unit[..., None], (sc_at + row * sc.shape[-1])[:, None, None] + lane] = sc


def _run_page(s):
    if own:
        import random_access_kv_fq_b200 as fq
        lens, cu, slots, refused = fq.fq_page_step(s["lens"], s["new_lens"], s["tables"], s["free_list"], s["free_count"],
                                                   s["page"], s["n_slots"], free_count_out=s["free_count_out"])
        return {"lens": lens, "cu": cu, "slots": slots, "refused": refused, "tables": s["tables"], "free_list": s["free_list"],
                "free_count": s["free_count_out"]}
    tables, free, page, n_slots = s["tables"], s["free_list"], s["page"], s["n_slots"]
    B, mb = tables.shape
    nb, dev = free.shape[0], tables.device
    held, new = s["lens"].long().clamp(0, mb * page), s["new_lens"].long()
    pages = (held + page - 1) // page
    gone = torch.where(new < 0, pages, torch.zeros_like(pages)).cumsum(0)
    count = s["free_count"].long().clamp(0, nb)
    avail = (count + gone[-1]).clamp(max=nb)
    # pages of finished requests go onto the stack, in request order
    r = torch.arange(nb, device=dev)
    b = torch.searchsorted(gone, r, right=True).clamp(max=B - 1)
    j = (r - (gone[b] - pages[b])).clamp(0, mb - 1)
    back = tables[b, j]
    src = (r - count).clamp(0, nb - 1)
    free.copy_(torch.where((r >= count) & (r < avail), back[src], free))
    add = new.clamp(min=0)
    cu = torch.cat([torch.zeros_like(add[:1]), add.cumsum(0)])
    fits = (new >= 0) & (held + add <= mb * page) & (cu[1:] <= n_slots)
    need = torch.where(fits, (held + add + page - 1) // page - pages, torch.zeros_like(pages))
    upto = need.cumsum(0)
    served = fits & ((need == 0) | (upto <= avail))
    taken = torch.where(served & (need > 0), upto, torch.zeros_like(upto)).amax()
    # the a-th page handed out is the a-th from the stack's top
    a = torch.arange(nb, device=dev)
    b = torch.searchsorted(upto, a, right=True).clamp(max=B - 1)
    at = b * mb + pages[b] + a - (upto[b] - need[b])
    grown = torch.cat([tables.reshape(-1), tables.new_zeros(1)])
    grown[torch.where(a < taken, at, torch.full_like(at, B * mb))] = free[(avail - 1 - a).clamp(0, nb - 1)]
    tables.copy_(grown[:-1].view(B, mb))
    i = torch.arange(n_slots, device=dev)
    b = torch.searchsorted(cu[1:], i, right=True)
    real = b < B
    b = b.clamp(max=B - 1)
    pos = (held[b] + i - cu[b]).clamp(0, mb * page - 1)
    p = tables[b, pos // page].long()
    slots = torch.where(real & served[b] & (p >= 0) & (p < nb), p * page + pos % page, torch.full_like(p, -1))
    s["free_count_out"].copy_(avail - taken)
    lens = torch.where(new < 0, torch.zeros_like(held), torch.where(served, held + add, held))
    refused = ((new >= 0) & ~served).sum().reshape(1)
    return {"lens": lens.to(torch.int32), "cu": cu.clamp(max=2 ** 31 - 1).to(torch.int32), "slots": slots.to(torch.int32),
            "refused": refused.to(torch.int32), "tables": tables, "free_list": free, "free_count": s["free_count_out"]}


# ------------------------------------------------------------------------------------ exact values

def exact(case, seed):
    """From the definitions, in 64 bits, a sequence and a kv head at a time. Whole numbers have no such value."""
    if case["op"] == "page":
        return None
    if case["op"] == "write":
        s = prepare(case, seed)
        return {"cache": None, "k": _exact_values(s["k"], case["group"]), "v": _exact_values(s["v"], case["group"])}
    s = prepare(case, seed)
    dev, d, group, page, hkv, hq = s["q"].device, case["d"], case["group"], case["page"], case["hkv"], case["hq"]
    out = torch.zeros((s["q"].shape[0], hq, d), dtype=torch.float64, device=dev)
    cu, lens, tables, ng = s["cu_q"].tolist(), s["kv_lens"].tolist(), s["tables"], d // group
    words = s["cache"][..., :UNIT * d].contiguous().view(torch.int32).view(*s["cache"].shape[:3], 2, UNIT, d // 8)
    halves = s["cache"][..., UNIT * d:].contiguous().view(torch.float16).double()
    coord = torch.arange(d, device=dev)
    for b in range(case["B"]):
        n, m = lens[b], cu[b + 1] - cu[b]
        if n == 0 or m == 0:
            continue
        pos = torch.arange(n, device=dev)
        blk = tables[b, pos // page].long()
        u, t = (pos % page) // UNIT, pos % UNIT
        krow = 2 * (t % 4) + (t // 4) % 2 + 8 * (t // 8)
        kword = (coord // 8) % 4 * (d // 32) + coord // 32
        vword = coord // 8 + torch.zeros_like(t)[:, None]
        if d == 128:
            vword = torch.where(((t // 2) % 2 == 1)[:, None], (vword + 8) % 16, vword)
        for h in range(hkv):
            kw = words[blk, h, u, 0, krow][:, kword]
            vw = torch.gather(words[blk, h, u, 1, t], 1, vword)
            sh = (4 * (coord % 8)).to(torch.int32)
            kc, vc = ((kw >> sh) & 15).double(), ((vw >> sh) & 15).double()
            hs = halves[blk, h, u]
            g = coord // group
            ks = torch.gather(hs, 1, krow[:, None] * 2 * ng + g)
            kz = torch.gather(hs, 1, krow[:, None] * 2 * ng + ng + g)
            vs = torch.gather(hs, 1, 32 * ng + (t[:, None] * ng + g) * 2)
            vz = torch.gather(hs, 1, 32 * ng + (t[:, None] * ng + g) * 2 + 1)
            k, v = kc * ks + kz, vc * vs + vz
            r = hq // hkv
            q = s["q"][cu[b]:cu[b + 1], h * r:(h + 1) * r].double()
            sc = torch.einsum("mgd,ld->mgl", q, k) * case_scale(d)
            end = n - m + 1 + torch.arange(m, device=dev)
            seen = pos < end[:, None]
            if case["window"]:
                seen = seen & (pos >= end[:, None] - case["window"])
            sc = sc.masked_fill(~seen[:, None], -math.inf)
            w = torch.softmax(sc, -1)
            w = torch.where(torch.isnan(w), torch.zeros_like(w), w)
            out[cu[b]:cu[b + 1], h * r:(h + 1) * r] = torch.einsum("mgl,ld->mgd", w, v)
    return out


def _exact_values(x, group):
    """c s + z in 64 bits, with the roundings that the definition of z, s and c names."""
    x = x.double()
    g = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    z = g.min(-1, keepdim=True).values.half().double()
    s = ((g.max(-1, keepdim=True).values - z).float().double() * float(np.float32(1 / 15))).float().half().double()
    inv = (1 / s).float().double()
    c = torch.round(((g - z).float().double() * inv).float().double()).clamp(0, 15)
    return (torch.where(s > 0, c, torch.zeros_like(c)) * s + z).reshape(x.shape)


def case_scale(d):
    return 1.0 / math.sqrt(d)
