"""Plain 64-bit restatement of the 4-bit paged cache (layout, write, attention, page step), written
from the header's definitions one token and one request at a time."""
import numpy as np

UNIT = 16


def unit_bytes(d, group):
    return 16 * d + 128 * (d // group)


def key_row(t):
    return 2 * (t & 3) + ((t >> 2) & 1) + (t & 8)


def key_code_at(t, i, d):
    """(byte in the unit, 0 for the low half) of key coordinate i of token t."""
    w, e = divmod(i, 8)
    word = (w & 3) * (d // 32) + (w >> 2)
    return key_row(t) * (d // 2) + 4 * word + e // 2, e % 2


def value_code_at(t, i, d):
    w, e = divmod(i, 8)
    word = w ^ 8 if d == 128 and t & 2 else w
    return 8 * d + t * (d // 2) + 4 * word + e // 2, e % 2


def key_scale_at(t, g, d, group):
    """Bytes of s and z of group g of token t's key."""
    ng = d // group
    row = 16 * d + key_row(t) * 4 * ng
    return row + 2 * g, row + 2 * (ng + g)


def value_scale_at(t, g, d, group):
    ng = d // group
    row = 16 * d + 64 * ng + t * 4 * ng
    return row + 4 * g, row + 4 * g + 2


def quantise(x, group):
    """Codes, s and z (fp16) of x [..., d] (any type that fp32 holds), with the defined roundings."""
    g = np.asarray(x, dtype=np.float32).reshape(*x.shape[:-1], -1, group)
    lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
    z = np.clip(lo, np.float32(-65504), np.float32(65504)).astype(np.float16)
    z32 = z.astype(np.float32)
    with np.errstate(over="ignore", under="ignore"):
        s = np.clip((hi - z32) * np.float32(1 / 15), 0, 65504).astype(np.float16)
        s32 = s.astype(np.float32)
        inv = np.where(s32 > 0, np.float32(1) / np.where(s32 > 0, s32, np.float32(1)), np.float32(0))
        c = np.clip(np.rint((g - z32) * inv), 0, 15)
    return c.astype(np.uint8).reshape(x.shape), s[..., 0], z[..., 0]


def values(c, s, z, group):
    """c s + z in 64 bits, [..., d]."""
    rep = lambda a: np.repeat(a.astype(np.float64), group, -1)  # noqa: E731
    with np.errstate(invalid="ignore"):  # bytes that no write has filled may read as inf or NaN
        return c.astype(np.float64) * rep(s) + rep(z)


def write(cache, k, v, slots, group):
    """Writes k, v [n, Hkv, d] at their slots of cache [n_blocks, Hkv, page / 16, unit] in place."""
    n, hkv, d = k.shape
    page = 16 * cache.shape[2]
    parts = [(quantise(k, group), key_code_at, key_scale_at), (quantise(v, group), value_code_at, value_scale_at)]
    for i in range(n):
        slot = int(slots[i])
        if not 0 <= slot < cache.shape[0] * page:
            continue
        t = slot % UNIT
        unit = cache[slot // page, :, slot % page // UNIT]
        for (c, s, z), code_at, scale_at in parts:
            for j in range(d):
                at, high = code_at(t, j, d)
                old = unit[:, at]
                unit[:, at] = (old & 0x0F) | (c[i, :, j] << 4) if high else (old & 0xF0) | c[i, :, j]
            for g in range(d // group):
                a, b = scale_at(t, g, d, group)
                unit[:, a:a + 2] = s[i, :, g, None].view(np.uint8)
                unit[:, b:b + 2] = z[i, :, g, None].view(np.uint8)


def read(cache, slots, d, group):
    """Keys and values [n, Hkv, d] in 64 bits of the tokens at `slots`."""
    page = 16 * cache.shape[2]
    slots = np.asarray(slots, dtype=np.int64)
    units = cache[slots // page, :, slots % page // UNIT]          # [n, Hkv, unit]
    tok = slots % UNIT
    out = []
    for code_at, scale_at in ((key_code_at, key_scale_at), (value_code_at, value_scale_at)):
        at = np.array([[code_at(t, i, d) for i in range(d)] for t in range(UNIT)])
        sc = np.array([[scale_at(t, g, d, group) for g in range(d // group)] for t in range(UNIT)])
        ix = at[tok][:, None, :, 0]
        b = np.take_along_axis(units, np.broadcast_to(ix, units.shape[:2] + (d,)), 2)
        c = np.where(at[tok][:, None, :, 1] == 1, b >> 4, b & 15)
        half = []
        for w in (0, 1):
            lo = np.take_along_axis(units, np.broadcast_to(sc[tok][:, None, :, w], units.shape[:2] + (d // group,)), 2)
            hi = np.take_along_axis(units, np.broadcast_to(sc[tok][:, None, :, w] + 1, units.shape[:2] + (d // group,)), 2)
            half.append((lo.astype(np.uint16) | (hi.astype(np.uint16) << 8)).view(np.float16))
        out.append(values(c, half[0], half[1], group))
    return out


def attend(q, cache, tables, kv_lens, group, cu_q=None, window=0, scale=None):
    """out [n_q, Hq, d] in 64 bits, and per (row, head) the weights' sums that error bounds need:
    A = sum_t p_t |v_t| per coordinate and S = max_t sum_i |q_i k_ti| scale."""
    n_q, hq, d = q.shape
    B, hkv = len(kv_lens), cache.shape[1]
    page = 16 * cache.shape[2]
    scale = 1 / np.sqrt(d) if scale is None else scale
    if cu_q is None:
        cu_q = np.arange(B + 1)
    out = np.zeros((n_q, hq, d))
    A, S = np.zeros((n_q, hq, d)), np.zeros((n_q, hq))
    room = tables.shape[1] * page
    for b in range(B):
        n, m = int(np.clip(kv_lens[b], 0, room)), int(cu_q[b + 1] - cu_q[b])
        pos = np.arange(n)
        blk = tables[b, pos // page].astype(np.int64)
        pos = pos[(blk >= 0) & (blk < cache.shape[0])]
        if m == 0 or len(pos) == 0:
            continue
        k, v = read(cache, tables[b, pos // page].astype(np.int64) * page + pos % page, d, group)
        for i in range(m):
            e = n - m + i + 1
            seen = (pos < e) & (pos >= (e - window if window else 0))
            if not seen.any():
                continue
            for h in range(hq):
                g = h // (hq // hkv)
                qr = q[cu_q[b] + i, h].astype(np.float64)
                s = k[seen, g] @ qr * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[cu_q[b] + i, h] = p @ v[seen, g]
                A[cu_q[b] + i, h] = p @ np.abs(v[seen, g])
                S[cu_q[b] + i, h] = (np.abs(k[seen, g]) @ np.abs(qr)).max() * abs(scale)
    return out, A, S


def page_step(lens, new_lens, tables, free_list, free_count, page, n_slots):
    """The step, one request after another.  tables and free_list are changed in place; returns
    (lens_out, cu_new, slots, refused, free_count_out)."""
    B, mb = tables.shape
    nb = len(free_list)
    room = mb * page
    held = [min(max(int(x), 0), room) for x in lens]
    pages = [-(-h // page) for h in held]
    count = min(max(int(free_count), 0), nb)
    for b in range(B):
        if new_lens[b] < 0:
            for j in range(pages[b]):
                if count < nb:
                    free_list[count] = tables[b, j]
                    count += 1
    avail, wanted, used = count, 0, 0
    cu, slots, lens_out, refused = [0], np.full(n_slots, -1, dtype=np.int64), [], 0
    for b in range(B):
        add = int(new_lens[b])
        if add < 0:
            lens_out.append(0)
            cu.append(cu[-1])
            continue
        cu.append(cu[-1] + add)
        ok = held[b] + add <= room and cu[-1] <= n_slots
        if ok:
            need = -(-(held[b] + add) // page) - pages[b]
            first = wanted
            wanted += need
            ok = need == 0 or wanted <= avail
        if not ok:
            refused += 1
            lens_out.append(held[b])
            continue
        for j in range(need):
            tables[b, pages[b] + j] = free_list[avail - 1 - (first + j)]
        used += need
        for j in range(add):
            pos = held[b] + j
            t = int(tables[b, pos // page])
            if 0 <= t < nb:
                slots[cu[-2] + j] = t * page + pos % page
        lens_out.append(held[b] + add)
    return (np.array(lens_out, dtype=np.int64), np.minimum(cu, 2 ** 31 - 1), slots, refused, avail - used)
