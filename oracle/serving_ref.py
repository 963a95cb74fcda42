"""Float64 oracle of the serving operators: rotary positions, the key/value
cache on min-max grids, and attention of drafted tokens over it.

Plain loops and numpy, written from the formulas; shares no code with the GPU
path.  The grid's decisions are the float32 steps that define it; everything
else is float64.
"""
import math

import numpy as np

F = np.float32


# --------------------------------------------------------------- rotary --
def rope_frequencies(rot, base=10000.0, scaling=None):
    """Radians per position of every pair."""
    sc = dict(scaling or {})
    kind, factor = sc.get("kind"), sc.get("factor", 1.0)
    if kind == "base":
        base = base * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        w = base ** (-2.0 * i / rot)
        if kind == "linear":
            w = w / factor
        if kind == "parts":
            turns = sc["original"] / (2.0 * math.pi / w)  # how often it turns over the original length
            low, high = sc.get("low", 1.0), sc.get("high", 32.0)
            keep = 0.0 if turns <= low else 1.0 if turns >= high else (turns - low) / (high - low)
            w = (1.0 - keep) * (w / factor) + keep * w
        out.append(w)
    return np.array(out)


def rope_table(length, rot, base=10000.0, scaling=None):
    """[length, 2, rot/2] in float64."""
    w = rope_frequencies(rot, base, scaling)
    mag = dict(scaling or {}).get("magnitude", 1.0)
    t = np.zeros((length, 2, rot // 2))
    for p in range(length):
        t[p, 0], t[p, 1] = mag * np.cos(p * w), mag * np.sin(p * w)
    return t


def rope(x, positions, table, layout="half", inverse=False):
    """x [tokens, heads, dim] -> rotated float64."""
    x = np.asarray(x, np.float64)
    half = table.shape[2]
    y = x.copy()
    for t, p in enumerate(positions):
        if not 0 <= p < table.shape[0]:
            y[t, :, :2 * half] = np.nan
            continue
        for i in range(half):
            ia, ib = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
            c, s = float(table[p, 0, i]), float(table[p, 1, i])
            if inverse:
                s = -s
            a, b = x[t, :, ia], x[t, :, ib]
            y[t, :, ia], y[t, :, ib] = a * c - b * s, b * c + a * s
    return y


# ---------------------------------------------------------------- cache --
def kv_grid(row, bits):
    """(scale, zero, codes) of one row: float32 steps by definition."""
    row = np.asarray(row, F)
    maxq = F((1 << bits) - 1)
    with np.errstate(all="ignore"):
        lo, hi = min(row.min(), F(0)), max(row.max(), F(0))
        span = F(hi - lo)
        if not np.all(np.isfinite(row)) or not np.isfinite(span):
            return F(np.nan), 0, np.zeros(row.shape, np.uint8)
        if span < F(2.0 ** -100):
            return F(1), 0, np.zeros(row.shape, np.uint8)
        s = F(span * F(F(1) / maxq))
        r = F(F(1) / s)
        z = min(max(np.rint(F(-lo * r)), F(0)), maxq)
        x = (row * r).astype(F)
        q = np.clip(np.rint((x + z).astype(F)), 0, maxq)
    return s, int(z), q.astype(np.uint8)


def kv_values(s, z, q):
    """fl32(s (q - z)), what a read returns before it is rounded to its type."""
    return (F(s) * (q.astype(F) - F(z))).astype(F)


def empty_pool(pages, heads, page, dim, bits):
    rb = dim * bits // 8
    return dict(k_codes=np.zeros((pages, heads, page, rb), np.uint8), k_scales=np.zeros((pages, heads, page), F),
                k_zeros=np.zeros((pages, heads, page), np.uint8), v_codes=np.zeros((pages, heads, rb, page), np.uint8),
                v_scales=np.zeros((pages, heads, page), F), v_zeros=np.zeros((pages, heads, page), np.uint8))


def kv_write(pool, k, v, slots, bits):
    """Write rows k, v [tokens, heads, dim] into the pool in place."""
    page = pool["k_codes"].shape[2]
    pages = pool["k_codes"].shape[0]
    half = k.shape[2] // 2
    for t, slot in enumerate(slots):
        if not 0 <= slot < pages * page:
            continue
        a, o = divmod(int(slot), page)
        for h in range(k.shape[1]):
            s, z, q = kv_grid(k[t, h], bits)
            pool["k_scales"][a, h, o], pool["k_zeros"][a, h, o] = s, z
            pool["k_codes"][a, h, o] = q if bits == 8 else q[0::2] | (q[1::2] << 4)
            s, z, q = kv_grid(v[t, h], bits)
            pool["v_scales"][a, h, o], pool["v_zeros"][a, h, o] = s, z
            pool["v_codes"][a, h, :, o] = q if bits == 8 else q[:half] | (q[half:] << 4)


def kv_codes(pool, a, h, o, bits):
    """(K codes, V codes) of one (page, head, offset)."""
    kb, vb = pool["k_codes"][a, h, o], pool["v_codes"][a, h, :, o]
    if bits == 8:
        return kb, vb
    k = np.empty(2 * kb.size, np.uint8)
    k[0::2], k[1::2] = kb & 15, kb >> 4
    return k, np.concatenate([vb & 15, vb >> 4])


def kv_read(pool, slots, bits):
    """(k, v) float32 [tokens, heads, dim]; zeros for slots outside."""
    pages, heads, page, rb = pool["k_codes"].shape
    dim = rb * 8 // bits
    k, v = np.zeros((len(slots), heads, dim), F), np.zeros((len(slots), heads, dim), F)
    for t, slot in enumerate(slots):
        if not 0 <= slot < pages * page:
            continue
        a, o = divmod(int(slot), page)
        for h in range(heads):
            kq, vq = kv_codes(pool, a, h, o, bits)
            k[t, h] = kv_values(pool["k_scales"][a, h, o], pool["k_zeros"][a, h, o], kq)
            v[t, h] = kv_values(pool["v_scales"][a, h, o], pool["v_zeros"][a, h, o], vq)
    return k, v


# ------------------------------------------------------------ attention --
def visible(lengths, tokens, mask, b, t, capacity):
    """Positions that drafted token t of sequence b sees (before page numbers are looked at)."""
    n = int(lengths[b])
    if n < 0:
        return []
    got = list(range(min(n, capacity)))
    for i in range(tokens):
        if n + i >= capacity:
            break
        if mask is None:
            on = i <= t
        else:
            on = (int(mask[b, t, i // 32]) >> (i % 32)) & 1
        if on:
            got.append(n + i)
    return got


def tree_attention(q, pool, tables, lengths, bits, mask=None, scale=None):
    """(o, spread, top) in float64: o [seqs, tokens, heads, dim]; for error bounds, spread = sum_j p_j |v_j| of
    every output and top [seqs, tokens, heads, 2] = the largest scale sum_d |q_d| |k_jd| of a row's scores and the
    largest |score|."""
    q = np.asarray(q, np.float64)
    seqs, tokens, heads, dim = q.shape
    pages, kv_heads, page, _ = pool["k_codes"].shape
    group = heads // kv_heads
    scale = dim ** -0.5 if scale is None else scale
    o, spread = np.zeros(q.shape), np.zeros(q.shape)
    top = np.zeros((seqs, tokens, heads, 2))
    rows = {}
    for b in range(seqs):
        for t in range(tokens):
            pos = [j for j in visible(lengths, tokens, mask, b, t, tables.shape[1] * page)
                   if 0 <= tables[b, j // page] < pages]
            if not pos:
                continue
            for h in range(kv_heads):
                ks, vs = [], []
                for j in pos:
                    key = (int(tables[b, j // page]), h, j % page)
                    if key not in rows:
                        kq, vq = kv_codes(pool, *key, bits)
                        s, z = float(pool["k_scales"][key]), float(pool["k_zeros"][key])
                        sv, zv = float(pool["v_scales"][key]), float(pool["v_zeros"][key])
                        rows[key] = s * (kq.astype(np.float64) - z), sv * (vq.astype(np.float64) - zv)
                    kr, vr = rows[key]
                    ks.append(kr)
                    vs.append(vr)
                ks, vs = np.array(ks), np.array(vs)
                for g in range(group):
                    row = q[b, t, h * group + g]
                    x = scale * (ks @ row)
                    p = np.exp(x - x.max())
                    p /= p.sum()
                    o[b, t, h * group + g] = p @ vs
                    spread[b, t, h * group + g] = p @ np.abs(vs)
                    top[b, t, h * group + g] = abs(scale) * (np.abs(ks) @ np.abs(row)).max(), np.abs(x).max()
    return o, spread, top


def bf16(x):
    """float64 rounded to 8 significant bits, ties to even."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def attention_bound(o, spread, top, dim):
    """Largest allowed |error| of a bf16 result, from the widths of the operands.

    Scores: queries (bf16, times a power of two) and code - zero point are exact in float16 and so are their products
    in float32; their sum over dim has float32's roundings, random-walk growth with a factor of four.  Its products
    with the scale and the factor to powers of two, the reference and their difference: 2^-21 of the largest score.
    Weights: times their position's scale, two bfloat16 numbers to nearest, 2^-16.  Sums over up to 2^14
    positions in float32, random-walk growth with a factor of four: 2^-15.  All of that is relative to spread,
    with the scores' error twice (weight and sum).  The result is then rounded to bf16: it lies between the rounded
    ends of that interval, which for most values are the same number."""
    delta = 4.0 * math.sqrt(dim) * 2.0 ** -24 * top[..., 0] + 2.0 ** -21 * top[..., 1]
    eps = (2.0 ** -16 + 2.0 ** -15 + 2.0 * delta[..., None]) * spread
    return np.maximum(np.abs(bf16(o + eps) - o), np.abs(bf16(o - eps) - o)) + 1e-30
