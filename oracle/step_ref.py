"""Float64 oracle of a served step round the attention: adapters beside a
quantised product, probabilities, drafted tokens checked, pages of the cache.

Plain loops and numpy, written from the formulas; shares no code with the GPU path.
"""
import numpy as np

U = 2.0 ** -24


# ------------------------------------------------------------- adapters --
def gemm_adapters(X, weights, down, up, ids, alpha=None):
    """(Y, bound) of Y = X weights^T + alpha_a (X down_a^T) up_a^T in float64: X [M, K], weights [N, K] as the
    matrix unit is given them, down [count, r, K], up [count, N, r], ids [M].

    bound: K sums in float32 of each product, in any order, are off by at most gamma_K of the sum of magnitudes; X
    down^T by that, alpha and the shares of K (16 more roundings at most); it is all there in three bf16 numbers (8 bits
    each, and each one's rounding error has the next one's); then the second product's sums over 3 r terms and its
    addition."""
    X, weights = np.asarray(X, np.float64), np.asarray(weights, np.float64)
    K = X.shape[1]

    def gamma(n):
        return n * U / (1 - n * U)
    Y = X @ weights.T
    bound = gamma(K + 16) * (np.abs(X) @ np.abs(weights).T)
    for m, a in enumerate(ids):
        if not 0 <= a < down.shape[0]:
            continue
        d, u = np.asarray(down[a], np.float64), np.asarray(up[a], np.float64)
        f = 1.0 if alpha is None else float(alpha[a])
        t, size = f * (d @ X[m]), abs(f) * (np.abs(d) @ np.abs(X[m]))
        Y[m] += u @ t
        part = np.abs(u) @ size
        bound[m] += (gamma(K + 32) + gamma(3 * d.shape[0] + 16)) * 1.01 * part
        bound[m] += 16 * U * np.abs(Y[m])
    return Y, bound


# -------------------------------------------------------- probabilities --
def probabilities(logits, temperature=None):
    """[seqs, tokens, vocab] float64 from logits of that shape; temperature [seqs]."""
    x = np.asarray(logits, np.float64)
    p = np.zeros(x.shape)
    for b in range(x.shape[0]):
        t = 1.0 if temperature is None else float(temperature[b])
        for i in range(x.shape[1]):
            row = x[b, i]
            if not 0 <= t < np.inf or np.isnan(row).any() or (t > 0 and np.isposinf(row).any()):
                p[b, i] = np.nan
            elif np.isneginf(row).all():
                continue
            elif t == 0:
                p[b, i, int(np.argmax(row))] = 1.0  # the first of equals
            else:
                with np.errstate(over="ignore"):
                    e = np.exp((row - row.max()) / t)
                p[b, i] = e / e.sum()
    return p


# --------------------------------------------------------- verification --
def verify_draft(p, draft, uniforms, q=None, parents=None):
    """(path, counts, next) of float32 arrays, every step in float64."""
    seqs, tokens, vocab = p.shape
    path, counts = np.full((seqs, tokens), -1, np.int32), np.zeros(seqs, np.int32)
    following = np.full(seqs, -1, np.int32)

    def clean(row):
        return np.where(row > 0, row, 0.0).astype(np.float64)
    with np.errstate(invalid="ignore"):
        for b in range(seqs):
            walk = [0]
            while True:
                c = walk[-1]
                r, mass = clean(p[b, c]), 1.0
                qc = clean(q[b, c]) if q is not None else None
                for i in range(c + 1, tokens):
                    parent = i - 1 if parents is None else parents[b, i]
                    x = draft[b, i]
                    if parent != c or not 0 <= x < vocab:
                        continue
                    if float(uniforms[b, i]) * (qc[x] if qc is not None else 1.0) * mass < r[x]:
                        walk.append(i)
                        break
                    if qc is not None:
                        r = np.maximum(r - mass * qc, 0.0)
                        mass = r.sum()
                    else:
                        mass -= r[x]
                        r[x] = 0.0
                if walk[-1] == c:
                    break
            if not r.sum() > 0:
                r = clean(p[b, c])
            upto = np.cumsum(r)
            past = np.nonzero((upto > float(uniforms[b, 0]) * upto[-1]) & (r > 0))[0]
            some = np.nonzero(r > 0)[0]
            path[b, :len(walk)], counts[b] = walk, len(walk)
            following[b] = past[0] if past.size else some[-1] if some.size else -1
    return path, counts, following


# ---------------------------------------------------------------- pages --
FIELDS = ("k_codes", "k_scales", "k_zeros", "v_codes", "v_scales", "v_zeros")


def kv_copy(pool, src, dst):
    """Pages in place in a pool of numpy arrays (serving_ref.empty_pool)."""
    pages = pool["k_codes"].shape[0]
    for s, d in zip(src, dst):
        if 0 <= s < pages and 0 <= d < pages:
            for name in FIELDS:
                pool[name][d] = pool[name][s]


def kv_compact(pool, tables, lengths, path, counts):
    """Tokens moved in place, one after the other."""
    pages, _, page, _ = pool["k_codes"].shape
    seqs, width = tables.shape
    tokens = path.shape[1]
    for b in range(seqs):
        if lengths[b] < 0:
            continue

        def slot(pos):
            i, o = divmod(int(pos), page)
            return (int(tables[b, i]), o) if i < width and 0 <= tables[b, i] < pages else None
        before = -1
        for j in range(min(int(counts[b]), tokens)):
            at = int(path[b, j])
            if not before < at < tokens:
                break
            before = at
            s, d = slot(int(lengths[b]) + at), slot(int(lengths[b]) + j)
            if at == j or s is None or d is None:
                continue
            for name in FIELDS:
                t = pool[name]
                if name == "v_codes":
                    t[d[0], :, :, d[1]] = t[s[0], :, :, s[1]]
                else:
                    t[d[0], :, d[1]] = t[s[0], :, s[1]]


def pages_of(n, page):
    return max(0, -(-int(n) // page))


def pages_free(refs, tables, lengths, page):
    for b in range(tables.shape[0]):
        for i in range(pages_of(lengths[b], page), tables.shape[1]):
            if 0 <= tables[b, i] < refs.size:
                refs[tables[b, i]] -= 1
            tables[b, i] = -1


def pages_fork(refs, tables, lengths, src, dst, page):
    seqs, width = tables.shape
    given = set()
    for s, d in zip(src, dst):
        if not (0 <= s < seqs and 0 <= d < seqs):
            continue
        left_out = d in list(src) or d in given
        given.add(d)
        if left_out:
            continue
        for i in range(width):
            if 0 <= tables[d, i] < refs.size:
                refs[tables[d, i]] -= 1
            e = tables[s, i] if i < pages_of(lengths[s], page) else -1
            tables[d, i] = e if 0 <= e < refs.size else -1
            if tables[d, i] >= 0:
                refs[tables[d, i]] += 1


def pages_extend(refs, tables, lengths, added, page):
    """(copies [2, seqs], info [2]); refs and tables in place, entry after entry."""
    seqs, width = tables.shape
    copies = np.full((2, seqs), -1, np.int32)
    new_refs, new_tables = refs.copy(), tables.copy()
    free, taken, lacking = [e for e in range(refs.size) if refs[e] <= 0], 0, 0
    for b in range(seqs):
        if lengths[b] < 0 or added[b] <= 0:
            continue
        first, end = int(lengths[b]) // page, pages_of(int(lengths[b]) + int(added[b]), page)
        lacking += end - max(first, width) if end > width else 0
        for i in range(first, min(end, width)):
            e = new_tables[b, i]
            there = 0 <= e < refs.size
            if there and new_refs[e] <= 1:
                continue
            if taken == len(free):
                lacking += 1
                if there:
                    new_refs[e] -= 1
                continue
            new = free[taken]
            taken += 1
            if there:
                new_refs[e] -= 1
                if i * page < lengths[b]:
                    copies[:, b] = e, new
            new_refs[new], new_tables[b, i] = 1, new
    if lacking:
        return np.full((2, seqs), -1, np.int32), np.array([0, lacking], np.int32)
    refs[:], tables[:] = new_refs, new_tables
    return copies, np.array([taken, 0], np.int32)
