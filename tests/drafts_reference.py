"""Trees of drafted tokens, their verification and compaction, and the norm and rotation in front of the cache, in 64
bits on the CPU with numpy, one node and one value at a time where that is plainer.  Shares nothing with the library."""
import numpy as np

from tests import kv_reference as kv


def random_parents(rng, n, reach=None):
    """Parents of n nodes: each one of the `reach` nodes in front of it (any of them without)."""
    return np.array([-1] + [rng.randint(max(0, i - (reach or i)), i) for i in range(1, n)][:max(n - 1, 0)], np.int32)[:n]


def ancestors(parents, i):
    """Node i and its ancestors, itself first."""
    out = []
    while i >= 0:
        out.append(i)
        i = int(parents[i])
    return out


def trees(parents, lengths, q_start, words, window, tokens):
    """(masks uint64 [tokens][words], positions)"""
    mask, positions = np.zeros((tokens, words), np.uint64), np.full(tokens, -1, np.int32)
    for r in range(len(lengths)):
        a, b = int(q_start[r]), int(q_start[r + 1])
        for i in range(b - a):
            way = ancestors(parents[a:b], i)
            positions[a + i] = lengths[r] - (b - a) + len(way) - 1
            for j in way[:window] if window else way:
                mask[a + i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return mask, positions


def verify(target, draft, drafts, parents, q_start, accept, sample):
    """(path, tokens, counts)"""
    path, tokens = np.full(len(drafts), -1, np.int32), np.full(len(drafts), -1, np.int32)
    counts = np.zeros(len(q_start) - 1, np.int32)
    for r in range(len(counts)):
        a, b = int(q_start[r]), int(q_start[r + 1])
        if a == b:
            continue
        u, way = 0, [0]
        left = taken = None
        i, refused = 1, set()
        left, taken = 1.0, 0.0
        while i < b - a:
            if parents[a + i] == u:
                x = int(drafts[a + i])
                p = float(target[a + u, x])
                if draft is None:
                    p = 0.0 if x in refused else p
                    ok = float(accept[a + i]) * left < p
                else:
                    q = float(draft[a + u, x])
                    ok = float(accept[a + i]) * q * left < max(p - taken * q, 0.0)
                if ok:
                    u, left, taken, refused = i, 1.0, 0.0, set()
                    way.append(i)
                elif draft is None:
                    left -= p
                    refused.add(x)
                else:
                    taken += left
                    left = np.maximum(target[a + u].astype(np.float64) - taken * draft[a + u], 0).sum()
            i += 1
        last = target[a + u].astype(np.float64)
        if draft is not None:
            last = np.maximum(last - taken * draft[a + u], 0)
        elif refused:
            last[list(refused)] = 0
        if last.sum() == 0:
            last = target[a + u].astype(np.float64)
        upto = np.cumsum(last)
        if upto[-1] > 0:
            tokens[a + len(way) - 1] = np.flatnonzero(upto > float(sample[r]) * upto[-1])[0]
        path[a:a + len(way)] = way
        tokens[a:a + len(way) - 1] = [drafts[a + j] for j in way[1:]]
        counts[r] = len(way)
    return path, tokens, counts


def compact(path, counts, lengths, q_start, tables, codes, scale, elem):
    """(codes, scale, kept lengths) of one of the two caches"""
    table, p = kv.decode_table(elem), codes.shape[2]
    old, old_scale = codes.copy(), scale.astype(np.float64)
    codes, scale = codes.copy(), old_scale.copy()
    kept = []
    for r in range(len(lengths)):
        n = int(q_start[r + 1] - q_start[r])
        context = int(lengths[r]) - n
        kept.append(context + int(counts[r]))
        moves = [(int(path[q_start[r] + i]), i) for i in range(int(counts[r])) if path[q_start[r] + i] != i]
        for page in sorted({(context + i) // p for _, i in moves}):
            run = [(context + node, context + i) for node, i in moves if (context + i) // p == page]
            block, first = int(tables[r, page]), run[0][1] % p
            for h in range(codes.shape[1]):
                from_block = [int(tables[r, s // p]) for s, _ in run]
                from_scale = old_scale[from_block, h]
                from_codes = old[from_block, h, [s % p for s, _ in run]]
                with np.errstate(invalid="ignore"):
                    values = np.where(from_scale[:, None] == 0, 0.0, table[from_codes] * from_scale[:, None])
                was = now = old_scale[block, h]
                other = values[from_scale != was]
                most = np.max(np.abs(other[np.isfinite(other)]), initial=0.0)
                if was == 0:
                    now = kv.scale_for(other, elem)
                elif most > kv.MAX[elem] * was:
                    now = max(was, kv.scale_for(other, elem))
                if now != was:
                    with np.errstate(invalid="ignore"):
                        front = table[codes[block, h, :first]] * (was / now)
                    codes[block, h, :first] = 0 if was == 0 else kv.encode(front, elem)
                for (s, d), c, x, z in zip(run, from_codes, values, from_scale):
                    codes[block, h, d % p] = c if z == now else kv.encode(x / now, elem)
                scale[block, h] = now
    return codes, scale.astype(np.float32), np.array(kept, np.int32)


# ------------------------------------------------------------------ norm and rotation
def turn(x, table, positions, interleaved, back=False):
    """(x turned, the sum of the magnitudes that make each value)"""
    y, most = x.copy(), np.abs(x)
    if table is None:
        return y, most
    half = table.shape[1] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        c, s = table[positions, i].astype(np.float64)[:, None], table[positions, half + i].astype(np.float64)[:, None]
        s = -s if back else s
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        most[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
        most[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, most


def norm(x, w, table, positions, eps, interleaved, half_step, smallest):
    """(y, tolerance).  In FP32 the sum of D squares is off by at most D 2^-24 of itself, r by half of that and the 2^-22
    of its function, each of the three products by 2^-24, a turned value by 2^-23 of its terms: (D / 2 + 10) 2^-24 of the
    terms in all, and D 2^-24 holds room for the second order; then the output is rounded by half a step."""
    d = x.shape[2]
    n = x / np.sqrt((x * x).mean(2, keepdims=True) + eps) * w
    y, most = turn(n, table, positions, interleaved)
    return y, np.abs(y) * half_step + most * (d + 10) * 2.0 ** -24 * (1 + half_step) + smallest


def norm_backward(dy, x, w, table, positions, eps, interleaved, half_step, smallest):
    """(dx, dw, tolerance of dx, of dw).  As above: r off by (D / 2 + 4) 2^-24, g by 2^-23 of its terms, the dot product
    w g xh by (D + 8) 2^-24 of the sum of its terms' magnitudes; so dx by at most (2 D + 32) 2^-24 of r (|w| G + |xh| M),
    G the magnitude of g's terms and M the mean of |w| G |xh|.  dw sums T terms, each off by (D / 2 + 8) 2^-24, in sums
    that lose at most T 2^-24 of the sum of their magnitudes."""
    t, h, d = x.shape
    g, most = turn(dy, table, positions, interleaved, back=True)
    r = 1 / np.sqrt((x * x).mean(2, keepdims=True) + eps)
    xh = x * r
    dx = r * (w * g - xh * (w * g * xh).mean(2, keepdims=True))
    dw = (g * xh).sum((0, 1))
    bound = r * (np.abs(w) * most + np.abs(xh) * (np.abs(w) * most * np.abs(xh)).mean(2, keepdims=True))
    return (dx, dw, np.abs(dx) * half_step + bound * (2 * d + 32) * 2.0 ** -24 * (1 + half_step) + smallest,
            (most * np.abs(xh)).sum((0, 1)) * (t * h + d + 16) * 2.0 ** -24)


# ------------------------------------------------------------------ attention of a tree's queries
def sees(mask, positions, lengths, q_start, window):
    """For each request, bool [rows][length]: which tokens each of its rows sees."""
    out = []
    for r, length in enumerate(lengths):
        a, b = int(q_start[r]), int(q_start[r + 1])
        context = int(length) - (b - a)
        s = np.zeros((b - a, int(length)), bool)
        for i in range(b - a):
            first = max(0, int(positions[a + i]) - window + 1) if window else 0
            s[i, first:context] = True
            for j in range(b - a):
                s[i, context + j] = int(mask[a + i, j // 64]) >> (j % 64) & 1
        out.append(s)
    return out


def tree_attention(q, k_codes, v_codes, k_scale, v_scale, tables, lengths, q_start, seen, elem, softmax_scale):
    """(out, lse, out's tolerance but for its own rounding, lse's): the formula and the tolerances of
    kv_reference.attention, for rows that see what `seen` says."""
    table, p = kv.decode_table(elem), k_codes.shape[2]
    t, heads, d = q.shape
    group = heads // k_codes.shape[1]
    out, lse = np.zeros((t, heads, d)), np.full((t, heads), -np.inf)
    tol, lse_tol = np.zeros((t, heads, d)), np.zeros((t, heads))
    q = q.astype(np.float64)
    for r, length in enumerate(lengths):
        a, b = int(q_start[r]), int(q_start[r + 1])
        if a == b:
            continue
        blocks = tables[r, :-(-int(length) // p)]
        for h in range(k_codes.shape[1]):
            k = (table[k_codes[blocks, h]] * k_scale[blocks, h].astype(np.float64)[:, None, None]).reshape(-1, d)[:length]
            c = table[v_codes[blocks, h]].reshape(-1, d)[:length]
            sv = np.repeat(v_scale[blocks, h].astype(np.float64), p)[:length]
            for i in range(a, b):
                at = np.flatnonzero(seen[r][i - a])
                if not len(at):
                    continue
                mine = slice(h * group, (h + 1) * group)
                with np.errstate(invalid="ignore"):
                    z = softmax_scale * q[i, mine] @ k[at].T
                    zabs = softmax_scale * np.abs(q[i, mine]) @ np.abs(k[at]).T
                    m = z.max(1, keepdims=True)
                    e = np.exp(z - m)
                    l = e.sum(1, keepdims=True)
                    w, v, n = e / l, c[at] * sv[at, None], len(at)
                    dz = (d + 8) * 2.0 ** -24 * zabs.max(1, keepdims=True)
                    out[i, mine] = w @ v
                    lse[i, mine] = (m + np.log(l))[:, 0]
                    tol[i, mine] = (w @ np.abs(v) * (2.0 ** -11 + 2 * dz + n * 2.0 ** -23 + 2.0 ** -20)
                                    + 2.0 ** -25 * np.abs(c[at]).sum(0) * sv[at].max())
                    lse_tol[i, mine] = (dz + n * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(m + np.log(l)))[:, 0]
    return out, lse, tol, lse_tol
