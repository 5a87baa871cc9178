"""The 8-bit key/value cache in 64 bits, on the CPU with numpy: block tables and slots one by one, the
append rule on exact values, attention by its formula.  Shares nothing with the library."""
import numpy as np

MAX = {0: 448.0, 1: 57344.0}          # E4M3, E5M2
MANTISSA = {0: 3, 1: 2}
LOWEST = {0: -6, 1: -14}              # exponent of the smallest normal


def decode_table(elem):
    """The 256 values of the format's codes (NaN and, for E5M2, infinities included)."""
    m, out = MANTISSA[elem], np.empty(256)
    bias = 7 if elem == 0 else 15
    for c in range(256):
        sign = -1.0 if c & 0x80 else 1.0
        e, f = (c & 0x7F) >> m, c & ((1 << m) - 1)
        if elem == 0 and (c & 0x7F) == 0x7F:
            out[c] = np.nan
        elif elem == 1 and e == 31:
            out[c] = np.nan if f else sign * np.inf
        elif e == 0:
            out[c] = sign * f * 2.0 ** (1 - bias - m)
        else:
            out[c] = sign * (1 + f / (1 << m)) * 2.0 ** (e - bias)
    return out


def encode(x, elem):
    """Codes of x: nearest, ties to even, saturating, NaN -> 0x7F."""
    x = np.asarray(x, np.float64)
    m, nan = MANTISSA[elem], np.isnan(x)
    a = np.minimum(np.abs(np.where(nan, 0.0, x)), MAX[elem])
    e = np.maximum(np.frexp(a)[1] - 1, LOWEST[elem])
    n = np.rint(a / 2.0 ** (e - m))                    # in units of the binade's step
    up = n >= 2 ** (m + 1)
    n, e = np.where(up, n / 2, n), np.where(up, e + 1, e)
    over = n * 2.0 ** (e - m) > MAX[elem]
    code = np.where(n >= 2 ** m, ((e - LOWEST[elem] + 1) << m) + n.astype(np.int64) - 2 ** m, n.astype(np.int64))
    assert not over.any()
    code = code + np.where(np.signbit(x), 0x80, 0)
    return np.where(nan, 0x7F, code).astype(np.uint8)


def scale_for(x, elem):
    """The scale of a block with values x."""
    x = np.abs(np.asarray(x, np.float64))
    amax = np.max(np.where(np.isfinite(x), x, 0.0), initial=0.0)
    if amax == 0:
        return 1.0
    k = -48
    while k < 48 and MAX[elem] * 2.0 ** k < amax:
        k += 1
    return 2.0 ** k


def tables(block_tables, before, after, free_list, count, num_tokens, p):
    """(tables, free list, q_start, slots, positions, info), one block and one token at a time."""
    t, free = block_tables.copy(), free_list.copy()
    stack = list(free[:count])
    ceil = lambda n: -(-int(n) // p)  # noqa: E731
    for r in range(len(before)):
        for b in range(ceil(after[r]), ceil(before[r])):
            stack.append(t[r, b])
    new = [max(int(b) - int(a), 0) for a, b in zip(before, after)]
    q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    slots, positions = np.full(num_tokens, -1, np.int64), np.full(num_tokens, -1, np.int32)
    need = sum(max(ceil(b) - ceil(a), 0) for a, b in zip(before, after))
    if need > len(stack):
        return t, free, q_start, slots, positions, np.array([count, need - len(stack)], np.int32)
    for r in range(len(before)):
        for b in range(ceil(before[r]), ceil(after[r])):
            t[r, b] = stack.pop()
    free[:len(stack)] = stack
    i = 0
    for r in range(len(before)):
        for pos in range(int(before[r]), int(after[r])):
            slots[i], positions[i] = int(t[r, pos // p]) * p + pos % p, pos
            i += 1
    return t, free, q_start, slots, positions, np.array([len(stack), 0], np.int32)


def append(x, slots, codes, scale, elem):
    """(codes, scale) after x [tokens][kv heads][D] was written at slots."""
    codes, scale = codes.copy(), scale.astype(np.float64)
    table, p = decode_table(elem), codes.shape[2]
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == slots[t] + n and slots[t + n] % p:
            n += 1
        block, off = divmod(int(slots[t]), p)
        for h in range(x.shape[1]):
            new = x[t:t + n, h].astype(np.float64)
            s = scale_for(new, elem)
            if off:
                some = np.any(np.isfinite(new) & (new != 0))
                s = max(s, scale[block, h]) if some else scale[block, h]
                if s != scale[block, h]:
                    codes[block, h, :off] = encode(table[codes[block, h, :off]] * (scale[block, h] / s), elem)
            codes[block, h, off:off + n] = encode(new / s, elem)
            scale[block, h] = s
        t += n
    return codes, scale.astype(np.float32)


def attention(q, k_codes, v_codes, k_scale, v_scale, block_tables, lengths, q_start, elem, softmax_scale, causal, window):
    """(out, lse, out's tolerance but for the output's own rounding, lse's tolerance), in 64 bits.

    Tolerances, for a kernel with FP32 sums, FP16 weights and a softmax reference within 2^8 of the
    maximum: an FP32 score of magnitude Z = scale * sum |q k| is off by dz <= (D + 8) 2^-24 Z, a weight
    by the factor exp(+-dz), its rounding to FP16 by 2^-11 (normal) or 2^-25 of the reference
    (subnormal), sums over n weights by n 2^-24.  So out is off by at most
    A (2^-11 + 2 dz + n 2^-23 + 2^-20) + 2^-25 sum |code_j| max s_V, A = sum w |v|."""
    table, p = decode_table(elem), k_codes.shape[2]
    t, heads, d = q.shape
    group = heads // k_codes.shape[1]
    out, lse = np.zeros((t, heads, d)), np.full((t, heads), -np.inf)
    tol, lse_tol = np.zeros((t, heads, d)), np.zeros((t, heads))
    q = q.astype(np.float64)
    for r, length in enumerate(lengths):
        a, b = int(q_start[r]), int(q_start[r + 1])
        if length == 0 or a == b:
            continue
        blocks = block_tables[r, :-(-int(length) // p)]
        for h in range(k_codes.shape[1]):
            k = (table[k_codes[blocks, h]] * k_scale[blocks, h].astype(np.float64)[:, None, None]).reshape(-1, d)[:length]
            c = table[v_codes[blocks, h]].reshape(-1, d)[:length]
            sv = np.repeat(v_scale[blocks, h].astype(np.float64), p)[:length]
            for i in range(a, b):
                pos = int(length) - (b - i)
                lo = max(0, pos - window + 1) if window else 0
                hi = min(int(length), pos + 1) if causal else int(length)
                if hi <= lo:
                    continue
                with np.errstate(invalid="ignore"):
                    qs = q[i, h * group:(h + 1) * group]
                    z = softmax_scale * qs @ k[lo:hi].T
                    zabs = softmax_scale * np.abs(qs) @ np.abs(k[lo:hi]).T
                    m = z.max(1, keepdims=True)
                    e = np.exp(z - m)
                    l = e.sum(1, keepdims=True)
                    w, v, n = e / l, c[lo:hi] * sv[lo:hi, None], hi - lo
                    o = w @ v
                    dz = (d + 8) * 2.0 ** -24 * zabs.max(1, keepdims=True)
                    out[i, h * group:(h + 1) * group] = o
                    lse[i, h * group:(h + 1) * group] = (m + np.log(l))[:, 0]
                    tol[i, h * group:(h + 1) * group] = (
                        w @ np.abs(v) * (2.0 ** -11 + 2 * dz + n * 2.0 ** -23 + 2.0 ** -20)
                        + 2.0 ** -25 * np.abs(c[lo:hi]).sum(0) * sv[lo:hi].max())
                    lse_tol[i, h * group:(h + 1) * group] = (
                        dz + n * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(m + np.log(l)))[:, 0]
    return out, lse, tol, lse_tol
