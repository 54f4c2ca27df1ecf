"""Plain float64 restatement of rotary positions with several axes and of the
8-bit key/value cache: blocks and slots, appending rows, attention.

Loops over sequences, heads and blocks; no code of the library. A cache is kept
as numbers: `codes` (n_blocks, h, block_tokens, d) holds the values of the
e4m3 numbers (not their bytes), `scale` (n_blocks, h) their scales.
"""

import math

import numpy as np

E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

def rotary_frequencies(sections, base=10000.0, per_axis=False):
    """Radians per position of every pair."""
    P = sum(sections)
    if per_axis:
        return [base ** (-j / m) for m in sections for j in range(m)]
    return [base ** (-i / P) for i in range(P)]


def rotary(X, positions, frequencies, sections, interleaved=False, inverse=False):
    """X (B, h, T, d), positions (n_axes, B, T): pair i of each row turned by
    positions[axis(i)] * frequencies[i], or by the opposite angle."""
    Y = np.array(X, dtype=np.float64)
    P = sum(sections)
    axis = [a for a, m in enumerate(sections) for _ in range(m)]
    for i in range(P):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + P)
        theta = positions[axis[i]].astype(np.float64) * frequencies[i]
        if inverse:
            theta = -theta
        c, s = np.cos(theta)[:, None, :], np.sin(theta)[:, None, :]
        x, y = np.float64(X[..., a]), np.float64(X[..., b])
        Y[..., a], Y[..., b] = x * c - y * s, x * s + y * c
    return Y


# ---------------------------------------------------------------------------
# Blocks and slots
# ---------------------------------------------------------------------------

def reserve(cached_len, new_len, free_blocks, n_free, table, block_tokens, n):
    """One sequence after the other takes the blocks that it needs from the top
    of the free stack. Returns (total_len, slot_map, n_free, table, full, bad)."""
    table = np.array(table)
    total, slots = [], np.full((len(cached_len), n), -1, dtype=np.int64)
    full = bad = False
    asked = 0  # blocks asked for so far, by those that got none as well
    left = n_free
    for b, (L, a) in enumerate(zip(cached_len, new_len)):
        if L < 0 or a < 0 or a > n or L + a > table.shape[1] * block_tokens:
            bad = True
            total.append(L)
            continue
        have, want = -(-L // block_tokens), -(-(L + a) // block_tokens)
        asked += want - have
        if want > have and asked > n_free:
            full = True
            total.append(L)
            continue
        for j in range(have, want):
            left -= 1
            table[b, j] = free_blocks[left]
        for i in range(a):
            p = L + i
            slots[b, i] = int(table[b, p // block_tokens]) * block_tokens + p % block_tokens
        total.append(L + a)
    return total, slots, left, table, full, bad


def release(cached_len, finished, free_blocks, n_free, table, block_tokens):
    free = list(free_blocks[:n_free])
    total = []
    for b, (L, f) in enumerate(zip(cached_len, finished)):
        if f:
            free += [int(x) for x in table[b][:-(-L // block_tokens)]]
        total.append(0 if f else L)
    return total, free


# ---------------------------------------------------------------------------
# e4m3 and the cache
# ---------------------------------------------------------------------------

def e4m3_value(byte):
    """Sign, 4 exponent bits of bias 7, 3 mantissa bits; 0x7f is NaN."""
    e, m = byte >> 3 & 15, byte & 7
    if e == 15 and m == 7:
        return math.nan
    v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -v if byte & 128 else v


E4M3 = np.array([e4m3_value(c) for c in range(256)])


def e4m3_round(x):
    """The nearest e4m3 number, ties to the even mantissa; beyond 448 to 448."""
    x = np.asarray(x, dtype=np.float64)
    e = np.maximum(np.frexp(np.abs(x))[1] - 1, -6)
    step = np.ldexp(1.0, e - 3)
    with np.errstate(invalid="ignore"):
        return np.clip(np.where(np.isinf(x), x, np.round(x / step) * step), -E4M3_MAX, E4M3_MAX)


def block_scale(rows):
    """The smallest power of two s >= 2^-126 with |x| <= 448 s for every finite x."""
    a = np.abs(rows[np.isfinite(rows)])
    top = a.max() if a.size else 0.0
    s = 2.0 ** -126
    while s * E4M3_MAX < top:
        s *= 2
    return s


def append(X, slots, codes, scale, block_tokens):
    """Rows X (B, h, n, d) into the slots (B, n); codes and scale in place."""
    B, h, n, _ = X.shape
    for b in range(B):
        i = 0
        while i < n and slots[b, i] >= 0:
            block, o = divmod(int(slots[b, i]), block_tokens)
            m = 1
            while o + m < block_tokens and i + m < n and slots[b, i + m] == slots[b, i] + m:
                m += 1
            for j in range(h):
                rows = np.float64(X[b, j, i:i + m])
                s = block_scale(rows)
                if o:
                    old = scale[block, j]
                    s = max(s, old)
                    if s > old:
                        codes[block, j, :o] = e4m3_round(codes[block, j, :o] * (old / s))
                codes[block, j, o:o + m] = e4m3_round(rows / s)
                scale[block, j] = s
            i += m


def cache_rows(codes, scale, blocks, total, head, block_tokens):
    """The first `total` rows of a sequence with these blocks, of one head."""
    rows = [codes[blocks[p // block_tokens], head, p % block_tokens]
            * scale[blocks[p // block_tokens], head] for p in range(total)]
    return np.array(rows).reshape(total, codes.shape[3])


def attention_cache(Q, K_codes, V_codes, K_scale, V_scale, table, total, new, c, causal_tail):
    """Z (B, n_q, h d_vh), and a tuple of what error bounds are made of, each of
    Z's shape: A, the same sums with |v| for v; S, per row, the largest
    c sum |q| |k|; N, the sums of |v| over the keys seen, without weights; T, per
    row, the largest c max |q| sum |k|."""
    B, h, n_q, _ = Q.shape
    h_kv, bt, d_vh = V_codes.shape[1], V_codes.shape[2], V_codes.shape[3]
    Z = np.zeros((B, n_q, h, d_vh))
    A = np.zeros((B, n_q, h, d_vh))
    S = np.zeros((B, n_q, h, 1))
    N = np.zeros((B, n_q, h, d_vh))
    T = np.zeros((B, n_q, h, 1))
    for b in range(B):
        for kv in range(h_kv):
            if total[b] <= 0 or new[b] <= 0:
                continue
            K = cache_rows(K_codes, K_scale, table[b], total[b], kv, bt)
            V = cache_rows(V_codes, V_scale, table[b], total[b], kv, bt)
            for j in range(kv * (h // h_kv), (kv + 1) * (h // h_kv)):
                for i in range(new[b]):
                    seen = total[b] - new[b] + i + 1 if causal_tail else total[b]
                    if seen <= 0:
                        continue
                    q = np.float64(Q[b, j, i])
                    s = c * (K[:seen] @ q)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    Z[b, i, j] = p @ V[:seen]
                    A[b, i, j] = p @ np.abs(V[:seen])
                    N[b, i, j] = np.abs(V[:seen]).sum(axis=0)
                    S[b, i, j] = abs(c) * (np.abs(K[:seen]) @ np.abs(q)).max()
                    T[b, i, j] = abs(c) * np.abs(q).max() * np.abs(K[:seen]).sum(axis=1).max()
    flat = lambda x: x.reshape(B, n_q, -1)
    wide = lambda x: flat(np.repeat(x, d_vh, axis=3))
    return flat(Z), (flat(A), wide(S), flat(N), wide(T))
