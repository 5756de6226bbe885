"""64-bit definitions of the paged-cache operators, token by token with numpy:
what the CUDA results are compared with.  It shares no code with the library."""
import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative
HALF_STEP = {"f32": U, "bf16": 2.0 ** -8}


def rope_table(positions, rot, base):
    p = np.arange(positions, dtype=np.float64)[:, None]
    angle = p * base ** (-2.0 * np.arange(rot // 2) / rot)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1)


def rotate(x, row, rot, interleaved):
    """x: heads x D, row: the table's row of the position."""
    y = x.copy()
    c, s = row[: rot // 2], row[rot // 2:]
    j = np.arange(rot // 2)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
    y[:, a] = x[:, a] * c - x[:, b] * s
    y[:, b] = x[:, b] * c + x[:, a] * s
    return y


def tokens_of(lengths, counts, starts):
    """(token, sequence, position) of every new token."""
    for b, (n, start) in enumerate(zip(counts, starts)):
        for i in range(n):
            yield start + i, b, int(lengths[b]) - n + i


def append(k, v, k_cache, v_cache, table, lengths, counts, starts, rope, rot, interleaved, q=None):
    """New caches and rotated queries (rows of no token: NaN)."""
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    pages, size = k_cache.shape[:2]
    q_out = None if q is None else np.full(q.shape, np.nan)
    for t, b, p in tokens_of(lengths, counts, starts):
        row = rope[min(max(p, 0), rope.shape[0] - 1)] if rot else None
        turn = (lambda x: rotate(x, row, rot, interleaved)) if rot else (lambda x: x)
        if q is not None:
            q_out[t] = turn(q[t])
        if 0 <= p < table.shape[1] * size and 0 <= table[b, p // size] < pages:
            k_cache[table[b, p // size], p % size] = turn(k[t])
            v_cache[table[b, p // size], p % size] = v[t]
    return k_cache, v_cache, q_out


def attention(q, k_cache, v_cache, table, lengths, counts, starts, scale, causal=True, window=0, dtype="f32"):
    """(out, bound): the result (rows of no token: NaN) and how far off each
    element may be.

    A score is a sum of D products: off by at most (D + 2) steps of fp32 of the
    sum of their sizes, twice that for sums that cut off instead of rounding.  The
    exponent adds its own rounding (relative 2 U of its size and of the largest
    score, twice) and 2^-22 for the power of two.  Numerator and sum together
    are off by twice that; sums of n terms add (n + 8) U.  bf16 weights add a half
    step each, and the output its own."""
    T, H, D = q.shape
    size, G = k_cache.shape[1], H // k_cache.shape[2]
    out, bound = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    step = HALF_STEP[dtype]
    with np.errstate(invalid="ignore", over="ignore"):
        for t, b, p in tokens_of(lengths, counts, starts):
            stop = min(int(lengths[b]), table.shape[1] * size)
            hi = min(stop, p + 1) if causal else stop
            j = np.arange(max(p - window + 1, 0) if window else 0, max(hi, 0))
            page = np.clip(table[b, j // size], 0, k_cache.shape[0] - 1)
            for h in range(H):
                K, V = k_cache[page, j % size, h // G], v_cache[page, j % size, h // G]
                x = scale * (K @ q[t, h])
                if j.size == 0 or np.all(x == -np.inf):
                    out[t, h], bound[t, h] = 0.0, 0.0
                    continue
                w = np.exp(x - x.max())
                w /= w.sum()
                out[t, h] = w @ V
                size_of = scale * (np.abs(K) @ np.abs(q[t, h])).max()
                x = x[np.isfinite(x)]
                ds = 2 * (D + 2) * U * size_of + 4 * U * (np.abs(x).max() + np.ptp(x)) + 2.0 ** -22 if x.size else 0.0
                rel = 2 * ds + (j.size + 8) * U + (step if dtype == "bf16" else 0.0)
                bound[t, h] = 1.01 * rel * (w @ np.abs(V)) + step * np.abs(out[t, h])
    return out, bound
