"""64-bit definitions of the sparse-attention operators, entry by entry with
numpy: what the CUDA results are compared with.  It shares no code with the
library."""
import math

import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative


def rows_of(ro):
    return np.repeat(np.arange(ro.size - 1), np.diff(ro))


def blocks_of(M, seg_rows):
    return M if seg_rows <= 0 or seg_rows > M else seg_rows


def head_of_rows(M, seg_rows, heads):
    return np.arange(M) // blocks_of(M, seg_rows) % heads


def log_bucket(d, num_buckets, max_distance, causal):
    """Bucket of relative position d, with the boundaries found by comparing
    whole numbers: n lies in bucket e + i or above once (n/e)^(b-e) >=
    (max_distance/e)^i, that is n^(b-e) * e^i >= max_distance^i * e^(b-e)."""
    b = num_buckets if causal else num_buckets // 2
    n = max(-d, 0) if causal else abs(d)
    e = b // 2
    k = n
    if n >= e:
        k, w = e, b - e
        while k + 1 < b and n ** w * e ** (k + 1 - e) >= max_distance ** (k + 1 - e) * e ** w:
            k += 1
    return k + (b if not causal and d > 0 else 0)


def bucket_of_entries(ro, ci, bucket_map, seg_rows, seg_cols, q_offset, buckets):
    M = ro.size - 1
    seg = blocks_of(M, seg_rows)
    reach = (bucket_map.size - 1) // 2
    out = np.zeros(ci.size, dtype=np.int64)
    for r in range(M):
        s, e = int(ro[r]), int(ro[r + 1])
        if s == e:
            continue
        query = r % seg + (0 if q_offset is None else int(q_offset[r // seg]))
        start = int(ci[s]) // seg_cols * seg_cols if seg_cols > 0 else 0
        d = np.clip(ci[s:e].astype(np.int64) - start - query, -reach, reach)
        out[s:e] = np.clip(bucket_map[d + reach], 0, buckets - 1)
    return out


def row_softmax(ro, scores):
    """Softmax of each row; rows that hold only -inf are zero."""
    out = np.zeros(scores.size)
    with np.errstate(invalid="ignore"):
        for s, e in zip(ro[:-1], ro[1:]):
            x = scores[s:e].astype(np.float64)
            if x.size and not np.all(x == -np.inf):
                w = np.exp(x - x.max())
                out[s:e] = w / w.sum()
    return out


def row_dot(ro, p, d, masked):
    """Each row's sum of p*d over the entries that are not masked."""
    x = np.where(masked, 0.0, p * np.where(masked, 0.0, d))
    return np.array([x[s:e].sum() for s, e in zip(ro[:-1], ro[1:])])


def softmax_grad(ro, scores, dout):
    p, r = row_softmax(ro, scores), rows_of(ro)
    masked = scores == -np.inf
    c = row_dot(ro, p, dout, masked)
    return np.where(masked, 0.0, p * np.where(masked, 0.0, dout - c[r])), p, c


def diff_map(ro, s1, s2, lam_rows):
    return row_softmax(ro, s1) - lam_rows[rows_of(ro)] * row_softmax(ro, s2)


def diff_grad(ro, s1, s2, lam_rows, dout, heads, head_rows):
    r = rows_of(ro)
    g1, p1, c1 = softmax_grad(ro, s1, dout)
    g2, p2, c2 = softmax_grad(ro, s2, dout)
    dlam = -np.bincount(head_rows, c2, heads)
    return g1, -lam_rows[r] * g2, dlam


def attention(ro, ci, maps, V, scale, lam_rows, bias=None):
    """maps: one or two (Q, K) pairs."""
    out = np.zeros((ro.size - 1, V.shape[1]))
    for i in range(ro.size - 1):
        s, e = int(ro[i]), int(ro[i + 1])
        if s == e:
            continue
        keys, p, used = ci[s:e], 0.0, np.zeros(e - s, dtype=bool)
        for (Q, K), w in zip(maps, (1.0, -lam_rows[i])):
            x = scale * (K[keys] @ Q[i]) + (0.0 if bias is None else bias[s:e])
            used |= x != -np.inf
            p = p + w * row_softmax(np.array([0, e - s]), x)
        out[i] = np.where(used, p, 0.0) @ np.where(used[:, None], V[keys], 0.0)
    return out


def softmax_error(longest, spread):
    """Bound of a probability's relative error in fp32 for rows of at most
    `longest` entries whose scores lie within `spread` of their maximum: the
    exponential (CUDA's documented 2 + 1.17|x| steps of 2^-23), the rounding of
    s - m (spread * U), twice (numerator and sum), the sum's additions in any
    order of lanes (longest/32 + 16 along a path) and reciprocal and product."""
    one = (2 + 1.17 * spread) * 2 * U + spread * U
    return 2 * one + (longest / 32 + 16 + 4) * U


def bf16_half_step(x, dtype):
    return np.abs(x) * (2.0 ** -8 if dtype == "bf16" else 0.0)
