"""Sparse-attention operators on the GPU against their 64-bit definitions
(attention_ref): position bias and its gradient, differential map and its
gradients, softmax gradient, attention of few rows, and the chain they form
with the SDDMM, SpMM and transpose."""
import numpy as np
import pytest

import attention_ref as R
import workloads as W
from parity_util import dev, host

pytestmark = pytest.mark.gpu

U = R.U


def masks():
    """name -> (row lengths, columns of a block, seg_rows).  Rows of no entry,
    of one, around the sizes at which kernels change form, and far longer than
    the others; M is not always a multiple of seg_rows (a last, shorter block)."""
    rng = np.random.default_rng(3)
    ragged = rng.integers(0, 90, 203)
    ragged[::7] = 0
    sizes = np.array([0, 1, 2, 3, 4, 5, 31, 32, 33, 127, 128, 129, 511, 512, 513, 1023, 1024, 1025, 2047, 2048, 2049,
                      4095, 4096, 4097, 0, 8191, 8192, 8193, 9000])
    return {
        "single": (np.array([1]), 1, 1),
        "ragged": (ragged, 96, 29),
        "sizes": (sizes, 9000, 3),
        "one_long": (np.array([40001]), 50000, 1),
        "skewed": (np.concatenate([rng.integers(1, 20, 700), [20000], rng.integers(1, 20, 300)]), 20000, 0),
        "tokens": (rng.integers(0, 400, 24), 512, 1),
        "long_tokens": (rng.integers(5000, 12000, 6), 16384, 1),
    }


MASKS = masks()
HEADS = 3


def make(name):
    lengths, cols, seg = MASKS[name]
    rng = np.random.default_rng([11, sorted(MASKS).index(name)])
    M = lengths.size
    segr = R.blocks_of(M, seg)
    base = np.arange(M) // segr * cols
    ro, ci = W.csr_from_lengths(rng, lengths.astype(np.int64), cols, base)
    blocks = -(-M // segr)
    return dict(rng=rng, ro=ro, ci=ci, M=M, K=blocks * cols, cols=cols, seg=seg, blocks=blocks, nnz=ci.size,
                heads=R.head_of_rows(M, seg, HEADS), longest=int(lengths.max()))


def shifted(x, dtype="f32"):
    """A device copy whose data starts one element past a 16-byte boundary."""
    import torch
    t = dev(x, dtype)
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    buf[1:] = t
    return buf[1:]


def rounded(x, dtype):
    """fp32 values as the given type holds them."""
    x = x.astype(np.float32)
    return W.bf16_bits_to_f32(W.f32_to_bf16_bits(x)) if dtype == "bf16" else x


def put(x, dtype="f32", aligned=True):
    x = x.astype(np.float32)
    bits = W.f32_to_bf16_bits(x) if dtype == "bf16" else x
    return dev(bits, dtype) if aligned else shifted(bits, dtype)


def got(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


def scores_of(p, rng, masked=True):
    """Scores in [-8, 8], some -inf, and one row wholly -inf."""
    s = np.clip(2.5 * rng.standard_normal(p["nnz"]), -8, 8).astype(np.float32)
    if masked and p["nnz"] > 8:
        s[rng.random(s.size) < 0.05] = -np.inf
        whole = int(np.argmax(np.diff(p["ro"]) > 1))
        s[p["ro"][whole]:p["ro"][whole + 1]] = -np.inf
    return s


SPREAD = 16.0  # the largest distance of a score from its row's maximum


def assert_near(x, ref, bound, what):
    assert x.shape == ref.shape, (what, x.shape, ref.shape)
    bad = ~(np.abs(x - ref) <= bound)
    if bad.any():
        i = int(np.flatnonzero(bad.ravel())[0])
        b = np.broadcast_to(bound, ref.shape).ravel()[i]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: {x.ravel()[i]!r} against "
                             f"{ref.ravel()[i]!r}, bound {b!r}")


# ---------------------------------------------------------------------------
# Position bias
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("buckets,reach,causal", [(32, 128, False), (32, 128, True), (2, 3, True), (4, 2, False),
                                                  (33, 77, True), (64, 8192, False), (256, 4096, True)])
def test_bucket_map(usm, buckets, reach, causal):
    m = host(usm.rel_bucket_map(buckets, reach, causal))
    step = 1 if reach < 1000 else 37
    at = np.arange(0, 2 * reach + 1, step)
    want = np.array([R.log_bucket(int(d) - reach, buckets, reach, causal) for d in at])
    assert np.array_equal(m[at], want)


def bias_inputs(p, buckets=12, reach=40):
    rng = p["rng"]
    bmap = rng.integers(-2, buckets + 2, 2 * reach + 1).astype(np.int32)  # some outside [0, buckets): clamped
    q_offset = rng.integers(-50, p["cols"] + 50, p["blocks"]).astype(np.int32)
    return bmap, q_offset, rng.standard_normal((HEADS, buckets)).astype(np.float32)


@pytest.mark.parametrize("name", sorted(MASKS))
@pytest.mark.parametrize("table_dtype,offset,aligned", [("f32", True, True), ("bf16", False, False)])
def test_rel_bias(usm, name, table_dtype, offset, aligned):
    p = make(name)
    bmap, q_offset, table = bias_inputs(p)
    q_offset = q_offset if offset else None
    scores = scores_of(p, p["rng"])
    table = rounded(table, table_dtype)
    k = R.bucket_of_entries(p["ro"], p["ci"], bmap, p["seg"], p["cols"], q_offset, table.shape[1])
    want = scores + table[p["heads"][R.rows_of(p["ro"])], k]  # one fp32 addition: the same bits
    sd = put(scores, aligned=aligned)
    args = (dev(p["ro"]), dev(p["ci"]), sd, put(table, table_dtype), dev(bmap))
    kw = dict(seg_rows=p["seg"], seg_cols=p["cols"], q_offset=None if q_offset is None else dev(q_offset))
    out = usm.rel_bias(*args, **kw)
    assert np.array_equal(host(out), want)
    assert usm.rel_bias(*args, out=sd, **kw) is sd  # in place
    assert np.array_equal(host(sd), want)


def test_rel_bias_far_offsets(usm):
    """Query offsets at both ends of 32 bits clip to the ends of the map."""
    ro, ci = np.array([0, 2, 4], dtype=np.int32), np.array([0, 9, 10, 19], dtype=np.int32)
    bmap = np.arange(7, dtype=np.int32)
    table = np.arange(7, dtype=np.float32)[None]
    out = usm.rel_bias(dev(ro), dev(ci), put(np.zeros(4)), put(table), dev(bmap), seg_rows=1, seg_cols=10,
                       q_offset=dev(np.array([2**31 - 1, -2**31], dtype=np.int32)))
    assert np.array_equal(host(out), np.array([0, 0, 6, 6], dtype=np.float32))


@pytest.mark.parametrize("name", sorted(MASKS))
@pytest.mark.parametrize("dtype,aligned", [("f32", True), ("bf16", False)])
def test_rel_bias_grad(usm, name, dtype, aligned):
    p = make(name)
    bmap, q_offset, table = bias_inputs(p)
    k = R.bucket_of_entries(p["ro"], p["ci"], bmap, p["seg"], p["cols"], q_offset, table.shape[1])
    flat = p["heads"][R.rows_of(p["ro"])] * table.shape[1] + k
    count = np.bincount(flat, minlength=table.size).reshape(table.shape)
    args = (dev(p["ro"]), dev(p["ci"]))
    kw = dict(seg_rows=p["seg"], seg_cols=p["cols"], q_offset=dev(q_offset))
    # Whole numbers below 2^24 in sum: exact in any order.
    ds = p["rng"].integers(-8, 9, p["nnz"]).astype(np.float32)
    want = np.bincount(flat, ds, table.size).reshape(table.shape)
    out = usm.rel_bias_grad(*args, put(ds, dtype, aligned), *table.shape, dev(bmap), **kw)
    assert np.array_equal(got(out), want)
    # Real ones: n - 1 additions of relative error U each at most.
    ds = rounded(p["rng"].standard_normal(p["nnz"]), dtype)
    want = np.bincount(flat, ds, table.size).reshape(table.shape)
    size = np.bincount(flat, np.abs(ds), table.size).reshape(table.shape)
    dsd = put(ds, dtype, aligned)
    out = usm.rel_bias_grad(*args, dsd, *table.shape, dev(bmap), **kw)
    assert_near(got(out), want, count * U * size, "dtable")
    again = usm.rel_bias_grad(*args, dsd, *table.shape, dev(bmap), **kw)
    assert np.array_equal(host(out), host(again))


@pytest.mark.parametrize("heads,buckets", [(1, 1), (7, 512), (64, 32)])
def test_rel_bias_grad_sizes(usm, heads, buckets):
    """One bucket, the most buckets, and more heads than blocks (zero rows of
    the table for the heads that have none)."""
    rng = np.random.default_rng(5)
    csr = W.random_csr([heads, buckets], 60, 300, 0.3)
    bmap = (np.arange(2 * 300 + 1) % buckets).astype(np.int32)
    ds = rng.integers(-8, 9, csr.nnz).astype(np.float32)
    k = R.bucket_of_entries(csr.row_offsets, csr.col_indices, bmap, 20, 300, None, buckets)
    flat = R.head_of_rows(60, 20, heads)[R.rows_of(csr.row_offsets)] * buckets + k
    out = usm.rel_bias_grad(dev(csr.row_offsets), dev(csr.col_indices), put(ds), heads, buckets, dev(bmap), seg_rows=20,
                            seg_cols=300)
    assert np.array_equal(got(out).ravel(), np.bincount(flat, ds, heads * buckets))


def test_empty_masks(usm):
    """No entries at all: nothing but the reductions is written, with zeros."""
    import torch
    ro, none = dev(np.zeros(9, dtype=np.int32)), torch.empty(0, device="cuda")
    ci = torch.empty(0, dtype=torch.int32, device="cuda")
    bmap, lam = dev(np.zeros(5, dtype=np.int32)), put(np.ones(2))
    assert usm.rel_bias(ro, ci, none, put(np.ones((2, 4))), bmap, seg_rows=4).numel() == 0
    assert np.array_equal(got(usm.rel_bias_grad(ro, ci, none, 2, 4, bmap, seg_rows=4)), np.zeros((2, 4)))
    assert usm.diff_softmax(ro, none, none, lam, seg_rows=4).numel() == 0
    assert np.array_equal(got(usm.diff_softmax_grad(ro, none, none, lam, none, seg_rows=4)[2]), np.zeros(2))
    assert usm.row_softmax_grad(ro, none, none).numel() == 0
    x = put(np.ones((8, 8)))
    assert np.array_equal(got(usm.attention(ro, ci, x, x, x)), np.zeros((8, 8)))


# ---------------------------------------------------------------------------
# Maps and their gradients
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("name", sorted(MASKS))
@pytest.mark.parametrize("dtype,aligned", [("f32", True), ("bf16", True), ("f32", False), ("bf16", False)])
def test_diff_softmax(usm, name, dtype, aligned):
    import torch
    p = make(name)
    s1, s2 = scores_of(p, p["rng"]), scores_of(p, p["rng"], masked=False)
    lam = p["rng"].uniform(0.1, 0.9, HEADS).astype(np.float32)
    lr = lam.astype(np.float64)[p["heads"]]
    want = R.diff_map(p["ro"], s1, s2, lr)
    r = R.rows_of(p["ro"])
    size = R.row_softmax(p["ro"], s1) + lr[r] * R.row_softmax(p["ro"], s2)
    tol = (R.softmax_error(p["longest"], SPREAD) + 2 * U) * size
    od = torch.bfloat16 if dtype == "bf16" else torch.float32
    out = usm.diff_softmax(dev(p["ro"]), put(s1, aligned=aligned), put(s2, aligned=aligned), put(lam), seg_rows=p["seg"],
                           out_dtype=od)
    assert out.dtype == od
    assert_near(got(out), want, tol + R.bf16_half_step(np.abs(want) + tol, dtype), "map")


def grad_bound(p, s, dout, weight):
    """Error bound of weight·P·(d - c) in fp32: P and c carry the softmax's
    relative error E, c the sum's too (its terms at most P|d|), and the
    difference and products a few roundings more."""
    E = R.softmax_error(p["longest"], SPREAD)
    prob, r = R.row_softmax(p["ro"], s), R.rows_of(p["ro"])
    masked = s == -np.inf
    cabs = R.row_dot(p["ro"], prob, np.abs(np.where(masked, 0, dout)), masked)
    return weight * prob * (np.abs(np.where(masked, 0, dout)) + cabs[r]) * (3 * E + 8 * U), cabs * (3 * E + 8 * U)


@pytest.mark.parametrize("name", sorted(MASKS))
@pytest.mark.parametrize("din,dtype,aligned", [("f32", "f32", True), ("f32", "bf16", True), ("bf16", "bf16", False),
                                               ("bf16", "f32", True), ("f32", "f32", False)])
def test_softmax_gradients(usm, name, din, dtype, aligned):
    import torch
    p = make(name)
    rng = p["rng"]
    s1, s2 = scores_of(p, rng), scores_of(p, rng)
    dout = rounded(rng.standard_normal(p["nnz"]), din)
    lam = rng.uniform(0.1, 0.9, HEADS).astype(np.float32)
    lr = lam.astype(np.float64)[p["heads"]]
    g1, g2, dlam = R.diff_grad(p["ro"], s1, s2, lr, dout, HEADS, p["heads"])
    od = torch.bfloat16 if dtype == "bf16" else torch.float32
    ro, a1, a2, ad = dev(p["ro"]), put(s1, aligned=aligned), put(s2, aligned=aligned), put(dout, din, aligned)
    o1, o2, ol = usm.diff_softmax_grad(ro, a1, a2, put(lam), ad, seg_rows=p["seg"], out_dtype=od)
    r = R.rows_of(p["ro"])
    t1, _ = grad_bound(p, s1, dout, 1.0)
    t2, c2 = grad_bound(p, s2, dout, lr[r])
    assert o1.dtype == od and o2.dtype == od
    assert_near(got(o1), g1, t1 + R.bf16_half_step(np.abs(g1) + t1, dtype), "dscores1")
    assert_near(got(o2), g2, t2 + R.bf16_half_step(np.abs(g2) + t2, dtype), "dscores2")
    # Each row's own error, and the sum over the rows in any order.
    rows = np.bincount(p["heads"], minlength=HEADS)
    size = np.bincount(p["heads"], np.abs(R.softmax_grad(p["ro"], s2, dout)[2]), HEADS)
    assert_near(got(ol), dlam, np.bincount(p["heads"], c2, HEADS) + rows * U * size, "dlambda")
    again = usm.diff_softmax_grad(ro, a1, a2, put(lam), ad, seg_rows=p["seg"], out_dtype=od)
    for x, y in zip((o1, o2, ol), again):
        assert torch.equal(x, y)
    g, _, _ = R.softmax_grad(p["ro"], s1, dout)
    o = usm.row_softmax_grad(ro, a1, ad, out_dtype=od)
    assert_near(got(o), g, t1 + R.bf16_half_step(np.abs(g) + t1, dtype), "softmax gradient")
    if dtype == "f32":  # in place
        x1, x2 = a1.clone(), a2.clone()
        usm.diff_softmax_grad(ro, x1, x2, put(lam), ad, seg_rows=p["seg"], out1=x1, out2=x2)
        assert torch.equal(x1, o1) and torch.equal(x2, o2)
        x1 = a1.clone()
        usm.row_softmax_grad(ro, x1, ad, out=x1)
        assert torch.equal(x1, o)


@pytest.mark.parametrize("name", ["ragged", "skewed", "long_tokens"])
def test_masked_entries_ignore_their_gradient(usm, name):
    """NaN and infinities in dout under -inf scores reach nothing."""
    import torch
    p = make(name)
    s1 = scores_of(p, p["rng"])
    dout = p["rng"].standard_normal(p["nnz"]).astype(np.float32)
    masked = s1 == -np.inf
    bad = dout.copy()
    bad[masked] = np.resize([np.nan, np.inf, -np.inf], int(masked.sum()))
    ro, a, lam = dev(p["ro"]), put(s1), put(np.full(HEADS, 0.5))
    assert torch.equal(usm.row_softmax_grad(ro, a, put(bad)), usm.row_softmax_grad(ro, a, put(np.where(masked, 0, dout))))
    x = usm.diff_softmax_grad(ro, a, a, lam, put(bad), seg_rows=p["seg"])
    y = usm.diff_softmax_grad(ro, a, a, lam, put(np.where(masked, 0, dout)), seg_rows=p["seg"])
    for u, v in zip(x, y):
        assert torch.equal(u, v) and torch.isfinite(u).all()


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("name", ["ragged", "skewed", "long_tokens"])
def test_non_finite_scores_stay_in_their_row(usm, name, value):
    p = make(name)
    s = scores_of(p, p["rng"], masked=False)
    rows = np.flatnonzero(np.diff(p["ro"]) > 2)
    row = int(rows[np.argmax(np.diff(p["ro"])[rows])])
    s[p["ro"][row] + 1] = value
    out = got(usm.diff_softmax(dev(p["ro"]), put(s), put(scores_of(p, p["rng"], masked=False)), put(np.full(HEADS, 0.5)),
                               seg_rows=p["seg"]))
    inside = np.zeros(p["nnz"], dtype=bool)
    inside[p["ro"][row]:p["ro"][row + 1]] = True
    assert np.isnan(out[inside]).all() and np.isfinite(out[~inside]).all()


def test_large_scores(usm):
    """Scores far from zero, the type's lowest value among them."""
    p = make("ragged")
    low = float(np.finfo(np.float32).min)
    s1 = (scores_of(p, p["rng"], masked=False) + 30000).astype(np.float32)
    s2 = scores_of(p, p["rng"], masked=False)
    s2[::3] = low
    row = int(np.argmax(np.diff(p["ro"]) > 3))
    s2[p["ro"][row]:p["ro"][row + 1]] = low  # a row of the lowest value only: uniform
    lam = np.full(HEADS, 0.5, dtype=np.float32)
    want = R.diff_map(p["ro"], s1, s2, lam.astype(np.float64)[p["heads"]])
    size = R.row_softmax(p["ro"], s1) + 0.5 * R.row_softmax(p["ro"], s2)
    out = usm.diff_softmax(dev(p["ro"]), put(s1), put(s2), put(lam), seg_rows=p["seg"])
    assert_near(got(out), want, (R.softmax_error(p["longest"], SPREAD) + 2 * U) * size, "map")


# ---------------------------------------------------------------------------
# Attention of few rows
# ---------------------------------------------------------------------------
def attention_bound(ro, ci, maps, V, scale, lam_rows, bias, longest):
    """Bound of the output's error.  A score is a sum of D products in fp32
    (D/8 + 16 additions along a path at most and one rounding a product), the
    scale and the bias: off by ds.  Weights are off by 2·ds and the softmax's
    error relative to themselves, and the weighted sum adds its roundings."""
    out = np.zeros((ro.size - 1, V.shape[1]))
    for i in range(ro.size - 1):
        s, e = int(ro[i]), int(ro[i + 1])
        if s == e:
            continue
        keys = ci[s:e]
        for (Q, K), w in zip(maps, (1.0, lam_rows[i])):
            size = scale * (np.abs(K[keys]) @ np.abs(Q[i]))
            x = scale * (K[keys] @ Q[i]) + (0.0 if bias is None else bias[s:e])
            ok = x != -np.inf
            if not ok.any():
                continue
            ds = np.max((Q.shape[1] / 8 + 20) * U * size + 4 * U * np.abs(np.where(ok, x, 0)))
            spread = np.ptp(x[ok])
            p = R.row_softmax(np.array([0, e - s]), x)
            E = 2 * ds + R.softmax_error(longest, spread) + (longest / 8 + 40) * U
            out[i] += w * E * 2 * (p @ np.abs(np.where(ok[:, None], V[keys], 0.0)))
    return out


def attention_case(p, D, N, maps, dtype, biased, std=1.0):
    rng = p["rng"]
    mat = lambda r, c: rounded(std * rng.standard_normal((r, c)), dtype)
    Qs, Ks = [mat(p["M"], D) for _ in range(maps)], [mat(p["K"], D) for _ in range(maps)]
    V = rounded(rng.standard_normal((p["K"], N)), dtype)
    lam = rng.uniform(0.2, 0.8, HEADS).astype(np.float32) if maps == 2 else None
    bias = entry = None
    if biased:
        bmap, q_offset, table = bias_inputs(p)
        table[0, 3] = -np.inf  # a bucket that masks
        k = R.bucket_of_entries(p["ro"], p["ci"], bmap, p["seg"], p["cols"], q_offset, table.shape[1])
        entry = table[p["heads"][R.rows_of(p["ro"])], k].astype(np.float64)
        bias = dict(table=put(table), bucket_map=dev(bmap), q_offset=dev(q_offset), seg_cols=p["cols"])
    return Qs, Ks, V, lam, bias, entry


def run_attention(usm, p, D, N, maps, dtype, biased, pad=False, std=1.0):
    import torch
    Qs, Ks, V, lam, bias, entry = attention_case(p, D, N, maps, dtype, biased, std)
    scale = D ** -0.5 if D else 1.0

    def place(x):
        t = put(x, dtype)
        if not pad:
            return t
        # Rows inside a wider buffer of NaN: nothing beyond the columns is used.
        ld = -(-x.shape[1] // 8) * 8 + 8
        buf = torch.full((x.shape[0], ld), float("nan"), dtype=t.dtype, device="cuda")
        buf[:, : x.shape[1]] = t
        return buf[:, : x.shape[1]]

    kw = dict(bias or {})
    if maps == 2:
        kw.update(Q2=place(Qs[1]), K2=place(Ks[1]), lam=put(lam))
    args = (dev(p["ro"]), dev(p["ci"]), place(Qs[0]), place(Ks[0]), place(V))
    out = usm.attention(*args, scale=scale, seg_rows=p["seg"], **kw)
    lr = np.zeros(p["M"]) if lam is None else lam.astype(np.float64)[p["heads"]]
    q64 = [(q.astype(np.float64), k.astype(np.float64)) for q, k in zip(Qs, Ks)]
    want = R.attention(p["ro"], p["ci"], q64, V.astype(np.float64), scale, lr, entry)
    tol = attention_bound(p["ro"], p["ci"], q64, V.astype(np.float64), scale, lr, entry, p["longest"])
    assert_near(got(out), want, tol, "attention")
    assert torch.equal(out, usm.attention(*args, scale=scale, seg_rows=p["seg"], **kw))


@pytest.mark.parametrize("name", sorted(MASKS))
@pytest.mark.parametrize("maps,dtype,biased", [(1, "bf16", False), (2, "bf16", True), (1, "f32", True), (2, "f32", False)])
def test_attention_masks(usm, name, maps, dtype, biased):
    run_attention(usm, make(name), 32, 64, maps, dtype, biased)


@pytest.mark.parametrize("D,N", [(1, 1), (7, 5), (8, 64), (64, 8), (33, 100), (64, 128), (128, 128), (130, 72), (96, 192),
                                 (256, 256), (0, 16)])
@pytest.mark.parametrize("maps,dtype", [(1, "bf16"), (2, "bf16"), (1, "f32"), (2, "f32")])
def test_attention_widths(usm, D, N, maps, dtype):
    for name in ("tokens", "ragged"):
        run_attention(usm, make(name), D, N, maps, dtype, name == "tokens", pad=True)


@pytest.mark.parametrize("D,N", [(512, 512), (260, 40), (16, 300)])
def test_attention_widest_bf16(usm, D, N):
    run_attention(usm, make("tokens"), D, N, 2, "bf16", True, pad=True)


def test_attention_shared_keys(usm):
    """Four query heads over one block of keys (columns shared by blocks)."""
    p = make("tokens")
    p["ci"] = (p["ci"] % p["cols"] + (R.rows_of(p["ro"]) // 4) * p["cols"]).astype(np.int32)
    p["K"] = 6 * p["cols"]
    run_attention(usm, p, 64, 64, 2, "bf16", True)


def test_attention_many_rows(usm):
    """More rows than a GPU holds at once."""
    rng = np.random.default_rng(9)
    lengths = rng.integers(0, 12, 5000)
    ro, ci = W.csr_from_lengths(rng, lengths.astype(np.int64), 64)
    p = dict(rng=rng, ro=ro, ci=ci, M=5000, K=64, cols=64, seg=0, blocks=1, nnz=ci.size,
             heads=np.zeros(5000, dtype=np.int64), longest=12)
    run_attention(usm, p, 16, 16, 2, "f32", False)


def test_attention_unused_values(usm):
    """Rows of V under entries that no map uses may hold anything."""
    import torch
    p = make("tokens")
    Qs, Ks, V, lam, bias, entry = attention_case(p, 32, 32, 2, "f32", True)
    unused = np.zeros(p["K"], dtype=bool)
    unused[p["ci"][entry == -np.inf]] = True
    unused[p["ci"][entry != -np.inf]] = False
    assert unused.any()
    bad = V.copy()
    bad[unused] = np.nan
    kw = dict(scale=0.2, seg_rows=p["seg"], Q2=put(Qs[1]), K2=put(Ks[1]), lam=put(lam), **bias)
    call = lambda v: usm.attention(dev(p["ro"]), dev(p["ci"]), put(Qs[0]), put(Ks[0]), put(v), **kw)
    x, y = call(V), call(bad)
    assert torch.isfinite(x).all() and torch.equal(x, y)


def test_attention_far_rows(usm):
    """Keys whose byte offsets pass 32 bits (a cache of 4.6 GB)."""
    import torch
    K, D = 36_000_000, 64
    Km = torch.zeros((K, D), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(2)
    ci = np.sort(rng.choice(np.arange(K - 4000, K), 50, replace=False)).astype(np.int32)
    rows = rounded(rng.standard_normal((50, D)), "bf16")
    Km[torch.from_numpy(ci).long().cuda()] = put(rows, "bf16")
    q = rounded(rng.standard_normal((1, D)), "bf16")
    ro = np.array([0, 50], dtype=np.int32)
    out = usm.attention(dev(ro), dev(ci), put(q, "bf16"), Km, Km, scale=0.125)
    local = np.arange(50, dtype=np.int32)
    q64, k64 = q.astype(np.float64), rows.astype(np.float64)
    want = R.attention(ro, local, [(q64, k64)], k64, 0.125, np.zeros(1))
    assert_near(got(out), want, attention_bound(ro, local, [(q64, k64)], k64, 0.125, np.zeros(1), None, 50), "far rows")


# ---------------------------------------------------------------------------
# Calls: refusals, streams, graphs
# ---------------------------------------------------------------------------
def test_binding_refusals(usm):
    import torch
    p = make("ragged")
    ro, ci, s = dev(p["ro"]), dev(p["ci"]), put(np.zeros(p["nnz"]))
    table, bmap, lam = put(np.zeros((HEADS, 4))), dev(np.zeros(5, dtype=np.int32)), put(np.zeros(HEADS))
    with pytest.raises(ValueError, match="elements"):
        usm.rel_bias(ro, ci, s[:-1], table, bmap)
    with pytest.raises(ValueError, match="contiguous"):
        usm.rel_bias(ro, ci, torch.zeros(2 * p["nnz"], device="cuda")[::2], table, bmap)
    with pytest.raises(ValueError, match="bucket_map"):
        usm.rel_bias(ro, ci, s, table, bmap[:4])
    with pytest.raises(ValueError, match="q_offset"):
        usm.rel_bias(ro, ci, s, table, bmap, seg_rows=p["seg"], q_offset=bmap[:1])
    with pytest.raises(TypeError):
        usm.rel_bias(ro, ci, s.half(), table, bmap)
    with pytest.raises(ValueError, match="CUDA"):
        usm.rel_bias(ro, ci, s.cpu(), table, bmap)
    with pytest.raises(ValueError, match="fit 32 bits"):
        usm.rel_bias(ro, ci, s, table, bmap, seg_rows=2**31)
    with pytest.raises(usm.USMError):
        usm.rel_bias_grad(ro, ci, s, 0, 4, bmap)
    with pytest.raises(ValueError):
        usm.diff_softmax(ro, s, s[:-1], lam)
    with pytest.raises(TypeError):
        usm.diff_softmax(ro, s, s, lam, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="come together"):
        usm.attention(ro, ci, put(np.zeros((p["M"], 8))), put(np.zeros((p["K"], 8))), put(np.zeros((p["K"], 8))), lam=lam)
    q, k = put(np.zeros((p["M"], 8))), put(np.zeros((p["K"], 8)))
    with pytest.raises(ValueError, match="expected"):
        usm.attention(ro, ci, q[:-1], k, k)
    with pytest.raises(ValueError, match="heads"):
        usm.attention(ro, ci, q, k, k, Q2=q, K2=k, lam=lam, table=table[:1].contiguous(), bucket_map=bmap)
    with pytest.raises(usm.USMError, match="UNSUPPORTED"):
        usm.attention(ro, ci, put(np.zeros((p["M"], 260))), put(np.zeros((p["K"], 260))), k)


def chain_inputs(dtype="f32"):
    p = make("ragged")
    rng = p["rng"]
    D = 24
    m = lambda r, c: rounded(rng.standard_normal((r, c)), dtype)
    x = dict(Q1=m(p["M"], D), Q2=m(p["M"], D), K1=m(p["K"], D), K2=m(p["K"], D), V=m(p["K"], 2 * D), dO=m(p["M"], 2 * D),
             table=rounded(rng.standard_normal((HEADS, 8)), "f32"), lam=rng.uniform(0.2, 0.8, HEADS).astype(np.float32))
    x["bmap"] = rng.integers(0, 8, 2 * 30 + 1).astype(np.int32)
    return p, x


def run_chain(usm, p, t, ro, ci, keep=None):
    """Forward and backward of differential attention with a position bias, as
    a training step calls it.  Q1 and Q2 carry the scale."""
    kw = dict(seg_rows=p["seg"], seg_cols=p["cols"])
    s1, s2 = usm.sddmm(ro, ci, t["Q1"], t["K1"]), usm.sddmm(ro, ci, t["Q2"], t["K2"])
    usm.rel_bias(ro, ci, s1, t["table"], t["bmap"], out=s1, **kw)
    A = usm.diff_softmax(ro, s1, s2, t["lam"], seg_rows=p["seg"], out_dtype=t["V"].dtype)
    O = usm.spmm(ro, ci, A, t["V"])
    dA = usm.sddmm(ro, ci, t["dO"], t["V"])
    d1, d2, dlam = usm.diff_softmax_grad(ro, s1, s2, t["lam"], dA, seg_rows=p["seg"], out_dtype=t["V"].dtype)
    dT = usm.rel_bias_grad(ro, ci, d1, *t["table"].shape, t["bmap"], **kw)
    rt, ct, at, perm = usm.csr_transpose(ro, ci, A, p["K"], with_perm=True)
    return dict(O=O, dT=dT, dlam=dlam, dQ1=usm.spmm(ro, ci, d1, t["K1"]), dQ2=usm.spmm(ro, ci, d2, t["K2"]),
                dV=usm.spmm(rt, ct, at, t["dO"]),
                dK1=usm.spmm(rt, ct, usm.csr_permute_values(perm, d1), t["Q1"]),
                dK2=usm.spmm(rt, ct, usm.csr_permute_values(perm, d2), t["Q2"]))


def chain_reference(p, x):
    """The same in 64 bits by automatic differentiation of the dense masked form."""
    import torch
    t = {k: torch.from_numpy(v.astype(np.float64)).requires_grad_(k in ("Q1", "Q2", "K1", "K2", "V", "table", "lam"))
         for k, v in x.items() if k != "bmap"}
    r, c = torch.from_numpy(R.rows_of(p["ro"])), torch.from_numpy(p["ci"].astype(np.int64))
    mask = torch.zeros(p["M"], p["K"], dtype=torch.bool)
    mask[r, c] = True
    k = R.bucket_of_entries(p["ro"], p["ci"], x["bmap"], p["seg"], p["cols"], None, 8)
    head = torch.from_numpy(p["heads"])
    bias = torch.zeros(p["M"], p["K"], dtype=torch.float64)
    bias[r, c] = t["table"][head[r], torch.from_numpy(k)]
    some = mask.any(1)

    def softmax(s):
        s = s.masked_fill(~mask, float("-inf"))[some]
        return torch.zeros_like(mask, dtype=torch.float64).index_put((torch.nonzero(some)[:, 0],), torch.softmax(s, 1))

    A = softmax(t["Q1"] @ t["K1"].T + bias) - t["lam"][head][:, None] * softmax(t["Q2"] @ t["K2"].T)
    O = A @ t["V"]
    O.backward(t["dO"])
    return dict(O=O.detach(), dT=t["table"].grad, dlam=t["lam"].grad, dQ1=t["Q1"].grad, dQ2=t["Q2"].grad, dV=t["V"].grad,
                dK1=t["K1"].grad, dK2=t["K2"].grad)


def scaled(p, x):
    x = dict(x)
    for k in ("Q1", "Q2"):
        x[k] = x[k] * np.float32(0.25)  # a power of two: exact in every type
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_chain(usm, dtype):
    p, x = chain_inputs(dtype)
    x = scaled(p, x)
    t = {k: dev(v) if k == "bmap" else put(v, "f32" if k in ("table", "lam") else dtype) for k, v in x.items()}
    out = run_chain(usm, p, t, dev(p["ro"]), dev(p["ci"]))
    ref = chain_reference(p, x)
    # fp32: scores of size ~10 carry about 24·U·10 = 1.4e-5, which every
    # probability and gradient carries relative to itself: 1e-4 of the largest
    # value.  bf16: maps and score gradients are rounded to half a step of 2^-8
    # each, and a sum of them to at most that of its absolute terms, which is
    # within 4 times the largest result here: 2^-6.
    tol = 1e-4 if dtype == "f32" else 2.0 ** -6
    for k, v in ref.items():
        v = v.numpy()
        assert_near(got(out[k]), v, tol * np.abs(v).max(), k)


def test_chain_agrees_with_single_pass(usm):
    """The one-pass form of few rows gives the chain's rows."""
    p, x = chain_inputs()
    x = scaled(p, x)
    t = {k: dev(v) if k == "bmap" else put(v) for k, v in x.items()}
    ro, ci = dev(p["ro"]), dev(p["ci"])
    s1, s2 = usm.sddmm(ro, ci, t["Q1"], t["K1"]), usm.sddmm(ro, ci, t["Q2"], t["K2"])
    kw = dict(seg_rows=p["seg"], seg_cols=p["cols"])
    for s in (s1, s2):
        usm.rel_bias(ro, ci, s, t["table"], t["bmap"], out=s, **kw)
    O = usm.spmm(ro, ci, usm.diff_softmax(ro, s1, s2, t["lam"], seg_rows=p["seg"]), t["V"])
    one = usm.attention(ro, ci, t["Q1"], t["K1"], t["V"], Q2=t["Q2"], K2=t["K2"], lam=t["lam"], table=t["table"],
                        bucket_map=t["bmap"], **kw)
    # Both within 1e-4 of the largest value of the exact result (see above).
    assert_near(got(one), got(O), 2e-4 * np.abs(got(O)).max(), "one pass")


def test_other_stream(usm):
    """A call on a stream of the caller's waits for nothing but that stream,
    and its outputs and scratch belong to it."""
    import torch
    p, x = chain_inputs()
    t = {k: dev(v) if k == "bmap" else put(v) for k, v in scaled(p, x).items()}
    ro, ci = dev(p["ro"]), dev(p["ci"])
    s1, s2 = usm.sddmm(ro, ci, t["Q1"], t["K1"]), usm.sddmm(ro, ci, t["Q2"], t["K2"])
    dA = usm.sddmm(ro, ci, t["dO"], t["V"])

    def calls(stream):
        b = usm.rel_bias(ro, ci, s1, t["table"], t["bmap"], seg_rows=p["seg"], seg_cols=p["cols"], stream=stream)
        g = usm.diff_softmax_grad(ro, b, s2, t["lam"], dA, seg_rows=p["seg"], stream=stream)
        dT = usm.rel_bias_grad(ro, ci, g[0], HEADS, 8, t["bmap"], seg_rows=p["seg"], seg_cols=p["cols"], stream=stream)
        o = usm.attention(ro, ci, t["Q1"], t["K1"], t["V"], Q2=t["Q2"], K2=t["K2"], lam=t["lam"], seg_rows=p["seg"],
                          stream=stream)
        return [b, *g, dT, o, usm.diff_softmax(ro, b, s2, t["lam"], seg_rows=p["seg"], stream=stream),
                usm.row_softmax_grad(ro, b, dA, stream=stream)]

    want = calls(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        have = calls(side)
    side.synchronize()
    for a, b in zip(want, have):
        assert torch.equal(a, b)


def test_graph_replay(usm):
    """The whole step, captured and replayed on new inputs, while eager calls
    run between the replays."""
    import torch
    p, x = chain_inputs()
    t = {k: dev(v) if k == "bmap" else put(v) for k, v in scaled(p, x).items()}
    ro, ci = dev(p["ro"]), dev(p["ci"])
    step = lambda: run_chain(usm, p, t, ro, ci)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    for k in ("Q1", "dO", "table", "lam"):
        t[k].mul_(0.5)
    g.replay()
    eager = step()
    g.replay()
    torch.cuda.synchronize()
    for k, v in eager.items():
        assert torch.equal(v, captured[k]), k


@pytest.mark.parametrize("maps,dtype,D,N,biased", [(1, "bf16", 64, 64, True), (2, "bf16", 64, 128, False),
                                                   (2, "bf16", 72, 200, True), (1, "f32", 64, 64, False),
                                                   (2, "f32", 33, 100, True)])
@pytest.mark.parametrize("kind", ["even", "long", "skewed", "short"])
def test_attention_equal_shares(usm, kind, maps, dtype, D, N, biased):
    """Problems large enough to be dealt out in equal shares of the entries:
    rows inside a share, cut by one, and over many; empty rows everywhere."""
    rng = np.random.default_rng([17, sorted(["even", "long", "skewed", "short"]).index(kind)])
    cols = 30000 if kind == "long" else 4000
    lengths = {"even": rng.integers(300, 500, 260), "long": np.array([0, 29000, 30000, 17, 30000, 0]),
               "skewed": np.concatenate([rng.integers(0, 12, 3000), [4000] * 20, rng.integers(0, 12, 2000)]),
               "short": rng.integers(0, 12, 20000)}[kind]
    lengths[:: 5 if kind != "long" else 100] = 0
    seg = 1 if kind in ("even", "long") else 0
    base = np.arange(lengths.size) % 3 * cols if seg else None
    ro, ci = W.csr_from_lengths(rng, lengths.astype(np.int64), cols, base)
    p = dict(rng=rng, ro=ro, ci=ci, M=lengths.size, K=3 * cols if seg else cols, cols=cols, seg=seg,
             blocks=lengths.size if seg else 1, nnz=ci.size, heads=R.head_of_rows(lengths.size, seg, HEADS),
             longest=int(lengths.max()))
    need = usm.load().csr_attention_workspace_bytes(p["M"], p["K"], D, N, p["nnz"], int(maps == 2), int(dtype == "bf16"))
    assert need > 0
    run_attention(usm, p, D, N, maps, dtype, biased, pad=True)


def gaps(kind):
    """Runs of thousands of rows without entries: between rows, before the first
    and behind the last (a padded batch)."""
    rng = np.random.default_rng([23, sorted(["between", "ends"]).index(kind)])
    lengths = np.zeros(20000, dtype=np.int64)
    if kind == "between":
        lengths[rng.choice(20000, 300, replace=False)] = rng.integers(1, 700, 300)
        lengths[[5000, 5001, 5002, 5003, 12000]] = [1700, 3, 0, 5000, 2500]
    else:
        lengths[9000:9400] = rng.integers(0, 700, 400)
        lengths[9400] = 3000
    seg, cols = 1000, 6000
    ro, ci = W.csr_from_lengths(rng, lengths, cols, np.arange(20000) // seg * cols)
    return dict(rng=rng, ro=ro, ci=ci, M=20000, K=20 * cols, cols=cols, seg=seg, blocks=20, nnz=ci.size,
                heads=R.head_of_rows(20000, seg, HEADS), longest=int(lengths.max()))


@pytest.mark.parametrize("kind", ["between", "ends"])
def test_runs_of_empty_rows(usm, kind):
    p = gaps(kind)
    rng, ro, ci = p["rng"], dev(p["ro"]), dev(p["ci"])
    bmap, q_offset, table = bias_inputs(p)
    kw = dict(seg_rows=p["seg"], seg_cols=p["cols"], q_offset=dev(q_offset))
    k = R.bucket_of_entries(p["ro"], p["ci"], bmap, p["seg"], p["cols"], q_offset, table.shape[1])
    r = R.rows_of(p["ro"])
    s1, s2 = scores_of(p, rng), scores_of(p, rng)
    assert np.array_equal(host(usm.rel_bias(ro, ci, put(s1), put(table), dev(bmap), **kw)), s1 + table[p["heads"][r], k])
    ds = rng.integers(-8, 9, p["nnz"]).astype(np.float32)
    want = np.bincount(p["heads"][r] * table.shape[1] + k, ds, table.size).reshape(table.shape)
    assert np.array_equal(got(usm.rel_bias_grad(ro, ci, put(ds), *table.shape, dev(bmap), **kw)), want)
    lam = rng.uniform(0.1, 0.9, HEADS).astype(np.float32)
    lr = lam.astype(np.float64)[p["heads"]]
    E = R.softmax_error(p["longest"], SPREAD)
    size = R.row_softmax(p["ro"], s1) + lr[r] * R.row_softmax(p["ro"], s2)
    assert_near(got(usm.diff_softmax(ro, put(s1), put(s2), put(lam), seg_rows=p["seg"])), R.diff_map(p["ro"], s1, s2, lr),
                (E + 2 * U) * size, "map")
    dout = rng.standard_normal(p["nnz"]).astype(np.float32)
    g1, g2, dlam = R.diff_grad(p["ro"], s1, s2, lr, dout, HEADS, p["heads"])
    o1, o2, ol = usm.diff_softmax_grad(ro, put(s1), put(s2), put(lam), put(dout), seg_rows=p["seg"])
    t1, _ = grad_bound(p, s1, dout, 1.0)
    t2, c2 = grad_bound(p, s2, dout, lr[r])
    assert_near(got(o1), g1, t1, "dscores1")
    assert_near(got(o2), g2, t2, "dscores2")
    rows = np.bincount(p["heads"], minlength=HEADS)
    csize = np.bincount(p["heads"], np.abs(R.softmax_grad(p["ro"], s2, dout)[2]), HEADS)
    assert_near(got(ol), dlam, np.bincount(p["heads"], c2, HEADS) + rows * U * csize, "dlambda")
    assert_near(got(usm.row_softmax_grad(ro, put(s1), put(dout))), R.softmax_grad(p["ro"], s1, dout)[0], t1, "softmax gradient")
    for dtype in ("bf16", "f32"):
        run_attention(usm, p, 64, 64, 2, dtype, False)


@pytest.mark.parametrize("low", [-60.0, -1e9, float(np.finfo(np.float32).min), -np.inf])
def test_rows_that_begin_low(usm, low):
    """Padding at the left, by a finite value or -inf: the rows' first scores say
    nothing about their maxima.  Rows without padding lie between, and a row of
    nothing else."""
    rng = np.random.default_rng(29)
    lengths = rng.integers(1, 900, 400)
    lengths[::9] = 0
    lengths[17] = 1900
    ro, ci = W.csr_from_lengths(rng, lengths.astype(np.int64), 4000, None)
    heads = np.zeros(400, dtype=np.int64)
    nnz = ci.size
    s1, s2 = (np.clip(2.5 * rng.standard_normal(nnz), -8, 8).astype(np.float32) for _ in range(2))
    for r in range(400):
        if r % 3 == 0:
            s1[ro[r]:ro[r] + rng.integers(1, 200)] = low  # may run into the next rows
    s2[ro[30]:ro[31]] = low
    E = R.softmax_error(1900, SPREAD if low != -60.0 else 68.0)  # lower weights than e^-100 are 0 in both
    lam = np.array([0.7], dtype=np.float32)
    lr = np.full(400, np.float64(lam[0]))
    r = R.rows_of(ro)
    p1, p2 = R.row_softmax(ro, s1), R.row_softmax(ro, s2)
    rod, a1, a2, ld = dev(ro), put(s1), put(s2), put(lam)
    assert_near(got(usm.diff_softmax(rod, a1, a2, ld)), R.diff_map(ro, s1, s2, lr), (E + 2 * U) * (p1 + lr[r] * p2), "map")
    dout = rng.standard_normal(nnz).astype(np.float32)
    g1, g2, _ = R.diff_grad(ro, s1, s2, lr, dout, 1, heads)
    o1, o2, _ = usm.diff_softmax_grad(rod, a1, a2, ld, put(dout))
    for o, g, p, w, s in ((o1, g1, p1, 1.0, s1), (o2, g2, p2, lr[r], s2),
                          (usm.row_softmax_grad(rod, a1, put(dout)), g1, p1, 1.0, s1)):
        masked = s == -np.inf
        c = R.row_dot(ro, p, np.abs(np.where(masked, 0, dout)), masked)
        assert_near(got(o), g, w * p * (np.abs(np.where(masked, 0, dout)) + c[r]) * (3 * E + 8 * U), "gradient")


@pytest.mark.parametrize("captured", [False, True])
def test_results_are_there_for_the_next_kernel(usm, captured):
    """What follows a call of two kernels on its stream sees both done: a copy of
    the results, and a call that overwrites the inputs' memory."""
    import torch
    rng = np.random.default_rng(31)
    ro, ci = W.csr_from_lengths(rng, rng.integers(300, 500, 260), 4000, np.arange(260) % 3 * 4000)
    M, K, nnz = 260, 12000, ci.size
    rod, cid, lam = dev(ro), dev(ci), put(np.full(HEADS, 0.5))
    xs = [[torch.randn(n, 64, device="cuda").bfloat16() for n in (M, K, M, K)] + [torch.randn(K, 128, device="cuda").bfloat16()]
          for _ in range(2)]
    ss = [[torch.randn(nnz, device="cuda") for _ in range(3)] for _ in range(2)]
    x, s = [t.clone() for t in xs[0]], [t.clone() for t in ss[0]]

    def step():
        o = usm.attention(rod, cid, x[0], x[1], x[4], scale=0.125, Q2=x[2], K2=x[3], lam=lam, seg_rows=1)
        o2 = o * 1
        g = usm.diff_softmax_grad(rod, s[0], s[1], lam, s[2], seg_rows=1)
        g2 = [t * 1 for t in g]
        for a, b in zip(x + s, xs[1] + ss[1]):
            a.copy_(b)
        return [o2, *g2]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = step()
        for _ in range(10):
            for a, b in zip(x + s, xs[0] + ss[0]):
                a.copy_(b)
            if captured:
                graph.replay()
                have = [t.clone() for t in out]
            else:
                have = step()
            side.synchronize()
            for a, b in zip(want, have):
                assert torch.equal(a, b)


@pytest.mark.parametrize("mean", [1250, 1400, 2000, 4500])
def test_many_long_rows(usm, mean):
    """More long rows than the GPU has room for at once: a CTA to a row, which
    holds it in registers or reads it twice, next to short and empty rows."""
    rng = np.random.default_rng([37, mean])
    M = 640
    lengths = rng.integers(mean // 2, mean * 3 // 2, M)
    lengths[::50] = 0
    lengths[1::50] = 3
    lengths[2::50] = 3 * mean
    cols = 3 * mean
    ro, ci = W.csr_from_lengths(rng, lengths.astype(np.int64), cols, None)
    heads = np.arange(M) % HEADS
    s1, s2 = (np.clip(2.5 * rng.standard_normal(ci.size), -8, 8).astype(np.float32) for _ in range(2))
    s1[rng.random(ci.size) < 0.05] = -np.inf
    s1[ro[7]:ro[8]] = -np.inf
    lam = rng.uniform(0.1, 0.9, HEADS).astype(np.float32)
    lr = lam.astype(np.float64)[heads]
    r = R.rows_of(ro)
    p = dict(ro=ro, longest=3 * mean)
    rod, a1, a2, ld = dev(ro), put(s1), put(s2), put(lam)
    tol = (R.softmax_error(3 * mean, SPREAD) + 2 * U) * (R.row_softmax(ro, s1) + lr[r] * R.row_softmax(ro, s2))
    assert_near(got(usm.diff_softmax(rod, a1, a2, ld, seg_rows=1)), R.diff_map(ro, s1, s2, lr), tol, "map")
    dout = rng.standard_normal(ci.size).astype(np.float32)
    g1, g2, dlam = R.diff_grad(ro, s1, s2, lr, dout, HEADS, heads)
    o1, o2, ol = usm.diff_softmax_grad(rod, a1, a2, ld, put(dout), seg_rows=1)
    t1, _ = grad_bound(p, s1, dout, 1.0)
    t2, c2 = grad_bound(p, s2, dout, lr[r])
    assert_near(got(o1), g1, t1, "dscores1")
    assert_near(got(o2), g2, t2, "dscores2")
    size = np.bincount(heads, np.abs(R.softmax_grad(ro, s2, dout)[2]), HEADS)
    assert_near(got(ol), dlam, np.bincount(heads, c2, HEADS) + np.bincount(heads, minlength=HEADS) * U * size, "dlambda")
    assert_near(got(usm.row_softmax_grad(rod, a1, put(dout))), g1, t1, "softmax gradient")
    x = a1.clone()  # in place
    usm.row_softmax_grad(rod, x, put(dout), out=x)
    assert np.array_equal(host(x), host(usm.row_softmax_grad(rod, a1, put(dout))))
