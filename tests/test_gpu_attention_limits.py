"""Sparse-attention operators at the ends of their ranges: values, sums, sizes
and calls."""
import ctypes

import numpy as np
import pytest

import attention_ref as R
import workloads as W
from parity_util import dev, host
from test_gpu_attention import HEADS, assert_near, attention_case, got, make, put

pytestmark = pytest.mark.gpu

U = R.U

# ---------------------------------------------------------------------------
# Scores far from zero
# ---------------------------------------------------------------------------
# Row lengths for each form of the maps' kernels: rings (four and two rows at
# once, and one), rows over the ring among short ones (a CTA), mostly long rows
# (CTAs of four and of eight warps, one row past their registers), and clusters.
FORMS = {
    "ring": np.concatenate([np.arange(1, 200), [8] * 64, np.arange(200, 1500, 37), [1536, 0, 7]]),
    "over": np.concatenate([np.arange(1, 300), [2100, 9000, 3, 17000], np.arange(300)]),
    "cta4": np.concatenate([np.resize(np.arange(1250, 2200), 640 * 7)[::7], [9000]]),
    "cta8": np.concatenate([np.arange(1400, 2200, 4), [17000]]),
    "cluster": np.array([40000, 60001, 50000]),
}
FAR = [2e7, -2e7, 3e9, -3e9, 1e10, -1e10, 3e10, -3e10, 1e12, -1e20, 1e20, -1e30, 9e36, -9e36, 1e38, 3e38, -3e38]


def far_scores(rng, ro, value):
    """Rows of the value alone, of values next to it, and of ordinary scores
    with the value at the left, at the right, at one place or everywhere but at
    one; every other row also has entries of -inf."""
    nnz = int(ro[-1])
    s = np.clip(2.5 * rng.standard_normal(nnz), -8, 8).astype(np.float32)
    v = np.float32(value)
    for r in range(ro.size - 1):
        b, e = int(ro[r]), int(ro[r + 1])
        n = e - b
        if n == 0:
            continue
        kind = r % 6
        if kind == 0:
            s[b:e] = v
        elif kind == 1:
            s[b:e] = v * (1 + rng.integers(0, 8, n).astype(np.float32) * np.float32(2.0 ** -23))
        elif kind == 2:
            s[b:b + n // 2] = v
        elif kind == 3:
            s[b + n // 2:e] = v
        elif kind == 4:
            s[b + rng.integers(n)] = v
        else:
            keep = b + rng.integers(n)
            x = s[keep]
            s[b:e] = v
            s[keep] = x
        if r // 6 % 2:
            s[b:e][rng.random(n) < 0.1] = -np.inf
    return s


@pytest.mark.parametrize("value", FAR)
@pytest.mark.parametrize("form", sorted(FORMS))
def test_scores_far_from_zero(usm, form, value):
    """Every finite score counts: maps, gradients and dlambda of rows whose
    scores lie anywhere in fp32's range."""
    rng = np.random.default_rng([41, sorted(FORMS).index(form), FAR.index(value)])
    lengths = FORMS[form].astype(np.int64)
    ro = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    M, nnz, r = lengths.size, int(ro[-1]), R.rows_of(ro)
    heads = np.arange(M) % HEADS
    s1, s2 = far_scores(rng, ro, value), far_scores(rng, ro, -value if form == "ring" else value)
    dout = rng.standard_normal(nnz).astype(np.float32)
    lam = rng.uniform(0.1, 0.9, HEADS).astype(np.float32)
    lr = lam.astype(np.float64)[heads]
    # Weights count down to e^-90: lower ones may be flushed to zero, and are
    # below 2^-126 of the sum times at most 4.
    E, tiny = R.softmax_error(int(lengths.max()), 90.0), 2.0 ** -124
    p1, p2 = R.row_softmax(ro, s1), R.row_softmax(ro, s2)
    rod, a1, a2, ld, dd = dev(ro), put(s1), put(s2), put(lam), put(dout)
    assert_near(got(usm.diff_softmax(rod, a1, a2, ld, seg_rows=1)), p1 - lr[r] * p2,
                (E + 2 * U) * (p1 + lr[r] * p2) + 2 * tiny, "map")
    g1, g2, dlam = R.diff_grad(ro, s1, s2, lr, dout, HEADS, heads)
    o1, o2, ol = usm.diff_softmax_grad(rod, a1, a2, ld, dd, seg_rows=1)
    o = usm.row_softmax_grad(rod, a1, dd)
    for x, g, p, w, s, what in ((o1, g1, p1, 1.0, s1, "dscores1"), (o2, g2, p2, lr[r], s2, "dscores2"),
                                (o, g1, p1, 1.0, s1, "softmax gradient")):
        masked = s == -np.inf
        size = np.abs(np.where(masked, 0, dout))
        c = R.row_dot(ro, p, size, masked)
        assert_near(got(x), g, w * p * (size + c[r]) * (3 * E + 8 * U) + 20 * tiny, what)
    c = R.row_dot(ro, p2, np.abs(np.where(s2 == -np.inf, 0, dout)), s2 == -np.inf) * (3 * E + 8 * U)
    rows = np.bincount(heads, minlength=HEADS)
    csize = np.bincount(heads, np.abs(R.softmax_grad(ro, s2, dout)[2]), HEADS)
    assert_near(got(ol), dlam, np.bincount(heads, c, HEADS) + rows * U * csize + 1e-30, "dlambda")


# ---------------------------------------------------------------------------
# Attention: rows of V that nothing uses
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("maps,N", [(1, 32), (2, 32), (1, 200), (2, 72)])
@pytest.mark.parametrize("shares", [False, True])
def test_unused_rows_of_v(usm, shares, maps, N, dtype):
    """Rows of V under entries that are masked in every map may hold NaN and
    infinities, in both forms of the kernel."""
    import torch
    if shares:
        rng = np.random.default_rng(43)
        lengths, cols = rng.integers(600, 900, 200), 4000
        lengths[::7] = 0
        ro, ci = W.csr_from_lengths(rng, lengths.astype(np.int64), cols, np.arange(200) % 3 * cols)
        p = dict(rng=rng, ro=ro, ci=ci, M=200, K=3 * cols, cols=cols, seg=1, blocks=200, nnz=ci.size,
                 heads=R.head_of_rows(200, 1, HEADS), longest=900)
    else:
        p = make("tokens")
    D = 48
    Qs, Ks, V, lam, bias, entry = attention_case(p, D, N, maps, dtype, False)
    # A map of positions to buckets that sends every third key to a bucket of -inf.
    reach = p["cols"]
    bmap = (np.arange(2 * reach + 1) % 3).astype(np.int32)
    table = p["rng"].standard_normal((HEADS, 3)).astype(np.float32)
    table[:, 1] = -np.inf
    k = R.bucket_of_entries(p["ro"], p["ci"], bmap, p["seg"], p["cols"], None, 3)
    masked = table[p["heads"][R.rows_of(p["ro"])], k] == -np.inf
    unused = np.zeros(p["K"], dtype=bool)
    unused[p["ci"][masked]] = True
    unused[p["ci"][~masked]] = False
    assert unused.sum() > 100
    need = usm.load().csr_attention_workspace_bytes(p["M"], p["K"], D, N, p["nnz"], int(maps == 2), int(dtype == "bf16"))
    assert (need > 0) == shares
    kw = dict(scale=0.2, seg_rows=p["seg"], table=put(table), bucket_map=dev(bmap), seg_cols=p["cols"])
    if maps == 2:
        kw.update(Q2=put(Qs[1], dtype), K2=put(Ks[1], dtype), lam=put(lam))
    v = put(V, dtype)
    bad = v.clone()
    at = torch.from_numpy(np.flatnonzero(unused)).cuda()
    junk = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").repeat(at.numel())
    bad[at] = junk[:at.numel(), None].to(v.dtype)
    call = lambda t: usm.attention(dev(p["ro"]), dev(p["ci"]), put(Qs[0], dtype), put(Ks[0], dtype), t, **kw)
    x, y = call(v), call(bad)
    assert torch.isfinite(x).all() and torch.equal(x, y)


# ---------------------------------------------------------------------------
# Calls
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("which", ["attention", "attention_shares", "diff_softmax", "poll"])
def test_a_failed_launch_is_reported_once(usm, which):
    """What CUDA refuses (work on a stream whose capture was invalidated) fails
    that call alone: the next call, with nothing wrong, succeeds."""
    import torch
    lib, cu = usm.load(), ctypes.CDLL("libcuda.so.1")
    x = torch.zeros(1 << 16, device="cuda")
    shares = which == "attention_shares"
    nnz = 1 << 16 if shares else 4000
    ro, ci = dev(np.array([0, nnz], dtype=np.int32)), torch.zeros(nnz, dtype=torch.int32, device="cuda")
    out, ws = torch.zeros(1 << 16, device="cuda"), torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    bmap = torch.empty(257, dtype=torch.int32, device="cuda")
    lam = torch.ones(1, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    s = side.cuda_stream
    at = lambda t: t.data_ptr()
    D = 256 if shares else 8

    def call():
        if which == "poll":
            return lib.usm_poll_status(s)
        if which == "diff_softmax":
            return lib.csr_diff_softmax(1, nnz, at(ro), at(x), at(x), at(lam), 1, 1, at(out), 0, s)
        return lib.csr_attention(1, 4, D, D, nnz, at(ro), at(ci), at(x), D, at(x), D, None, 0, None, 0, at(x), D, 1.0, None, 1,
                                 1, None, at(out), D, 0, at(ws), ws.numel(), s)

    assert call() == 0  # nothing is wrong with the call itself
    side.synchronize()
    assert cu.cuStreamBeginCapture_v2(ctypes.c_void_p(s), 2) == 0  # relaxed
    assert cu.cuStreamSynchronize(ctypes.c_void_p(s)) != 0  # not allowed in a capture: it ends as a failure
    failed = call()
    graph = ctypes.c_void_p()
    assert cu.cuStreamEndCapture(ctypes.c_void_p(s), ctypes.byref(graph)) != 0
    assert failed == -4  # USM_ERR_CUDA
    assert lib.rel_bucket_build(32, 128, 0, at(bmap), s) == 0
    assert call() == 0
    side.synchronize()


def test_bucket_map_is_checked_before_memory_is_taken(usm):
    import torch
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    for reach in (8193, 10**9, 2**31 - 1):
        with pytest.raises(usm.USMError, match="UNSUPPORTED"):
            usm.rel_bucket_map(32, reach)
    assert torch.cuda.max_memory_allocated() == before


def test_bucket_map_stream_and_device_agree(usm):
    import torch

    class Elsewhere:  # a stream of another device
        device = torch.device("cuda", torch.cuda.device_count())

    with pytest.raises(ValueError, match="stream is on"):
        usm.rel_bucket_map(32, 128, False, "cuda:0", stream=Elsewhere())
    with pytest.raises(ValueError, match="stream is on"):
        usm.rel_bucket_map(32, 128, device=0, stream=Elsewhere())
    side = torch.cuda.Stream()
    want = host(usm.rel_bucket_map(32, 128))
    for device in (None, "cuda", "cuda:0", 0, torch.device("cuda", 0)):
        t = usm.rel_bucket_map(32, 128, device=device, stream=side)
        side.synchronize()
        assert np.array_equal(host(t), want)


def test_empty_batches(usm):
    """A batch of no sequences: no rows, no query blocks, no offsets."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    ro, none, ci = torch.zeros(1, **i32), torch.empty(0, device="cuda"), torch.empty(0, **i32)
    bmap, table = dev(np.zeros(5, dtype=np.int32)), put(np.ones((2, 4)))
    kw = dict(seg_rows=1, seg_cols=8, q_offset=torch.empty(0, **i32))
    assert usm.rel_bias(ro, ci, none, table, bmap, **kw).numel() == 0
    assert np.array_equal(got(usm.rel_bias_grad(ro, ci, none, 2, 4, bmap, **kw)), np.zeros((2, 4)))
    x = torch.empty((0, 8), device="cuda")
    assert usm.attention(ro, ci, x, x, x, table=table, bucket_map=bmap, **kw).shape == (0, 8)
    kw["q_offset"] = torch.zeros(1, **i32)  # "one block of M rows"
    assert usm.rel_bias(ro, ci, none, table, bmap, **kw).numel() == 0
    kw["q_offset"] = torch.zeros(2, **i32)
    with pytest.raises(ValueError, match="q_offset"):
        usm.rel_bias(ro, ci, none, table, bmap, **kw)


# ---------------------------------------------------------------------------
# Long sums
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("seg", [0, 1])
def test_dlambda_of_cancelling_rows(usm, seg):
    """Rows whose contributions cancel leave the others' sum: rows of one entry,
    dout = 1 but for pairs of 2^30 and -2^30.  Pairs cancel whatever a row's own
    arithmetic does to them, as it does the same to both; of the others it loses
    at most 4 U each, and the result is rounded once."""
    rng = np.random.default_rng(47)
    M, pairs, heads = 60000, 100, 1 if seg == 0 else 3
    dout = np.ones(M, dtype=np.float32)
    head = np.arange(M) % heads
    for h in range(heads):
        at = rng.choice(np.flatnonzero(head == h), 2 * pairs, replace=False)
        dout[at[:pairs]], dout[at[pairs:]] = 2.0 ** 30, -(2.0 ** 30)
    s = put(np.zeros(M))
    ro = dev(np.arange(M + 1, dtype=np.int32))
    dlam = usm.diff_softmax_grad(ro, s, s, put(np.full(heads, 0.5)), put(dout), seg_rows=seg)[2]
    want = -(np.bincount(head, minlength=heads) - 2.0 * pairs)
    assert_near(got(dlam), want, 5 * U * np.abs(want), "dlambda")


@pytest.mark.parametrize("side", ["back", "ahead"])
def test_bias_gradient_of_long_sums(usm, side):
    """Many equal entries beyond the map's reach.  A thread adds at most 16 of
    them in fp32 (15 roundings of relative size U), those sums with compensation
    (2 U in all, and U^2 an addition); 32 threads of a CTA are joined in 5
    levels, CTAs in 64 bits, and the result rounded: at most 25 U."""
    import torch
    rows, n, buckets = 3000, 4000, 512
    ro = np.arange(rows + 1, dtype=np.int64) * n
    ci = torch.arange(n, dtype=torch.int32, device="cuda").repeat(rows)
    x = torch.full((rows * n,), 0.1, device="cuda")
    bmap = dev(np.array([3, 4, 5], dtype=np.int32))
    q_offset = dev(np.array([2**30 if side == "back" else -2**30], dtype=np.int32))
    out = got(usm.rel_bias_grad(dev(ro.astype(np.int32)), ci, x, 1, buckets, bmap, q_offset=q_offset))
    want = np.zeros((1, buckets))
    want[0, 3 if side == "back" else 5] = rows * n * np.float64(np.float32(0.1))
    assert_near(out, want, 25 * U * want, "dtable")


# ---------------------------------------------------------------------------
# Row counts next to 2^31
# ---------------------------------------------------------------------------
def test_most_rows(usm):
    """2^31 - 2 rows (offsets of 8.6 GB), nearly all without entries: a few at
    the beginning, in the middle and at the very end, long ones among them."""
    import torch
    rng = np.random.default_rng(53)
    M = 2**31 - 2
    runs = {0: [3, 0, 700, 1, 8, 8, 8, 8], 2**30 - 2: [5, 5000, 0, 40], M - 200: [2100, 0, 9, 17], M - 6: [30, 1, 6000, 0, 2, 11]}
    rows = np.concatenate([first + np.arange(len(x)) for first, x in runs.items()])
    lengths = np.concatenate([np.array(x) for x in runs.values()])
    small = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    nnz = int(small[-1])
    ro = torch.full((M + 1,), nnz, dtype=torch.int32, device="cuda")
    ro[0] = 0
    done = 1
    for i, row in enumerate(rows):  # offsets of the rows without entries between two of them
        ro[done:int(row) + 1] = int(small[i])
        ro[int(row) + 1] = int(small[i + 1])
        done = int(row) + 2
    s1, s2 = (np.clip(2.5 * rng.standard_normal(nnz), -8, 8).astype(np.float32) for _ in range(2))
    dout, lam = rng.standard_normal(nnz).astype(np.float32), np.array([0.7], dtype=np.float32)
    r, lr = R.rows_of(small), np.full(lengths.size, np.float64(lam[0]))
    E = R.softmax_error(int(lengths.max()), 16.0)
    p1, p2 = R.row_softmax(small, s1), R.row_softmax(small, s2)
    a1, a2, dd, ld = put(s1), put(s2), put(dout), put(lam)
    assert_near(got(usm.diff_softmax(ro, a1, a2, ld)), p1 - lr[r] * p2, (E + 2 * U) * (p1 + lr[r] * p2), "map")
    g1, g2, dlam = R.diff_grad(small, s1, s2, lr, dout, 1, np.zeros(lengths.size, dtype=np.int64))
    o1, o2, ol = usm.diff_softmax_grad(ro, a1, a2, ld, dd)
    nomask = np.zeros(nnz, dtype=bool)
    for x, g, p, w in ((o1, g1, p1, 1.0), (o2, g2, p2, lr[r]), (usm.row_softmax_grad(ro, a1, dd), g1, p1, 1.0)):
        c = R.row_dot(small, p, np.abs(dout), nomask)
        assert_near(got(x), g, w * p * (np.abs(dout) + c[r]) * (3 * E + 8 * U), "gradient")
    c = R.row_dot(small, p2, np.abs(dout), nomask)
    assert_near(got(ol), dlam, c.sum() * (3 * E + 8 * U) + lengths.size * U * c.sum(), "dlambda")
    # Query positions are row numbers here: keys up to 4 ahead of the last row's.
    bmap, table = dev(np.arange(9, dtype=np.int32)), rng.standard_normal((1, 9)).astype(np.float32)
    ci = (np.minimum(rows[r] + rng.integers(-6, 7, nnz), 2**31 - 2).clip(0)).astype(np.int64)
    k = np.clip(ci - rows[r], -4, 4) + 4
    cid = dev(ci.astype(np.int32))
    assert np.array_equal(host(usm.rel_bias(ro, cid, a1, put(table), bmap)), s1 + table[0, k])
    ds = rng.integers(-8, 9, nnz).astype(np.float32)
    assert np.array_equal(got(usm.rel_bias_grad(ro, cid, put(ds), 1, 9, bmap))[0], np.bincount(k, ds, 9))


def test_runs_of_rows_without_entries_take_no_time(usm):
    """10^9 rows without entries before a long one: passed by a search (0.1 ms),
    not walked (seconds)."""
    import torch
    M = 10**9
    ro = torch.full((M + 1,), 3, dtype=torch.int32, device="cuda")
    ro[0], ro[M] = 0, 5003
    s, lam = torch.randn(5003, device="cuda"), torch.ones(1, device="cuda")
    calls = (lambda: usm.diff_softmax(ro, s, s, lam), lambda: usm.row_softmax_grad(ro, s, s))
    for call in calls:
        call()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        call()
        end.record()
        end.synchronize()
        assert begin.elapsed_time(end) < 250


def test_sums_that_are_not_finite(usm):
    """Infinities and NaN come through the sums in two numbers as through plain
    additions."""
    inf, nan = np.inf, np.nan
    # Bucket 0 for keys behind, 1 for the same position, 2 for keys ahead; one row.
    for value, other, want in ((inf, 1.0, inf), (-inf, 1.0, -inf), (nan, 1.0, nan), (inf, -inf, nan), (3e38, 3e38, inf)):
        for bucket, cols in enumerate((range(0, 8), (8, 8), range(9, 17))):
            ci = np.array(list(range(0, 8)) + [8, 8] + list(range(9, 17)), dtype=np.int32)
            ds = np.ones(ci.size, dtype=np.float32)
            at = [i for i in range(ci.size) if ci[i] in cols]
            ds[at[0]], ds[at[-1]] = value, other
            out = got(usm.rel_bias_grad(dev(np.array([0, ci.size], dtype=np.int32)), dev(ci), put(ds), 1, 3,
                                        dev(np.arange(3, dtype=np.int32)), q_offset=dev(np.array([8], dtype=np.int32))))
            expected = np.array([[8.0, 2.0, 8.0]])
            expected[0, bucket] = want
            assert np.array_equal(out, expected, equal_nan=True), (value, other, bucket, out)
    dout = np.ones(3000, dtype=np.float32)
    dout[300], dout[301], dout[302] = inf, nan, -1.0
    dout[601] = inf
    s, ro = put(np.zeros(3000)), dev(np.arange(3001, dtype=np.int32))
    dlam = got(usm.diff_softmax_grad(ro, s, s, put(np.full(3, 0.5)), put(dout), seg_rows=1)[2])
    assert dlam[0] == -inf and np.isnan(dlam[1]) and abs(dlam[2] + 998) <= 5 * U * 1000
