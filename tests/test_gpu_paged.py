"""The paged cache on the GPU against the 64-bit definitions in paged_ref:
rotation table, append with rotation, attention of new tokens over the pages,
and the three run together beside the library's other attention."""
import zlib

import numpy as np
import pytest

import paged_ref as R
import workloads as W
from parity_util import dev, host

pytestmark = pytest.mark.gpu

TYPES = ("f32", "bf16")


def rounded(x, dtype):
    x = np.asarray(x, dtype=np.float32)
    return W.bf16_bits_to_f32(W.f32_to_bf16_bits(x)) if dtype == "bf16" else x


def put(x, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(torch_type(dtype))


def torch_type(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def ints(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def got(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


def assert_near(x, ref, bound, what=""):
    assert x.shape == ref.shape, (what, x.shape, ref.shape)
    bad = ~(np.abs(x - ref) <= bound)
    if bad.any():
        i = tuple(int(v) for v in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: {x[i]!r} against {ref[i]!r}, "
                             f"bound {np.broadcast_to(bound, ref.shape)[i]!r}")


def same_values(x, ref):
    """Equal, NaN and infinities included."""
    return np.array_equal(x, ref, equal_nan=True)


class Problem:
    """A cache filled at random, its pages in random order, every slot that no
    sequence owns poisoned with NaN, and unused entries of the table wild."""

    def __init__(self, name, lengths, counts, heads=4, kv=2, D=64, page=16, dtype="bf16", before=0, behind=0, spare=3,
                 extra=2, std=1.0):
        rng = self.rng = np.random.default_rng(zlib.crc32(name.encode()))
        self.dtype, self.D, self.page = dtype, D, page
        self.lengths, self.counts = np.array(lengths), np.array(counts)
        self.starts = before + np.cumsum(self.counts) - self.counts
        self.T = before + int(self.counts.sum()) + behind
        per = -(-self.lengths // page)
        pages = int(per.sum()) + spare
        order = rng.permutation(pages)
        self.table = rng.integers(-2**31, 2**31 - 1, (len(lengths), int(per.max(initial=0)) + extra))
        self.k, self.v = (np.full((pages, page, kv, D), np.nan, dtype=np.float32) for _ in range(2))
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at : at + n]
            at += n
            p = np.arange(self.lengths[b])
            for c in (self.k, self.v):
                c[self.table[b, p // page], p % page] = rounded(std * rng.standard_normal((p.size, kv, D)), dtype)
        self.q = rounded(std * rng.standard_normal((self.T, heads, D)), dtype)
        uniform = before == behind == 0 and len(set(counts)) == 1
        self.offsets = None if uniform else np.append(self.starts, before + int(self.counts.sum()))

    def reference(self, scale, **kw):
        return R.attention(self.q.astype(np.float64), self.k.astype(np.float64), self.v.astype(np.float64), self.table,
                           self.lengths, self.counts, self.starts, scale, dtype=self.dtype, **kw)

    def on_device(self, heads_first=False):
        """(q, k_cache, v_cache, table, lengths, offsets)."""
        k, v = put(self.k, self.dtype), put(self.v, self.dtype)
        if heads_first:  # the same cache, each head's slots together
            k, v = (c.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3) for c in (k, v))
        return (put(self.q, self.dtype), k, v, ints(self.table), ints(self.lengths),
                None if self.offsets is None else ints(self.offsets))

    def run(self, usm, scale=None, out=None, heads_first=False, **kw):
        q, k, v, table, lengths, offsets = self.on_device(heads_first)
        scale = self.D ** -0.5 if scale is None else scale
        return usm.paged_attention(q, k, v, table, lengths, q_offsets=offsets, scale=scale, out=out, **kw)

    def check(self, usm, scale=None, **kw):
        import torch
        scale = self.D ** -0.5 if scale is None else scale
        out = torch.full((self.T, *self.q.shape[1:]), 77.0, device="cuda", dtype=torch_type(self.dtype))
        x = got(self.run(usm, scale, out=out, **kw))
        kw.pop("heads_first", None)
        ref, bound = self.reference(scale, **kw)
        idle = np.isnan(bound).all((1, 2))
        assert np.all(x[idle] == 77.0), "rows of no sequence were written"
        assert_near(x[~idle], ref[~idle], bound[~idle])
        assert usm.poll_status() == 0


# ---------------------------------------------------------------------------
# Rotation table and append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("positions,rot,base", [(1, 2, 10000.0), (77, 40, 10000.0), (5000, 128, 500000.0), (300, 6, 0.5)])
def test_rope_table(usm, positions, rot, base):
    x = got(usm.rope_table(positions, rot, base))
    ref = R.rope_table(positions, rot, base)
    # Angles in 64 bits: positions·2^-52 each way of forming the power, then one rounding.
    assert_near(x, ref, R.U * np.abs(ref) + 8 * (positions * max(base ** -1, 1.0)) * 2.0 ** -52 + 2.0 ** -52)


def test_rope_table_of_far_positions(usm):
    x = got(usm.rope_table(1 << 20, 4))[-5:]
    p = np.arange((1 << 20) - 5, 1 << 20)[:, None] * np.array([1.0, 0.01])
    assert_near(x, np.concatenate([np.cos(p), np.sin(p)], 1), R.U + 2.0 ** -30)


APPENDS = {  # name -> (kv heads, q heads, D, rot, page, counts, lengths)
    "tokens": (2, 8, 64, 64, 16, [1, 1, 1, 1, 1], [1, 16, 17, 300, 32]),
    "ragged": (3, 3, 80, 40, 24, [5, 0, 33, 1, 0, 64], [5, 9, 50, 1, 0, 200]),
    "wide": (1, 4, 256, 256, 7, [3, 40], [3, 41]),
    "narrow": (2, 2, 8, 8, 1, [9, 2], [12, 2]),
    "part": (2, 4, 96, 32, 16, [4, 4, 4], [4, 20, 16]),
    "odd": (2, 4, 72, 20, 16, [7, 3], [7, 35]),
    "pairs": (1, 1, 16, 2, 5, [6], [30]),
    "many": (8, 32, 128, 128, 64, [700, 1, 90], [700, 100, 128]),
}


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", sorted(APPENDS))
def test_append(usm, name, dtype, interleaved):
    kv, heads, D, rot, page, counts, lengths = APPENDS[name]
    p = Problem(name, lengths, counts, heads=heads, kv=kv, D=D, page=page, dtype=dtype, before=2, behind=1)
    rope = R.rope_table(400, rot, 10000.0).astype(np.float32)
    if name == "many":
        rope = R.rope_table(800, rot, 10000.0).astype(np.float32)
    k, v = (rounded(p.rng.standard_normal((p.T, kv, D)), dtype) for _ in range(2))
    q, kc, vc, table, lens, offsets = p.on_device()
    q_out = put(np.full(p.q.shape, 55.0), dtype)
    r = usm.paged_append(put(k, dtype), put(v, dtype), kc, vc, table, lens, q_offsets=offsets, rope=dev(rope), q=q,
                         q_out=q_out, interleaved=interleaved)
    assert r is q_out
    f = lambda x: x.astype(np.float64)
    rk, rv, rq = R.append(f(k), f(v), f(p.k), f(p.v), p.table, p.lengths, p.counts, p.starts, f(rope), rot, interleaved, f(p.q))
    assert same_values(got(vc), rv)
    # Each turned element: two products and a sum in fp32, then the rounding.
    size = 2 * max(np.abs(k).max(), np.abs(p.q).max())
    near = lambda x, ref: assert_near(np.nan_to_num(x, nan=9.0), np.nan_to_num(ref, nan=9.0), 3 * R.U * size + R.HALF_STEP[dtype] * np.abs(np.nan_to_num(ref)), name)
    near(got(kc), rk)
    assert same_values(got(kc)[..., rot:], rk[..., rot:])
    idle = np.isnan(rq).all((1, 2))
    assert idle.sum() == 3 and np.all(got(q_out)[idle] == 55.0)
    near(got(q_out)[~idle], rq[~idle])


@pytest.mark.parametrize("dtype", TYPES)
def test_append_without_rotation_or_queries(usm, dtype):
    p = Problem("plain", [40, 3, 9], [4, 3, 0], kv=2, D=24, page=8, dtype=dtype)
    k, v = (rounded(p.rng.standard_normal((p.T, 2, 24)), dtype) for _ in range(2))
    k[0, 0, :3] = [np.nan, np.inf, -np.inf]  # stored as they are
    _, kc, vc, table, lens, offsets = p.on_device()
    assert usm.paged_append(put(k, dtype), put(v, dtype), kc, vc, table, lens, q_offsets=offsets) is None
    rk, rv, _ = R.append(k, v, p.k, p.v, p.table, p.lengths, p.counts, p.starts, None, 0, False)
    assert same_values(got(kc), rk) and same_values(got(vc), rv)


def test_append_skips_pages_that_are_not_there(usm):
    """Tokens past the table, at positions below zero, on pages outside the cache."""
    p = Problem("bad", [20, 2, 9, -3], [3, 5, 2, 1], kv=1, heads=2, D=32, page=4, dtype="f32", extra=0)
    p.table[0, 4] = 10**6            # position 19 of sequence 0 has page 4: outside
    p.table[2, 2] = -1               # position 8 of sequence 2
    p.table = p.table[:, :5]
    p.lengths[0] = 22                # positions 19, 20, 21: the last two past the table
    k, v = (rounded(p.rng.standard_normal((p.T, 1, 32)), "f32") for _ in range(2))
    rope = R.rope_table(6, 32, 100.0).astype(np.float32)  # positions past it take its last row
    q, kc, vc, table, lens, offsets = p.on_device()
    qo = usm.paged_append(put(k, "f32"), put(v, "f32"), kc, vc, table, lens, q_offsets=offsets, rope=dev(rope), q=q, q_out=q)
    lengths = np.maximum(p.lengths, 0)
    rk, rv, rq = R.append(k, v, p.k, p.v, p.table, lengths, p.counts, p.starts, rope, 32, False, p.q)
    assert same_values(got(vc), rv)
    assert_near(np.nan_to_num(got(kc)), np.nan_to_num(rk), 16 * R.U)
    assert_near(got(qo), rq, 16 * R.U)


@pytest.mark.parametrize("dtype", TYPES)
def test_append_takes_strides(usm, dtype):
    """Keys, values and queries as slices of one projection; caches with heads first."""
    import torch
    p = Problem("strides", [33, 8], [17, 8], heads=4, kv=2, D=64, page=16, dtype=dtype)
    x = rounded(p.rng.standard_normal((p.T, 8, 64)), dtype)
    X = put(x, dtype)
    q, k, v = X[:, :4], X[:, 4:6], X[:, 6:]
    rope = R.rope_table(64, 64, 10000.0).astype(np.float32)
    caches = []
    for first in (False, True):
        _, kc, vc, table, lens, offsets = p.on_device(heads_first=first)
        qo = usm.paged_append(k, v, kc, vc, table, lens, q_offsets=offsets, rope=dev(rope), q=q)
        caches.append((got(kc), got(vc), got(qo)))
    for a, b in zip(*caches):
        assert same_values(a, b)
    whole = usm.paged_append(k.contiguous(), v.contiguous(), *p.on_device()[1:3], table, lens, q_offsets=offsets,
                             rope=dev(rope), q=q.contiguous())
    assert same_values(got(whole), caches[0][2])
    # Rows that are not 16-byte aligned are copied first.
    off = torch.empty(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape).copy_(q)
    again = usm.paged_append(k, v, *p.on_device()[1:3], table, lens, q_offsets=offsets, rope=dev(rope), q=off)
    assert same_values(got(again), caches[0][2])


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
SHAPES = {  # name -> Problem's arguments
    "one": dict(lengths=[1], counts=[1], heads=1, kv=1),
    "token": dict(lengths=[1000], counts=[1], heads=8, kv=8),
    "tokens": dict(lengths=[1, 127, 128, 129, 2000, 0, 31], counts=[1] * 7, heads=8, kv=2, D=128),
    "tokens of 7 heads": dict(lengths=[500, 3, 77], counts=[1] * 3, heads=7, kv=1, D=80, page=24),
    "tokens of 64 heads": dict(lengths=[300, 40], counts=[1] * 2, heads=64, kv=1, D=64, page=32),
    "tokens of 300 heads": dict(lengths=[140, 12], counts=[1] * 2, heads=300, kv=1, D=32, page=32),
    "draft": dict(lengths=[260, 5, 1025], counts=[5] * 3, heads=8, kv=2, D=128, page=32),
    "prompt": dict(lengths=[300], counts=[300], heads=2, kv=2, D=64, page=64),
    "prompt of 257": dict(lengths=[257, 1], counts=[257, 1], heads=2, kv=1, D=128, page=128),
    "chunks": dict(lengths=[400, 130, 700, 20, 0], counts=[100, 130, 1, 0, 0], heads=6, kv=2, D=96, page=16, before=3,
                   behind=2),
    "pages of one": dict(lengths=[200, 90], counts=[3, 90], heads=4, kv=2, D=40, page=1),
    "large pages": dict(lengths=[333, 800], counts=[33, 8], heads=4, kv=4, D=64, page=500),
    "narrow": dict(lengths=[150, 64], counts=[20, 64], heads=4, kv=4, D=8, page=7),
    "width 136": dict(lengths=[150, 64], counts=[20, 64], heads=4, kv=2, D=136),
    "width 256": dict(lengths=[150, 700], counts=[20, 1], heads=4, kv=1, D=256),
    "more tokens than cache": dict(lengths=[5, 40], counts=[9, 50], heads=2, kv=1, D=64),
    "far apart": dict(lengths=[3000, 0, 2, 0, 0, 1500], counts=[2, 0, 1, 0, 0, 40], heads=4, kv=1, D=128, page=16),
}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", sorted(SHAPES))
def test_attention(usm, name, dtype):
    kw = dict(SHAPES[name])
    Problem(name, kw.pop("lengths"), kw.pop("counts"), dtype=dtype, **kw).check(usm)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 2, 100, 128, 129, 5000, 2**31 - 1])
@pytest.mark.parametrize("dtype", TYPES)
def test_windows(usm, dtype, window, causal):
    Problem("window", [300, 150, 513, 40], [150, 1, 260, 40], heads=4, kv=2, D=64, dtype=dtype).check(
        usm, window=window, causal=causal)


@pytest.mark.parametrize("dtype", TYPES)
def test_layout_of_the_cache(usm, dtype):
    p = Problem("layout", [300, 150], [30, 150], heads=4, kv=2, D=80, dtype=dtype)
    p.check(usm, heads_first=True)
    assert same_values(got(p.run(usm)), got(p.run(usm, heads_first=True)))


@pytest.mark.parametrize("dtype", TYPES)
def test_queries_and_outputs_with_strides(usm, dtype):
    import torch
    p = Problem("query strides", [300, 150], [30, 150], heads=4, kv=2, D=64, dtype=dtype)
    q, k, v, table, lens, offsets = p.on_device()
    plain = usm.paged_attention(q, k, v, table, lens, q_offsets=offsets)
    by_head = q.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty((4, p.T, 64 + 8), dtype=q.dtype, device="cuda").transpose(0, 1)[..., :64]
    usm.paged_attention(by_head, k, v, table, lens, q_offsets=offsets, out=out)
    assert torch.equal(out, plain)
    off = torch.empty(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape).copy_(q)
    assert torch.equal(usm.paged_attention(off, k, v, table, lens, q_offsets=offsets), plain)


@pytest.mark.parametrize("dtype", TYPES)
def test_shared_pages(usm, dtype):
    """Sequences with a common prefix list the same pages."""
    p = Problem("shared", [64, 64, 64], [1, 1, 1], heads=4, kv=2, D=64, dtype=dtype)
    p.table[1:, :3] = p.table[0, :3]
    p.check(usm)


@pytest.mark.parametrize("where", ["later tokens", "before the window", "seen"])
@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nan_in_values(usm, dtype, where):
    """What a token does not see never touches its row; what it sees does."""
    p = Problem("values", [300, 200], [150, 60], heads=4, kv=2, D=64, dtype=dtype)
    at = {"later tokens": 260, "before the window": 90, "seen": 20}[where]
    window = 100 if where == "before the window" else 0
    page, slot = p.table[0, at // 16], at % 16
    p.v[page, slot, 0, 5], p.v[page, slot, 0, 6], p.v[page, slot, 1, 7] = np.nan, np.inf, -np.inf
    p.k[page, slot, 1, 3] = np.nan if where != "seen" else 1.0
    import torch
    out = got(p.run(usm, window=window))
    with np.errstate(invalid="ignore"):
        ref, bound = p.reference(64 ** -0.5, window=window)
    finite = np.isfinite(ref)
    assert 0 < (~finite).sum() < ref.size
    assert np.array_equal(np.isfinite(out), finite)
    b = np.where(np.isfinite(bound), bound, 0)
    assert_near(np.where(finite, out, 0), np.where(finite, ref, 0), b)


@pytest.mark.parametrize("D", [24, 64, 128, 136, 200, 256])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("dtype", TYPES)
def test_single_tokens_of_few_rows(usm, dtype, group, D):
    Problem("few", [700, 33, 1], [1, 1, 1], heads=2 * group, kv=2, D=D, dtype=dtype).check(usm)


@pytest.mark.parametrize("length", [40, 1040])
@pytest.mark.parametrize("heads", [1, 2, 8])
@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f32", 160), ("bf16", 64), ("bf16", 160)])
def test_infinity_under_a_weight_of_zero(usm, dtype, D, heads, length):
    """An infinity that a token sees reaches its row although its weight is 0 in
    fp32 (0·inf is not finite either); the token before does not see it."""
    p = Problem("zero weight", [length], [3], heads=heads, kv=1, D=D, dtype=dtype)
    key = length - 2
    p.q[..., 0] = 40
    p.k[..., 0] = np.where(np.isnan(p.k[..., 0]), np.nan, 0)
    p.k[p.table[0, key // 16], key % 16, 0, 0] = -40  # 2^-2308 against a score of 0, the others within 2^60
    p.v[p.table[0, key // 16], key % 16, 0, 5] = np.inf
    seen = np.zeros((3, heads, D), bool)
    seen[1:, :, 5] = True
    assert np.array_equal(~np.isfinite(got(p.run(usm, scale=1.0))), seen)


@pytest.mark.parametrize("lengths", [[9], [3000], [700] * 40])
@pytest.mark.parametrize("heads,count", [(1, 1), (2, 1), (4, 1), (8, 1), (2, 45)])
@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f32", 160), ("bf16", 64), ("bf16", 160)])
def test_nan_in_a_query(usm, dtype, D, heads, count, lengths):
    """A token with a NaN gets NaN, however its keys are divided; its neighbours
    keep their bits."""
    p = Problem("query", lengths, [min(count, n) for n in lengths], heads=heads, kv=1, D=D, dtype=dtype)
    before = got(p.run(usm))
    p.q[-1, 0, 3] = np.nan
    x = got(p.run(usm))
    assert np.isnan(x[-1, 0]).all()
    x[-1, 0] = before[-1, 0]
    assert np.isfinite(before).all() and np.array_equal(x, before)


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_scores(usm, dtype):
    """Keys whose score is -inf weigh nothing; a row of them is zero."""
    p = Problem("masked", [200, 70], [20, 70], heads=2, kv=1, D=32, dtype=dtype)
    p.q[:] = np.abs(p.q) + 0.5
    for b, keys in ((0, range(0, 200, 3)), (1, range(70))):
        for j in keys:
            p.k[p.table[b, j // 16], j % 16, 0, 4] = -np.inf
    p.check(usm)


@pytest.mark.parametrize("size", [30.0, 3e3, 1e6, 1e16])
@pytest.mark.parametrize("dtype", TYPES)
def test_scores_far_from_zero(usm, dtype, size):
    """All scores of a row near one large value, of either sign."""
    for sign in (1.0, -1.0):
        p = Problem("far", [300, 40], [20, 40], heads=2, kv=1, D=32, dtype=dtype)
        p.k[..., 0], p.q[..., 0] = np.where(np.isnan(p.k[..., 0]), np.nan, sign * size), size
        p.k[..., 1:] = np.where(np.isnan(p.k[..., 1:]), np.nan, np.round(p.k[..., 1:]))
        p.q[..., 1:] = np.round(p.q[..., 1:])
        p.k, p.q = rounded(p.k, dtype), rounded(p.q, dtype)
        if size < 1e4:
            p.check(usm, scale=1.0)
        else:  # the other products are lost beside it in fp32: an average of values, whatever it is
            x = got(p.run(usm, 1.0))
            assert np.isfinite(x).all() and np.abs(x).max() <= np.nanmax(np.abs(p.v)) * 1.01
            assert np.abs(x).max(2).min() > 0


def test_rising_scores(usm):
    """A maximum that grows in every tile, by little and by much."""
    for step in (0.01, 1.0, 40.0):
        for dtype in TYPES:
            p = Problem("rising", [1500], [40], heads=2, kv=1, D=16, dtype=dtype)
            p.q[:] = 0
            p.q[..., 0] = 1
            j = np.arange(1500)
            p.k[p.table[0, j // 16], j % 16, 0, 0] = rounded(step * j, dtype)
            p.check(usm, scale=1.0)


def test_scale_of_zero(usm):
    for dtype in TYPES:
        Problem("zero", [300, 5], [40, 5], heads=2, kv=1, D=64, dtype=dtype).check(usm, scale=0.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_sequences(usm, dtype):
    """More sequences than a CTA has threads, many without new tokens."""
    rng = np.random.default_rng(5)
    counts = rng.integers(0, 4, 1300) * (rng.random(1300) < 0.4)
    counts[200:600] = 0
    lengths = counts + rng.integers(0, 40, 1300)
    Problem("many", lengths, counts, heads=2, kv=1, D=32, page=8, dtype=dtype, behind=4).check(usm)


@pytest.mark.parametrize("dtype", TYPES)
def test_one_long_sequence(usm, dtype):
    """One row over many CTAs, and a batch in which one sequence dwarfs the others."""
    Problem("long", [70000], [1], heads=1, kv=1, D=64, page=64, dtype=dtype).check(usm)
    Problem("dwarfs", [30, 40000, 7], [3, 2, 7], heads=3, kv=1, D=64, page=64, dtype=dtype).check(usm)


@pytest.mark.parametrize("dtype", TYPES)
def test_lengths_past_the_table(usm, dtype):
    """A length beyond the listed pages sees what they hold; negative ones nothing."""
    p = Problem("past", [64, 64, 10], [4, 70, 2], heads=2, kv=1, D=64, dtype=dtype, extra=0)
    p.lengths = np.array([66, 80, -5])
    scale = 0.125
    x = got(p.run(usm, scale))
    q = p.q.astype(np.float64)
    ref, bound = R.attention(q, p.k.astype(np.float64), p.v.astype(np.float64), p.table, np.maximum(p.lengths, 0),
                             p.counts, p.starts, scale, dtype=dtype)
    assert_near(x, ref, bound)


def test_same_bits_again(usm):
    for dtype in TYPES:
        p = Problem("again", [3000, 200, 900], [3, 200, 1], heads=8, kv=2, D=128, dtype=dtype)
        a = p.run(usm)
        for _ in range(3):
            assert same_values(got(p.run(usm)), got(a))


def test_no_tokens(usm):
    import torch
    for dtype in TYPES:
        p = Problem("none", [10, 20], [0, 0], heads=2, kv=1, D=64, dtype=dtype)
        assert p.run(usm).shape == (0, 2, 64)
        q, k, v, table, lens, offsets = p.on_device()
        empty = torch.empty((0, 1, 64), dtype=k.dtype, device="cuda")
        assert usm.paged_append(empty, empty, k, v, table, lens, q=q).shape == (0, 2, 64)


# ---------------------------------------------------------------------------
# Arguments, streams, graphs
# ---------------------------------------------------------------------------
def test_refusals(usm):
    import torch
    p = Problem("refusals", [30, 20], [2, 2], heads=4, kv=2, D=64)
    q, k, v, table, lens, _ = p.on_device()
    new = q[:, :2].contiguous()
    run = lambda **kw: usm.paged_attention(**{**dict(q=q, k_cache=k, v_cache=v, page_table=table, lengths=lens), **kw})
    add = lambda **kw: usm.paged_append(**{**dict(k=new, v=new, k_cache=k, v_cache=v, page_table=table, lengths=lens), **kw})
    for f in (run, add):
        for kw in (dict(k_cache=k.cpu()), dict(v_cache=v[:, :, :1]), dict(k_cache=k[0]), dict(page_table=table[0]),
                   dict(lengths=lens[:1]), dict(q_offsets=lens), dict(page_table=table.t()), dict(k_cache=None),
                   dict(k_cache=k.transpose(2, 3).contiguous().transpose(2, 3)[..., :64], v_cache=v)):
            with pytest.raises((ValueError, TypeError)):
                f(**kw)
        for kw in (dict(k_cache=k.float()), dict(lengths=lens.long()), dict(page_table=table.long()),
                   dict(k_cache=k.half(), v_cache=v.half())):
            with pytest.raises(TypeError):
                f(**kw)
    for kw in (dict(q=q[0]), dict(q=q[..., :32]), dict(out=q[:1]), dict(window=2**31), dict(out=q.cpu()), dict(q=None)):
        with pytest.raises(ValueError):
            run(**kw)
    for kw in (dict(q=q[:3]), dict(q=q[:, :3]), dict(scale=-1.0), dict(scale=float("nan")), dict(window=-1),
               dict(out=q[:1].expand(4, 4, 64))):
        with pytest.raises(usm.USMError):
            run(**kw)
    with pytest.raises(TypeError):
        run(q=q.float())
    for kw in (dict(v=new[:1]), dict(k=new[:, :1]), dict(q_out=q), dict(q=q, q_out=q[:1]),
               dict(rope=torch.zeros(8, 128, device="cuda")[:, ::2])):
        with pytest.raises(ValueError):
            add(**kw)
    for kw in (dict(rope=torch.zeros(8, 66, device="cuda")), dict(rope=torch.zeros(8, 7, device="cuda")),
               dict(rope=torch.zeros(0, 64, device="cuda"))):
        with pytest.raises(usm.USMError):
            add(**kw)
    with pytest.raises(usm.USMError):
        usm.rope_table(4, 3)
    with pytest.raises(usm.USMError):
        usm.rope_table(2**20, 2**20)
    assert usm.poll_status() == 0


def test_workspace_of_the_caller(usm):
    import torch
    p = Problem("workspace", [700, 90], [1, 90], heads=4, kv=2, D=64)
    a = p.run(usm)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")  # NaN in every word
    for _ in range(2):
        assert same_values(got(p.run(usm, workspace=ws)), got(a))
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    assert same_values(got(p.run(usm, workspace=small)), got(a))


def test_other_stream(usm):
    import torch
    p = Problem("stream", [900, 300], [1, 120], heads=4, kv=2, D=64)
    a = p.run(usm)
    q, k, v, table, lens, offsets = p.on_device()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = usm.paged_attention(q, k, v, table, lens, q_offsets=offsets, scale=0.125, stream=s)
    s.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
def test_captured(usm, dtype):
    """A decoding step captured once and replayed as the lengths grow, two graphs
    with one workspace in turn."""
    import torch
    p = Problem("graph", [40, 129, 290], [1, 1, 1], heads=4, kv=2, D=64, dtype=dtype)
    rope = usm.rope_table(512, 64)
    q, kc, vc, table, lens, _ = p.on_device()
    new_k, new_v = torch.randn_like(q[:, :2]), torch.randn_like(q[:, :2])
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")

    def step():
        turned = usm.paged_append(new_k, new_v, kc, vc, table, lens, rope=rope, q=q)
        return usm.paged_attention(turned, kc, vc, table, lens, scale=0.125, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for i in range(6):
        lens += 1
        new_k.normal_()
        new_v.normal_()
        q.normal_()
        graphs[i % 2].replay()
        first = outs[i % 2].clone()
        assert torch.equal(first, step())
        for c in (kc, vc):  # the new token is where it belongs
            for b in range(3):
                pos = int(lens[b]) - 1
                row = c[table[b, pos // 16].long(), pos % 16]
                assert torch.isfinite(row).all()
    assert usm.poll_status() == 0


# ---------------------------------------------------------------------------
# The calls together, and beside the library's other attention
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_in_chunks_equals_prompt_at_once(usm, dtype):
    """A prompt appended and attended in ragged chunks, then token by token, gives
    what the whole prompt gives, and both the dense definition."""
    import torch
    rng = np.random.default_rng(17)
    L, H, kv, D, size = 300, 4, 2, 64, 16
    q, k, v = (rounded(rng.standard_normal((L, n, D)), dtype) for n in (H, kv, kv))
    rope = usm.rope_table(L, D)
    table = ints(rng.permutation(19)[None])
    new = lambda: torch.full((19, size, kv, D), float("nan"), device="cuda", dtype=torch_type(dtype))
    Q, K, V = (put(x, dtype) for x in (q, k, v))

    def run(cuts):
        kc, vc, outs = new(), new(), []
        for a, b in zip(cuts[:-1], cuts[1:]):
            lens = ints([b])
            turned = usm.paged_append(K[a:b], V[a:b], kc, vc, table, lens, rope=rope, q=Q[a:b])
            outs.append(usm.paged_attention(turned, kc, vc, table, lens, scale=D ** -0.5))
        return got(torch.cat(outs)), got(kc)

    once, cache = run([0, L])
    parts, cache2 = run([0, 1, 17, 150, 278, 279, 280, 300])
    assert same_values(cache, cache2)
    t = got(rope)
    turned = lambda x: rounded(np.stack([R.rotate(x[p].astype(np.float64), t[p], D, False) for p in range(L)]), dtype)
    ref, bound = R.attention(turned(q).astype(np.float64), turned(k)[None].astype(np.float64), v[None].astype(np.float64),
                             np.zeros((1, 1), int), [L], [L], [0], D ** -0.5, dtype=dtype)
    # The turned rows may be a step apart where their fp32 value lies on a rounding's border.
    slack = 0.0 if dtype == "f32" else 2 * 2.0 ** -7 * np.abs(turned(q)).max() * np.abs(turned(k)).max() * D ** -0.5
    wide = bound + (4 * R.U * 64 + slack) * np.abs(v).max()
    assert_near(once, ref, wide)
    assert_near(parts, ref, wide)


@pytest.mark.parametrize("dtype", TYPES)
def test_beside_sparse_attention(usm, dtype):
    """The same cache, heads first, read by attention() through CSR rows that list
    every slot a token sees."""
    import torch
    p = Problem("beside", [130, 77], [1, 1], heads=2, kv=2, D=64, dtype=dtype, page=16)
    q, k, v, table, lens, _ = p.on_device(heads_first=True)
    dense = got(usm.paged_attention(q, k, v, table, lens, scale=0.125))
    slots = k.shape[0] * k.shape[1]
    rows, cols = [0], []
    for b in range(2):
        j = np.arange(p.lengths[b])
        at = np.sort(p.table[b, j // 16] * 16 + j % 16)
        for h in range(2):
            cols.append(h * slots + at)
            rows.append(rows[-1] + at.size)
    flat = lambda c: c.permute(2, 0, 1, 3).reshape(2 * slots, 64)
    listed = got(usm.attention(ints(rows), ints(np.concatenate(cols)), q.reshape(4, 64), flat(k), flat(v), scale=0.125))
    _, bound = p.reference(0.125)
    assert_near(dense.reshape(4, 64), listed, 2 * bound.reshape(4, 64))


# ---------------------------------------------------------------------------
# The ends of the ranges
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("seqs", [31, 32, 33, 127, 128, 129, 256, 257, 511, 512, 513])
def test_numbers_of_sequences(usm, dtype, seqs):
    """Around the sizes at which the division of the work changes its form."""
    rng = np.random.default_rng(seqs)
    counts = rng.integers(0, 3, seqs)
    counts[-1], counts[0] = 1, 0
    lengths = counts + rng.integers(0, 300, seqs) * (rng.random(seqs) < 0.3)
    Problem("numbers", lengths, counts, heads=4, kv=2, D=32, page=16, dtype=dtype).check(usm)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [1, 2, 4, 8, 12, 16, 64, 100, 128, 256, 384, 1000])
def test_page_sizes(usm, dtype, page):
    """Pages that divide a tile of keys, that tiles divide, and neither."""
    Problem("pages", [700, 129, 5, 384], [1, 129, 5, 3], heads=4, kv=2, D=72, page=page, dtype=dtype).check(usm, window=300)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 9, 17, 64, 127, 128, 129, 200, 255, 256, 257])
def test_numbers_of_heads(usm, dtype, group):
    """Query heads of a head of keys: rows of a token in one block of rows or several."""
    Problem("group", [90, 200], [3, 2], heads=group, kv=1, D=64, page=16, dtype=dtype).check(usm)


@pytest.mark.parametrize("dtype", TYPES)
def test_window_longer_than_any_position(usm, dtype):
    """Windows next to 2^31 with positions below zero, all keys in sight."""
    for window in (2**30 - 1, 2**30, 2**31 - 1):
        Problem("huge window", [5, 300], [9, 20], heads=2, kv=1, D=64, dtype=dtype).check(usm, window=window, causal=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_large_scales(usm, dtype):
    """A scale that makes the largest score the only one, up to the largest float."""
    p = Problem("scale", [150], [3], heads=1, kv=1, D=32, dtype=dtype)
    best = []
    for t in range(3):
        j = np.arange(147 + t + 1)
        x = p.k[p.table[0, j // 16], j % 16, 0].astype(np.float64) @ p.q[t, 0]
        best.append(p.v[p.table[0, j[x.argmax()] // 16], j[x.argmax()] % 16, 0])
    for scale in (1e6, 1e30, 3.4e38):
        x = got(p.run(usm, scale))[:, 0]
        assert_near(x, np.array(best, dtype=np.float64), R.HALF_STEP[dtype] * np.abs(best) + R.U)


@pytest.mark.parametrize("dtype", TYPES)
def test_cache_past_32_bits(usm, dtype):
    """Pages whose offset passes 2^31 elements, and 2^32 bytes."""
    import torch
    pages, size, kv, D = 17000, 16, 64, 128
    assert pages * size * kv * D > 2**31
    k = torch.empty((pages, size, kv, D), dtype=torch_type(dtype), device="cuda")
    v = torch.empty_like(k)
    p = Problem("far", [40, 20], [1, 20], heads=4, kv=2, D=D, page=size, dtype=dtype, extra=0)
    far = np.array([[16999, 3, 16998], [16390, 16997, 0]])
    table = np.zeros_like(p.table)
    for b in range(2):
        for i in range(-(-p.lengths[b] // size)):
            table[b, i] = far[b, i]
            k[far[b, i], :, 62:] = put(p.k[p.table[b, i]], dtype)
            v[far[b, i], :, 62:] = put(p.v[p.table[b, i]], dtype)
    _, _, _, _, lens, offsets = p.on_device()
    new = put(np.zeros((p.T, 2, D)), dtype)
    scale = D ** -0.5
    x = usm.paged_attention(put(p.q, dtype), k[:, :, 62:], v[:, :, 62:], ints(table), lens, q_offsets=offsets, scale=scale)
    ref, bound = p.reference(scale)
    assert_near(got(x), ref, bound)
    usm.paged_append(new + 3, new + 4, k[:, :, 62:], v[:, :, 62:], ints(table), lens, q_offsets=offsets)
    assert torch.all(k[far[0, 2], 39 % size, 62:] == 3) and torch.all(v[far[0, 2], 39 % size, 62:] == 4)
    assert torch.all(k[far[1, 0], :, 62:] == 3) and torch.all(v[far[1, 1], :4, 62:] == 4)


@pytest.mark.parametrize("dtype", TYPES)
def test_broadcast_queries(usm, dtype):
    """Rows of stride 0: one query for all tokens and heads, one key for all heads."""
    import torch
    p = Problem("broadcast", [300, 150], [30, 150], heads=4, kv=2, D=64, dtype=dtype)
    q, k, v, table, lens, offsets = p.on_device()
    one = q[:1, :1].expand(p.T, 4, 64)
    a = usm.paged_attention(one, k, v, table, lens, q_offsets=offsets)
    assert torch.equal(a, usm.paged_attention(one.contiguous(), k, v, table, lens, q_offsets=offsets))
    caches = [c.clone() for c in (k, v)]
    usm.paged_append(one[:, :2], one[:, :2], k, v, table, lens, q_offsets=offsets)
    usm.paged_append(one[:, :2].contiguous(), one[:, :2].contiguous(), *caches, table, lens, q_offsets=offsets)
    assert same_values(got(k), got(caches[0])) and same_values(got(v), got(caches[1]))


@pytest.mark.parametrize("dtype", TYPES)
def test_one_page_one_slot_one_head(usm, dtype):
    """Dimensions of one, whatever their strides."""
    import torch
    p = Problem("ones", [1], [1], heads=3, kv=1, D=64, page=1, dtype=dtype, spare=0, extra=0)
    q, k, v, table, lens, _ = p.on_device()
    odd = lambda c: torch.as_strided(c, c.shape, (1, 3, 5, 1))
    out = usm.paged_attention(q, odd(k), odd(v), table, lens)
    assert torch.equal(out, v.reshape(1, 1, 64).expand(1, 3, 64))


def test_two_calls_at_once(usm):
    """Calls on two streams, with other kernels of the library between them."""
    import torch
    ps = [Problem("first", [4000, 200, 900], [3, 200, 1], heads=8, kv=2, D=128), Problem("second", [3000] * 8, [1] * 8, heads=8, kv=8)]
    want = [p.run(usm, scale=0.125) for p in ps]
    args = [p.on_device() for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    outs = [[], []]
    for _ in range(20):
        for i, (q, k, v, table, lens, offsets) in enumerate(args):
            outs[i].append(usm.paged_attention(q, k, v, table, lens, q_offsets=offsets, scale=0.125, stream=streams[i]))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)
    assert usm.poll_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_junk_in_the_table_and_offsets(usm, dtype):
    """Arrays that break the contract give wrong numbers at most: wild pages in use,
    offsets out of order and out of range, lengths below zero and past the table."""
    import torch
    p = Problem("junk", [300, 150, 70], [30, 150, 2], heads=4, kv=2, D=64, dtype=dtype)
    q, k, v, table, lens, offsets = p.on_device()
    k, v = k.nan_to_num(0.0), v.nan_to_num(0.0)
    for bad in ([0, 500, -3, 182], [-2**31, 2**31 - 1, 5, 9], [182, 0, 182, 0]):
        usm.paged_attention(q, k, v, table, lens, q_offsets=ints(bad))
        usm.paged_append(q[:, :2], q[:, 2:], k, v, table, lens, q_offsets=ints(bad))
    for bad in ([-2**31, 2**31 - 1, 0], [10**6, -1, 300]):
        usm.paged_attention(q, k, v, table, ints(bad), q_offsets=offsets)
        usm.paged_append(q[:, :2], q[:, 2:], k, v, table, ints(bad), q_offsets=offsets)
    wild = p.rng.integers(-2**31, 2**31 - 1, table.shape)
    usm.paged_attention(q, k, v, ints(wild), lens, q_offsets=offsets)
    before = k.clone()
    usm.paged_append(q[:, :2], q[:, 2:], k, v, ints(wild), lens, q_offsets=offsets)
    assert torch.equal(k, before) or bool(((wild >= 0) & (wild < k.shape[0])).any())
    torch.cuda.synchronize()
    assert usm.poll_status() == 0


@pytest.mark.parametrize("page", [32, 24])
def test_few_rows_before_many(usm, page):
    """Blocks of few rows, whose halves leave their sums to one another, followed at
    once by blocks of many, whose queries take the same place."""
    import torch
    p = Problem("few and many", [827, 1700, 1309, 740, 1510], [101, 100, 94, 36, 79], heads=24, kv=3, D=80, page=page)
    p.check(usm)
    q, k, v, table, lens, offsets = p.on_device()
    q, lens = q.repeat(4, 1, 1), lens.repeat(4)
    counts = np.tile(p.counts, 4)
    offsets = ints(np.concatenate([[0], np.cumsum(counts)]))
    run = lambda: usm.paged_attention(q, k, v, table.repeat(4, 1), lens, q_offsets=offsets, scale=p.D ** -0.5)
    first = run()
    for part in first.split(p.T):
        # The same rows in another place of the batch: cut into parts elsewhere.
        assert_near(got(part), got(first[:p.T]), 3 * p.reference(p.D ** -0.5)[1])
    for _ in range(20):
        assert torch.equal(run(), first)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 2, 4, 5, 8, 9])
@pytest.mark.parametrize("width", [32, 64, 128, 136, 200, 256])
def test_single_tokens_of_all_widths(usm, width, rows, dtype):
    """Few rows a head of keys, around the sizes at which their kernel changes."""
    Problem("widths", [700, 3, 0, 130, 2000], [1] * 5, heads=2 * rows, kv=2, D=width, page=16, dtype=dtype).check(usm)
