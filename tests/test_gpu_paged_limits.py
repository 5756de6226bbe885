"""The paged cache where its calls could go wrong: precision of the weights,
sizes next to the limits, batches of unequal sequences, infinities under weights
of zero, calls beside other kernels.  Against the 64-bit definitions in paged_ref."""
import numpy as np
import pytest

import paged_ref as R
from test_gpu_paged import Problem, assert_near, got, rounded, torch_type

pytestmark = pytest.mark.gpu

TYPES = ("f32", "bf16")


# ---------------------------------------------------------------------------
# Precision
# ---------------------------------------------------------------------------
PRECISE = {  # name -> Problem's arguments
    "tokens": dict(lengths=[1000, 129, 2000], counts=[1] * 3, heads=8, kv=2, D=128),
    "draft": dict(lengths=[260, 1025], counts=[5] * 2, heads=8, kv=2, D=64, page=32),
    "chunk": dict(lengths=[700, 300], counts=[300, 300], heads=4, kv=2, D=128, page=64),
    "ragged": dict(lengths=[400, 130, 700], counts=[100, 130, 1], heads=6, kv=2, D=96, page=24),
    "wide": dict(lengths=[400, 130], counts=[100, 1], heads=4, kv=2, D=192),
}


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("name", sorted(PRECISE))
def test_weights_are_not_rounded_to_bf16(usm, name, window):
    """bf16 caches: beside the output's own rounding (2^-8) a weight is off by 2^-16 at
    most (its bf16 form leaves up to 2^-8 of it, held to 2^-8 again), and
    everything else as in fp32."""
    kw = dict(PRECISE[name])
    p = Problem(name, kw.pop("lengths"), kw.pop("counts"), dtype="bf16", **kw)
    scale = p.D ** -0.5
    x = got(p.run(usm, scale, window=window))
    args = lambda v: (p.q.astype(np.float64), p.k.astype(np.float64), v, p.table, p.lengths, p.counts, p.starts, scale)
    v = p.v.astype(np.float64)
    ref, bound = R.attention(*args(v), window=window, dtype="f32")
    mass, _ = R.attention(*args(np.abs(v)), window=window, dtype="f32")
    assert_near(x, ref, bound + 1.01 * 2.0 ** -16 * mass + R.HALF_STEP["bf16"] * np.abs(ref))


# ---------------------------------------------------------------------------
# Calls behind one another
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,D,count", [("f32", 64, 1), ("f32", 64, 40), ("f32", 160, 1), ("bf16", 160, 2), ("bf16", 64, 1), ("bf16", 128, 40)])
def test_results_of_the_call_before(usm, dtype, D, count):
    """Calls that follow one another at once, each reading what the last has written
    (slots, turned queries, lengths), give what they give one by one: kernels start
    before the last has ended, and read nothing of it before."""
    import torch
    p = Problem("behind", [300] * 12, [count] * 12, heads=4, kv=2, D=D, dtype=dtype)
    q0, kc0, vc0, table, lens0, _ = p.on_device()
    rope = usm.rope_table(512, D)
    new = torch.randn(8, 2, q0.shape[0], 2, D, device="cuda").to(q0.dtype)

    def run(after):
        kc, vc, lens, q, outs = kc0.clone(), vc0.clone(), lens0 - 8, q0.clone(), []
        after()
        for k, v in new:
            lens = lens + 1
            after()
            q = usm.paged_append(k, v, kc, vc, table, lens, rope=rope, q=q)
            after()
            outs.append(usm.paged_attention(q, kc, vc, table, lens, scale=D ** -0.5))
            after()
            q = outs[-1]
        torch.cuda.synchronize()
        return torch.stack(outs), kc, vc

    want = run(torch.cuda.synchronize)
    assert torch.isfinite(want[0]).all()
    for _ in range(5):
        assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(want, run(lambda: None)))


# ---------------------------------------------------------------------------
# Next to the limits
# ---------------------------------------------------------------------------
def test_append_of_nearly_2_to_31_heads(usm):
    """tokens·heads next to 2^31: the last step over the heads passes it."""
    import torch
    D, heads = 8, 2**31 - 3  # and one of keys, one of values
    q = torch.empty((1, heads, D), dtype=torch.bfloat16, device="cuda")
    q.view(-1)[: 1 << 20].normal_()
    tail = 1 << 12
    q[:, -tail:].normal_()
    k, v = torch.randn(2, 1, 1, D, device="cuda").bfloat16()
    kc, vc = torch.zeros(2, 1, 4, 1, D, device="cuda", dtype=torch.bfloat16)
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.full((1,), 3, dtype=torch.int32, device="cuda")
    rope = usm.rope_table(4, D)
    parts = [slice(0, 1000), slice(heads - tail, heads)]
    call = lambda x: usm.paged_append(k, v, kc, vc, table, lens, rope=rope, interleaved=True, q=x, q_out=x)
    want = [call(q[:, s].clone()) for s in parts]
    kc.zero_(), vc.zero_()
    call(q)
    for s, w in zip(parts, want):
        assert torch.equal(q[:, s], w)
    assert torch.equal(vc[0, 2], v[0]) and kc[0, 2].abs().sum() > 0
    assert not vc[0, [0, 1, 3]].any() and not kc[0, [0, 1, 3]].any()


def test_heads_and_positions_past_32_bits_are_refused(usm):
    """Numbers that the library's 32-bit arguments would cut to small ones."""
    import torch
    t = torch.zeros(8, device="cuda", dtype=torch.bfloat16)
    k, cache = t.view(1, 1, 8), t.clone().view(1, 1, 1, 8)
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    add = lambda **kw: usm.paged_append(k, k, cache, cache.clone(), table, lens, **kw)
    many = k.expand(1, 2**32 + 4, 8)
    with pytest.raises(ValueError):
        add(q=many, q_out=many)
    rope = torch.empty((2**32 + 5, 2), device="cuda")
    with pytest.raises(ValueError):
        add(rope=rope)
    with pytest.raises(ValueError):
        usm.paged_attention(many, cache, cache, table, lens)


@pytest.mark.parametrize("tokens,heads", [(1, 2**31 - 1), (2**31 - 1, 1), (2**16, 2**15 - 1)])
@pytest.mark.parametrize("dtype,D", [("f32", 4), ("bf16", 8)])
def test_attention_of_nearly_2_to_31_rows(usm, dtype, D, tokens, heads):
    """tokens·heads next to 2^31, all rows the same query: all give its row.  (Not to the
    last bit: a block of rows that a CTA's share cuts is the sum of two parts, in
    another order than that of whole ones, within the bound of any order.)"""
    import torch
    t = torch_type(dtype)
    q = torch.randn(1, 1, D, device="cuda").to(t)
    k, v = torch.randn(2, 1, 100, 1, D, device="cuda").to(t)
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.full((1,), 100, dtype=torch.int32, device="cuda")
    out = torch.full((tokens, heads, D), 7.0, dtype=t, device="cuda")
    usm.paged_attention(q.expand(tokens, heads, D), k, v, table, lens, causal=False, out=out)
    ref, bound = R.attention(got(q), got(k), got(v), np.zeros((1, 1), int), [100], [1], [0], 1.0, causal=False, dtype=dtype)
    for rows in out.view(-1, D).split(1 << 28):
        for c in range(D):
            low, high = (float(x) for x in rows[:, c].aminmax())
            assert abs(low - ref[0, 0, c]) <= bound[0, 0, c] and abs(high - ref[0, 0, c]) <= bound[0, 0, c]
    assert usm.poll_status() == 0


@pytest.mark.parametrize("page", [4096, 3000])
def test_items_that_take_seconds(usm, page):
    """2^30 tokens of a cache (one page listed over and over) before 256 rows of each of
    24 heads: an item's tiles take longer than a wait's limit, which counts from the
    last tile.  One key of the page outweighs all others, so that every sum is exact."""
    import torch
    kv, group, D = 24, 256, 64
    k = torch.randn(1, page, kv, D, device="cuda").bfloat16()
    v = torch.randn(1, page, kv, D, device="cuda").bfloat16()
    k[..., 0], k[:, 77, :, 0] = -50, 50
    v[:, 77] = torch.randint(-8, 9, (1, kv, D), device="cuda").bfloat16()
    q = torch.randn(1, kv * group, D, device="cuda").bfloat16()
    q[..., 0] = 4
    pages = 2**30 // page
    lens = torch.full((1,), pages * page - 1, dtype=torch.int32, device="cuda")
    out = usm.paged_attention(q, k, v, torch.zeros((1, pages), dtype=torch.int32, device="cuda"), lens)
    want = v[:, 77].repeat_interleave(group, 1)
    assert torch.equal(out, want)
    assert usm.poll_status() == 0


# ---------------------------------------------------------------------------
# Infinities under weights of zero
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("keys", ["some", "all"])
@pytest.mark.parametrize("length", [40, 1040, 20000])
@pytest.mark.parametrize("heads", [1, 2, 4, 8, 40])
@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f32", 160), ("bf16", 64), ("bf16", 160)])
def test_infinity_under_a_score_of_minus_infinity(usm, dtype, D, heads, length, keys):
    """A score of -inf weighs nothing, and nothing times an infinity is NaN: the
    infinity reaches the rows that see it however the keys are divided among lanes,
    warps and CTAs (whose whole share may be such keys), and no others."""
    p = Problem("minus infinity", [length], [3], heads=heads, kv=1, D=D, dtype=dtype)
    p.q[..., 0] = 1
    j = np.arange(length)
    hidden = j if keys == "all" else j[: length * 3 // 4]
    p.k[p.table[0, hidden // 16], hidden % 16, 0, 0] = -np.inf
    for key in (length // 3, length - 2):  # seen by all three tokens, by the last two
        p.v[p.table[0, key // 16], key % 16, 0, 5 + (key == length - 2)] = np.inf
    seen = np.zeros((3, heads, D), bool)
    seen[:, :, 5], seen[1:, :, 6] = True, True
    out = got(p.run(usm))
    assert np.array_equal(~np.isfinite(out), seen)
    if keys == "all":
        assert not out[~seen].any()


# ---------------------------------------------------------------------------
# Batches of unequal sequences
# ---------------------------------------------------------------------------
UNEQUAL = {  # new tokens of each sequence
    "chunk and idle": [70] + [0] * 20,
    "chunk and single": [90] + [1] * 15,
    "few and many": [1, 2, 3, 4, 5, 7, 8, 9, 10, 16, 17, 0, 33],
    "small": [3, 0, 2],
}


@pytest.mark.parametrize("group", [1, 2, 3, 4, 8, 9])
@pytest.mark.parametrize("name", sorted(UNEQUAL))
@pytest.mark.parametrize("dtype,D", [("f32", 40), ("f32", 128), ("f32", 200), ("bf16", 136), ("bf16", 256), ("bf16", 64)])
def test_unequal_sequences(usm, dtype, D, name, group):
    """Sequences of few rows and of many in one call, on either side of the number of
    rows that parts them, with sequences that bring nothing between them."""
    counts = UNEQUAL[name]
    rng = np.random.default_rng(len(counts))
    lengths = np.array(counts) + rng.integers(0, 400, len(counts))
    Problem(name, lengths, counts, heads=2 * group, kv=2, D=D, dtype=dtype, before=1, behind=2).check(usm)


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 192)])
@pytest.mark.parametrize("others", [0, 1])
def test_others_do_not_change_how_a_chunk_is_read(usm, dtype, D, others):
    """A chunk among sequences that bring nothing, or a token each (of one key), takes
    about the time that it takes alone: its rows still share the keys.  (By the
    average number of rows it would be read two or four rows at a time, in 128
    walks over the cache instead of four.)"""
    import torch
    chunk, length, seqs, kv = 256, 8192, 256 if others else 128, 8
    t = torch_type(dtype)
    k, v = torch.randn(2, length // 16, 16, kv, D, device="cuda").to(t)
    q = torch.randn(chunk + others * (seqs - 1), kv, D, device="cuda").to(t)
    table = torch.zeros((seqs, length // 16), dtype=torch.int32, device="cuda")
    table[0] = torch.arange(length // 16, device="cuda")
    lens = torch.ones(seqs, dtype=torch.int32, device="cuda")
    lens[0] = length
    offsets = chunk + others * torch.arange(-1, seqs, device="cuda", dtype=torch.int32)
    offsets[0] = 0

    def time(n, seqs):
        run = lambda: usm.paged_attention(q[:n], k, v, table[:seqs], lens[:seqs], q_offsets=offsets[: seqs + 1], scale=D ** -0.5)
        best = []
        for _ in range(10):
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            begin.record()
            out = run()
            end.record()
            torch.cuda.synchronize()
            best.append(begin.elapsed_time(end))
        return min(best), out

    alone, want = time(chunk, 1)
    among, out = time(q.shape[0], seqs)
    print(f"{dtype} {D}: {1e3 * alone:.0f} us alone, {1e3 * among:.0f} among others")
    assert (out[:chunk].float() - want.float()).abs().max() < 0.01
    assert among < 2 * alone


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 64), ("bf16", 128), ("bf16", 192)])
@pytest.mark.parametrize("count", [1, 3])
def test_workspace_of_equal_shares(usm, dtype, D, count):
    """The workspace of a batch whose sequences bring as many tokens each is that of one
    sequence: a call takes no more, and is content with it."""
    import torch
    p = Problem("equal", [300] * 64, [count] * 64, heads=8, kv=2, D=D, dtype=dtype)
    one = usm.load().paged_attention_workspace_bytes(count, 1, 8, 2, D, 0 if dtype == "f32" else 1)
    assert 0 < one <= usm.load().paged_attention_workspace_bytes(64 * count, 64, 8, 2, D, 0 if dtype == "f32" else 1)
    q, k, v, table, lens, offsets = p.on_device()
    assert offsets is None
    run = lambda **kw: usm.paged_attention(q, k, v, table, lens, scale=D ** -0.5, **kw)
    want = run()
    torch.cuda.synchronize()
    # Bytes asked for: those allocated depend on the blocks that the allocator has at hand.
    asked = lambda which: torch.cuda.memory_stats()[f"requested_bytes.all.{which}"]
    before = asked("current")
    torch.cuda.reset_peak_memory_stats()
    out = run()
    taken = asked("peak") - before
    assert taken == one + out.numel() * out.element_size(), (taken, one)
    ws = torch.empty(one, dtype=torch.uint8, device="cuda")
    assert torch.equal(run(workspace=ws), want)
    p.check(usm)


def test_calls_beside_other_kernels(usm):
    """Attention and appends on one stream, the library's sparse products (which use
    tensor memory too) and sparse attention on another, at once."""
    import torch
    import workloads as W
    p = Problem("beside others", [4000, 200, 900], [3, 200, 1], heads=8, kv=2, D=128)
    q, k, v, table, lens, offsets = p.on_device()
    rope = usm.rope_table(4096, 128)
    new = torch.randn(2, q.shape[0], 2, 128, device="cuda").bfloat16()
    csr = W.random_csr(3, 1024, 1024, 0.3)
    ro, ci = (torch.from_numpy(x).cuda() for x in (csr.row_offsets, csr.col_indices))
    val, B = torch.randn(ci.numel(), device="cuda"), torch.randn(1024, 2048, device="cuda")
    X, Y = (torch.randn(1024, 256, device="cuda").bfloat16() for _ in range(2))

    def paged():
        turned = usm.paged_append(new[0], new[1], k, v, table, lens, q_offsets=offsets, rope=rope, q=q)
        return usm.paged_attention(turned, k, v, table, lens, q_offsets=offsets, scale=0.1)

    def sparse():
        return [usm.spmm(ro, ci, val, B), usm.spmm(ro, ci, val.bfloat16(), B.bfloat16()), usm.sddmm(ro, ci, X, Y)]

    want, others = paged(), sparse()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got_a, got_b = [], []
    for _ in range(20):
        with torch.cuda.stream(a):
            got_a.append(paged())
        with torch.cuda.stream(b):
            got_b.append(sparse())
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got_a)
    assert all(torch.equal(x, y) for g in got_b for x, y in zip(g, others))
    assert usm.poll_status() == 0


@pytest.mark.parametrize("where", [130, 300])
def test_weights_of_different_references(usm, where):
    """Scores that are whole numbers far from zero, and so exact: a tile of keys at S and one
    key at S + 6 whose tile raises the reference (key 300: in the same half as the
    first tile; 130: in the other).  Their weights have to keep their ratio; V is chosen
    so that both nearly cancel.  Bounds: 2^-16 a weight, 130 additions, the power of
    two, the output's step."""
    scores = 20 + 47 * np.arange(60)
    p = Problem("references", [where + 1] * 60, [1] * 60, heads=1, kv=1, D=16, page=128)
    p.q[:] = 0
    p.q[..., 0] = p.q[..., 1] = 1
    for b, s in enumerate(scores):
        j = np.arange(where + 1)
        at = p.table[b, j // 128], j % 128, 0
        p.k[at], p.v[at] = 0, 0
        high, low = int(s) // 16 * 16, int(s) % 16  # both exact in bf16
        p.k[(*at, 0)] = np.where(j < 128, high, -500)
        p.k[(*at, 1)] = np.where(j < 128, low, -500)
        p.v[(*at, 0)] = 1
        heavy = p.table[b, where // 128], where % 128, 0
        p.k[(*heavy, 0)], p.k[(*heavy, 1)] = high, low + 6
        p.v[(*heavy, 0)] = -0.31640625
    p.k, p.v = rounded(p.k, "bf16"), rounded(p.v, "bf16")
    x = got(p.run(usm, scale=1.0))[:, 0, 0]
    w = np.exp(6.0)
    ref, mass = (128 - w * 0.31640625) / (128 + w), (128 + w * 0.31640625) / (128 + w)
    bound = (1.01 * 2.0 ** -16 + 2 * 138 * R.U + 2.0 ** -21) * mass + R.HALF_STEP["bf16"] * abs(ref)
    exact = p.k[p.table[:, 0], 0, 0, :2].sum(1)
    assert np.array_equal(exact, scores)
    off = np.abs(x - ref)
    assert off.max() <= bound, (off.max(), bound, scores[off.argmax()])


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 192), ("bf16", 64)])
def test_captured_with_unequal_sequences(usm, dtype, D):
    """A call captured once and replayed as its tokens change hands: sequences pass from
    few rows to many and back, with one workspace that two graphs share."""
    import torch
    total, heads, kv, size = 120, 4, 2, 16
    shares = [[100, 20], [1, 119], [119, 1], [60, 60], [0, 120], [116, 4], [4, 112]]
    p = Problem("captured", [700, 500], [100, 20], heads=heads, kv=kv, D=D, dtype=dtype, page=size)
    q, k, v, table, lens, offsets = p.on_device()
    need = usm.load().paged_attention_workspace_bytes(total, 2, heads, kv, D, 0 if dtype == "f32" else 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    run = lambda **kw: usm.paged_attention(q, k, v, table, lens, q_offsets=offsets, scale=D ** -0.5, workspace=ws, **kw)
    run()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    for i, counts in enumerate(shares):
        p.counts = np.array(counts)
        p.starts = np.cumsum(p.counts) - p.counts
        offsets.copy_(torch.tensor([0, counts[0], sum(counts)], dtype=torch.int32))
        out = outs[i % 2]
        out.fill_(77.0)
        graphs[i % 2].replay()
        ref, bound = p.reference(D ** -0.5)
        n = sum(counts)
        assert_near(got(out)[:n], ref[:n], bound[:n], counts)
        assert bool((out[n:] == 77.0).all())
        graphs[1 - i % 2].replay()
        assert torch.equal(outs[1 - i % 2][:n], out[:n])
    assert usm.poll_status() == 0
