"""Cases for the paged cache of keys and values: appending new tokens to it
with the position rotation applied on the way, and attention of a chunk of new
tokens (one or many of each sequence) over it.

`run` computes each in a plain form with elementary torch operations, or, with
`own` set, with the library's calls.  `exact` computes the same in 64 bits from
the definitions.

Layout of every case: sequence b of `batch` brings n_b new tokens and has
`lengths[b]` tokens in its cache with those included, so that its i-th new token
stands at position lengths[b] - n_b + i.  Caches are pages x `page` slots x
`kv` heads x `D`; position p of sequence b lies in slot p % page of page
page_table[b][p // page].  The new tokens of all sequences follow one another
in q (tokens x `heads` x D), k and v (tokens x `kv` x D).  Query head h reads
kv head h // (heads // kv).
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _case(op, name=None, **kw):
    c = dict(op=op, batch=1, new=1, ragged=False, singles=0, cache=4096, spread=0.0, heads=8, kv=8, D=64, page=16,
             dtype="bf16", window=0, rot=0, interleaved=False)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # One new token for each of 32 sequences: what every layer of a decoding step appends.
        _case("append", "append token 32x1", batch=32, cache=2048, spread=0.5, heads=32, kv=8, D=128, rot=128),
        # Four prompts of 4096 tokens.
        _case("append", "append prompt 4x4096", batch=4, new=4096, heads=32, kv=8, D=128, rot=128, page=64),
        # Ragged chunks, half of each head rotated in neighbouring pairs, pages that are no power of two.
        _case("append", "append odd 7x333", batch=7, new=333, ragged=True, cache=1531, spread=0.5, heads=9, kv=3, D=80,
              rot=40, interleaved=True, page=24, dtype="f32"),
        # One new token of one sequence, the library's attention sizes: the latency of the smallest call.
        _case("attention", "attention token 1x1", cache=4096),
        # A decoding step of 64 sequences whose caches are filled to different lengths.
        _case("attention", "attention batch 64x1", batch=64, cache=8192, spread=0.5, heads=32, kv=8, D=128),
        # Five tokens of each sequence at once: a draft that is being verified.
        _case("attention", "attention draft 24x5", batch=24, new=5, cache=4096, spread=0.7, heads=32, kv=8, D=128, page=32),
        # The prompt of the library's attention configuration, all of it new.
        _case("attention", "attention prompt 8x4096", new=4096, cache=4096, page=64),
        # A long prompt in chunks: 2048 new tokens of two sequences over caches of up to 16384.
        _case("attention", "attention chunk 2x2048", batch=2, new=2048, cache=16384, spread=0.1, heads=32, kv=8, D=128, page=64),
        # A served batch: the chunk of one sequence beside the single tokens of 16.
        _case("attention", "attention mixed 1000+16", batch=17, new=1000, singles=16, cache=4096, spread=0.5, heads=16, kv=2, D=128),
        # A layer with local attention over a long document, heads of an odd width.
        _case("attention", "attention local 1x16384", new=16384, cache=16384, window=1024, heads=8, kv=4, D=96, page=32),
        # Single tokens in fp32.
        _case("attention", "attention f32 16x1", batch=16, cache=4096, spread=0.3, dtype="f32"),
        # Ragged chunks in fp32 with odd sizes throughout.
        _case("attention", "attention f32 odd 5x211", batch=5, new=211, ragged=True, cache=1531, spread=0.6, heads=6, kv=3, D=80,
              page=24, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "attention"])
    kv = rng.choice([1, 2, 3, 4, 8])
    kw = dict(kv=kv, heads=kv * rng.choice([1, 1, 2, 3, 4, 7, 8]), D=rng.choice([32, 40, 64, 80, 96, 128, 128]),
              page=rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256]), dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]),
              batch=_log_int(rng, 1, 64), spread=rng.choice([0.0, 0.3, 0.9]), ragged=rng.random() < 0.5)
    kw["cache"] = _log_int(rng, 64, 16384)
    new = rng.choice([1, _log_int(rng, 1, 16), _log_int(rng, 2, 4096), _log_int(rng, 2, 4096)])
    kw["new"] = new = min(new, kw["cache"])
    # A pass costs no more than the largest listed ones (rows as the plain forms pad them).
    most = 2**31 // 8 if kw["dtype"] == "bf16" else 2**28 // 8
    while kw["batch"] > 1 and kw["batch"] * (new * kw["heads"] + 64 * kv) * kw["cache"] > most:
        kw["batch"] = (kw["batch"] + 1) // 2
    while kw["new"] > 1 and kw["batch"] * (kw["new"] * kw["heads"] + 64 * kv) * kw["cache"] > most:
        kw["new"] = (kw["new"] + 1) // 2
    if op == "attention":
        kw["window"] = rng.choice([0, 0, 0, _log_int(rng, 1, 4096)])
        kw["singles"] = rng.choice([0, rng.randint(0, kw["batch"] - 1)])
    else:
        kw["interleaved"] = rng.random() < 0.5
        kw["rot"] = rng.choice([0, kw["D"], kw["D"], kw["D"] // 2])
    return _case(op, **kw)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _shape(case):
    """New tokens and cache lengths of each sequence: a case's own, whatever
    the seed of its inputs.  The first `singles` sequences bring one token."""
    rng = np.random.default_rng([case["batch"], case["new"], case["cache"], case["heads"]])
    n = np.full(case["batch"], case["new"])
    if case["ragged"] and case["batch"] > 1:
        n = rng.integers(0, case["new"] + 1, case["batch"])
        n[-1] = case["new"]
    n[: case["singles"]] = 1
    lengths = np.rint(case["cache"] * (1 - case["spread"] * rng.random(case["batch"]))).astype(np.int64)
    lengths[0] = case["cache"]
    return n, np.maximum(lengths, n)


def _torch_dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _pages(case, lengths):
    return -(-lengths // case["page"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _torch_dtype(case)
    n, lengths = _shape(case)
    per = _pages(case, lengths)
    # The pages of all sequences, dealt out in random order, a few of them free.
    total = int(per.sum())
    order = torch.randperm(total + 3, generator=gen, device="cuda").to(torch.int32)
    first = torch.from_numpy(np.cumsum(per) - per).cuda()
    at = torch.arange(int(per.max()), device="cuda")
    real = at < torch.from_numpy(per).cuda()[:, None]
    table = torch.where(real, order[(first[:, None] + at).clamp(max=total - 1)], -1).to(torch.int32)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dt)

    T, D, kv = int(n.sum()), case["D"], case["kv"]
    offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).to(torch.int32).cuda()
    s = dict(case=case, table=table, lengths=torch.from_numpy(lengths).to(torch.int32).cuda(),
             # Where every sequence brings the same number of tokens no offsets are needed.
             offsets=None if (n == n[0]).all() else offsets, n=n, most=int(n.max()), longest=int(lengths.max()),
             k_cache=randn(total + 3, case["page"], kv, D), v_cache=randn(total + 3, case["page"], kv, D),
             q=randn(T, case["heads"], D))
    if case["op"] == "append":
        s["k"], s["v"] = randn(T, kv, D), randn(T, kv, D)
        if case["rot"]:
            j = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
            angle = torch.arange(case["cache"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2 * j / case["rot"])
            s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    return s


# ---------------------------------------------------------------------------
# The operators' plain forms
# ---------------------------------------------------------------------------
def _tokens(s):
    """Sequence and position of every new token."""
    c = s["case"]
    lengths = s["lengths"].long()
    if s["offsets"] is None:
        b = torch.arange(c["batch"], device="cuda").repeat_interleave(s["most"])
        i = torch.arange(s["most"], device="cuda").repeat(c["batch"])
        return b, i, lengths[b] - s["most"] + i
    offsets = s["offsets"].long()
    n = offsets[1:] - offsets[:-1]
    b = torch.repeat_interleave(torch.arange(c["batch"], device="cuda"), n, output_size=s["q"].shape[0])
    i = torch.arange(b.numel(), device="cuda") - offsets[b]
    return b, i, lengths[b] - n[b] + i


def _rotate(s, x, position):
    c, R = s["case"], s["case"]["rot"]
    x = x.float()
    if R == 0:
        return x
    cos, sin = s["rope"][position][:, None, :].split(R // 2, 2)
    if c["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
    else:
        a, b = x[..., : R // 2], x[..., R // 2 : R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
    return torch.cat([turned, x[..., R:]], 2)


def _plain_append(s):
    c, dt = s["case"], _torch_dtype(s["case"])
    b, _, position = _tokens(s)
    page = s["table"].long()[b, torch.div(position, c["page"], rounding_mode="floor")]
    s["k_cache"][page, position % c["page"]] = _rotate(s, s["k"], position).to(dt)
    s["v_cache"][page, position % c["page"]] = s["v"]
    return s["k_cache"], s["v_cache"], _rotate(s, s["q"], position).to(dt)


def _plain_attention(s):
    c = s["case"]
    B, kv, G, D, L = c["batch"], c["kv"], c["heads"] // c["kv"], c["D"], s["longest"]
    b, i, position = _tokens(s)
    key = torch.arange(L, device="cuda")
    page = s["table"].long()[:, torch.div(key, c["page"], rounding_mode="floor")].clamp(min=0)
    there = key < s["lengths"].long()[:, None]
    K = s["k_cache"][page, key % c["page"]].float()  # B x L x kv x D
    V = s["v_cache"][page, key % c["page"]].float().masked_fill(~there[:, :, None, None], 0.0)
    # Rows padded to the longest chunk; a padded row looks at the first key.
    q = torch.zeros(B, s["most"], c["heads"], D, device="cuda")
    q[b, i] = s["q"].float()
    p = torch.zeros(B, s["most"], dtype=torch.long, device="cuda")
    p[b, i] = position
    seen = (key <= p[:, :, None]) & there[:, None, :]
    if c["window"]:
        seen &= key > p[:, :, None] - c["window"]
    q = q.reshape(B, s["most"], kv, G, D).permute(0, 2, 3, 1, 4).reshape(B * kv, G * s["most"], D)
    x = torch.bmm(q, K.permute(0, 2, 3, 1).reshape(B * kv, D, L)).mul_(D**-0.5).reshape(B, kv * G, s["most"], L)
    x.masked_fill_(~seen[:, None], -math.inf)
    x = x.sub_(x.amax(3, keepdim=True).clamp(min=-3e38)).exp_()
    x = x.div_(x.sum(3, keepdim=True).clamp(min=1e-30)).reshape(B * kv, G * s["most"], L)
    out = torch.bmm(x, V.permute(0, 2, 1, 3).reshape(B * kv, L, D)).reshape(B, c["heads"], s["most"], D)
    return out[b, :, i].to(_torch_dtype(c))


def run(s):
    if own:
        return _run_own(s)
    return _plain_append(s) if s["case"]["op"] == "append" else _plain_attention(s)


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    import unstructured_sparse_matmul_gb300 as usm
    c = s["case"]
    if c["op"] == "append":
        q = usm.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], q_offsets=s["offsets"],
                             rope=s.get("rope"), interleaved=c["interleaved"], q=s["q"])
        return s["k_cache"], s["v_cache"], q
    return usm.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], q_offsets=s["offsets"],
                               scale=c["D"] ** -0.5, window=c["window"])


# ---------------------------------------------------------------------------
# Bytes and operations of one pass
# ---------------------------------------------------------------------------
def work(case):
    n, lengths = _shape(case)
    es = 2 if case["dtype"] == "bf16" else 4
    T, D, kv, heads, R = int(n.sum()), case["D"], case["kv"], case["heads"], case["rot"]
    first = lengths - n  # position of each sequence's first new token
    indices = 4 * (2 * case["batch"] + int(_pages(case, lengths).sum()))
    if case["op"] == "append":
        distinct = min(case["cache"], T)
        return {"bytes": 2 * es * T * D * (heads + 2 * kv) + 4 * R * distinct + indices, "flops": 3 * T * R * (heads + kv)}
    w = case["window"] or int(lengths.max())
    # Keys that the tokens at positions first..lengths-1 see: min(position + 1, window) each.
    up_to = lambda p: np.minimum(p, w) * (np.minimum(p, w) + 1) // 2 + np.maximum(p - w, 0) * w  # noqa: E731
    pairs = int((up_to(lengths) - up_to(first)).sum())
    keys = int(np.where(n > 0, lengths - np.maximum(first - w + 1, 0), 0).sum())
    return {"bytes": 2 * es * (keys * kv * D + T * heads * D) + indices, "flops": 4 * pairs * heads * D}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    n, lengths = _shape(case)
    ends = np.cumsum(n)
    table = s["table"].cpu().numpy().astype(np.int64)
    slots = [torch.from_numpy(table[b][np.arange(L) // case["page"]] * case["page"] + np.arange(L) % case["page"]).cuda()
             for b, L in enumerate(lengths)]
    flat = {k: s[k].double().reshape(-1, case["kv"], case["D"]) for k in ("k_cache", "v_cache")}
    if case["op"] == "append":
        R = case["rot"]
        q, k = s["q"].double(), s["k"].double()
        pairs = np.arange(R).reshape(-1, 2).T if case["interleaved"] else np.arange(R).reshape(2, -1)
        lower, upper = (torch.from_numpy(x).cuda() for x in pairs)
        for b, end in enumerate(ends):
            here = slice(end - n[b], end)
            if R:
                z = s["rope"][lengths[b] - n[b] : lengths[b]].double()
                z = torch.complex(z[:, : R // 2], z[:, R // 2 :])[:, None, :]
                for x in (q, k):
                    turned = torch.complex(x[here][..., lower], x[here][..., upper]) * z
                    x[here, :, lower], x[here, :, upper] = turned.real, turned.imag
            flat["k_cache"][slots[b][lengths[b] - n[b] :]] = k[here]
            flat["v_cache"][slots[b][lengths[b] - n[b] :]] = s["v"][here].double()
        return flat["k_cache"].reshape(s["k_cache"].shape), flat["v_cache"].reshape(s["v_cache"].shape), q
    G = case["heads"] // case["kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, end in enumerate(ends):
        for at in range(0, n[b], 2048):
            rows = torch.arange(at, min(at + 2048, n[b]), device="cuda")
            position = int(lengths[b] - n[b]) + rows
            low = max(int(position[0]) - case["window"] + 1, 0) if case["window"] else 0
            here = slots[b][low : int(position[-1]) + 1]
            ahead = torch.arange(low, low + here.numel(), device="cuda") - position[:, None]
            hidden = (ahead > 0) | (ahead <= -case["window"]) if case["window"] else ahead > 0
            for h in range(case["heads"]):
                x = s["q"][end - n[b] + rows, h].double() @ flat["k_cache"][here, h // G].T / math.sqrt(case["D"])
                out[end - n[b] + rows, h] = x.masked_fill(hidden, -math.inf).softmax(1) @ flat["v_cache"][here, h // G]
    return out
