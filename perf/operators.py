"""Cases for the operators of sparse attention beside the SDDMM and SpMM: the
relative position bias on CSR scores and its gradient, the differential
softmax map and its gradient, the row softmax's gradient, and attention of few
query rows over their listed keys.

`run` computes each in a plain form with elementary torch operations, or, with
`own` set, with the library's calls.  `exact` computes the same in 64 bits with
numpy from the definitions.

Layout of every case: `blocks` query blocks (batch x heads, heads fastest) of
`rows` query rows each; `group` consecutive blocks share one block of `cols`
keys.  The mask's row densities are lognormal around `density` with
coefficient of variation `cov`; `empty` of the rows have no entry, `whole` of
them every entry.
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _case(op, name=None, **kw):
    c = dict(op=op, heads=8, batch=1, rows=4096, cols=4096, group=1, density=0.1, cov=0.5, empty=0.0, whole=0.0,
             dtype="f32", buckets=32, reach=128, causal=False)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # The library's attention configuration: a prompt of 4096 tokens, 8 heads, a tenth of the keys kept.
        _case("bias", "bias prompt 8x4096"),
        # One new token for each of 8 sequences over a cache of 4096 tokens.
        _case("bias", "bias token 64x1", batch=8, rows=1, causal=True),
        # Training on the same prompt; the scores' gradient comes in bf16, as the products take it.
        _case("bias_grad", "bias grad prompt 8x4096", dtype="bf16"),
        # A short batch of odd sizes with padded (empty) rows.
        _case("bias_grad", "bias grad odd 6x777", heads=3, batch=2, rows=777, cols=1531, density=0.3, cov=0.3, empty=0.05),
        _case("diff", "diff map prompt 8x4096", dtype="bf16"),
        # Few long rows: tokens that look at half of a cache of 131072.
        _case("diff", "diff map long 32x1", heads=32, rows=1, cols=131072, density=0.5, cov=0.1),
        _case("diff_grad", "diff grad prompt 8x4096", dtype="bf16"),
        _case("diff_grad", "diff grad odd 6x777", heads=3, batch=2, rows=777, cols=1531, density=0.3, cov=0.3, empty=0.05),
        _case("softmax_grad", "softmax grad prompt 8x4096", dtype="bf16"),
        # A sparse mask in which a hundredth of the rows (global tokens) sees every key.
        _case("softmax_grad", "softmax grad global 4x2048", heads=4, rows=2048, cols=16384, density=0.01, whole=0.01),
        # One new token of one sequence: the latency of the smallest call.
        _case("attention", "attention token 8x1", rows=1, dtype="bf16", D=64, N=64, maps=1, bias=True, causal=True),
        # A serving batch of 32 sequences with 8 heads over a cache of 16384, two maps, values twice as wide.
        _case("attention", "attention batch 256x1", batch=32, rows=1, cols=16384, density=0.25, cov=0.2, dtype="bf16",
              D=64, N=128, maps=2, bias=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["bias", "bias_grad", "diff", "diff_grad", "softmax_grad", "attention"])
    kw = dict(dtype=rng.choice(["f32", "bf16"]), density=math.exp(rng.uniform(math.log(0.01), math.log(0.5))),
              cov=rng.choice([0.1, 0.3, 0.5]), empty=rng.choice([0.0, 0.05]), whole=rng.choice([0.0, 0.01]))
    if op == "bias":
        kw["dtype"] = "f32"
    heads, batch = rng.randint(1, 16), rng.randint(1, 8)
    if op == "attention":
        rows = rng.choice([1, 1, rng.randint(2, 5)])
        group = rng.choice([g for g in (1, 2, 4) if heads % g == 0])
        D = rng.choice([32, 40, 64, 96, 128])
        kw.update(group=group, D=D, N=rng.choice([D, 2 * D]), maps=rng.randint(1, 2), bias=rng.random() < 0.5)
        kw["whole"] = 0.0  # the plain form pads every row to the longest
        cols, most = _log_int(rng, 64, 32768), 600_000
    else:
        rows = rng.choice([1, _log_int(rng, 2, 4096), _log_int(rng, 2, 4096)])
        cols, most = _log_int(rng, 64, 131072 if rows == 1 else 16384), 9_000_000
    batch = max(1, min(batch, 32_000_000 // (heads * rows * cols)))
    rows = max(1, min(rows, 32_000_000 // (heads * batch * cols)))
    total = heads * batch * rows
    kw["density"] = min(max(min(kw["density"], most / (total * cols)), 64 / (total * cols)), 1.0)
    if total < 16:
        kw["empty"] = 0.0
    if "bias" in op or kw.get("bias"):
        kw.update(buckets=rng.choice([16, 32, 48, 64]), reach=rng.choice([64, 128, 200, 512]), causal=rng.random() < 0.5)
    return _case(op, heads=heads, batch=batch, rows=rows, cols=cols, **kw)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _bucket_map(buckets, reach, causal):
    """Bucket of each relative position -reach..reach (key minus query): small
    distances one each, larger ones on a logarithmic scale up to `reach`."""
    rel = np.arange(-reach, reach + 1)
    base = np.zeros_like(rel)
    if causal:
        n, b = np.maximum(-rel, 0), buckets
    else:
        n, b = np.abs(rel), buckets // 2
        base = b * (rel > 0)
    small = b // 2
    far = small + np.floor(np.log(np.maximum(n, 1) / small) / np.log(reach / small) * (b - small) + 1e-9)
    return (base + np.where(n < small, n, np.minimum(far, b - 1))).astype(np.int32)


def _torch_dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case):
    """Entries of each row: a case's own, whatever the seed of its inputs."""
    rng = np.random.default_rng([case["heads"], case["batch"], case["rows"], case["cols"]])
    R = case["batch"] * case["heads"] * case["rows"]
    sigma = math.sqrt(math.log(1 + case["cov"] ** 2))
    n = np.rint(case["cols"] * case["density"] * np.exp(sigma * rng.standard_normal(R) - sigma * sigma / 2))
    u = rng.random(R)
    n[u < case["whole"]] = case["cols"]
    n[u > 1 - case["empty"]] = 0
    n = np.minimum(n, case["cols"]).astype(np.int64)
    n[0] = max(n[0], 1)
    return n


def _mask(case, gen):
    """The mask in CSR: each row's columns drawn without replacement."""
    n = _lengths(case)
    lengths = torch.from_numpy(n).cuda()
    ro = torch.zeros(n.size + 1, dtype=torch.int32, device="cuda")
    ro[1:] = lengths.cumsum(0)
    longest, cols, parts = int(n.max()), case["cols"], []
    for at in range(0, n.size, max(1, 2**24 // cols)):
        part = lengths[at : at + max(1, 2**24 // cols)]
        order = torch.rand(part.numel(), cols, generator=gen, device="cuda").argsort(1)[:, :longest]
        kept = torch.zeros(part.numel(), cols, dtype=torch.bool, device="cuda")
        kept.scatter_(1, order, torch.arange(longest, device="cuda") < part[:, None])
        where = kept.nonzero()
        kv = torch.div(where[:, 0] + at, case["rows"] * case["group"], rounding_mode="floor")
        parts.append((where[:, 1] + kv * cols).to(torch.int32))
    return ro, torch.cat(parts), longest


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dt = case["op"], _torch_dtype(case)
    ro, ci, longest = _mask(case, gen)
    nnz, R, blocks = ci.numel(), ro.numel() - 1, case["batch"] * case["heads"]

    def randn(*shape, std=1.0, dtype=torch.float32):
        return (std * torch.randn(*shape, generator=gen, device="cuda")).to(dtype)

    s = dict(case=case, ro=ro, ci=ci, longest=longest)
    if op in ("bias", "bias_grad") or case.get("bias"):
        s["map"] = torch.from_numpy(_bucket_map(case["buckets"], case["reach"], case["causal"])).cuda()
        s["table"] = randn(case["heads"], case["buckets"])
        # A token's position is the last of its cache, whose filled length differs by sequence.
        fill = torch.randint(max(1, case["cols"] // 2), case["cols"] + 1, (case["batch"],), generator=gen, device="cuda")
        s["q_offset"] = (fill - 1).to(torch.int32).repeat_interleave(case["heads"]) if case["rows"] == 1 else None
    if op in ("bias", "diff", "diff_grad", "softmax_grad"):
        s["scores"] = randn(nnz, std=2.0)
    if op in ("diff", "diff_grad"):
        s["scores2"] = randn(nnz, std=2.0)
    if op in ("diff", "diff_grad") or case.get("maps") == 2:
        s["lam"] = torch.rand(case["heads"], generator=gen, device="cuda") * 0.6 + 0.2
    if op in ("bias_grad", "diff_grad", "softmax_grad"):
        s["grad"] = randn(nnz, dtype=dt if op == "bias_grad" else torch.float32)
    if op == "attention":
        D, N, kv = case["D"], case["N"], blocks // case["group"] * case["cols"]
        for n in ("", "2")[: case["maps"]]:
            s["Q" + n] = randn(R, D, dtype=dt)
            s["K" + n] = randn(kv, D, dtype=dt)
        s["V"] = randn(kv, N, dtype=dt)
    return s


# ---------------------------------------------------------------------------
# The operators' plain forms
# ---------------------------------------------------------------------------
def _rows(s):
    ro = s["ro"].long()
    return torch.repeat_interleave(torch.arange(ro.numel() - 1, device="cuda"), ro[1:] - ro[:-1],
                                   output_size=s["ci"].numel())


def _bias_index(s, r, col):
    """Entry of the flattened table for entries in rows r with columns col."""
    c = s["case"]
    block = torch.div(r, c["rows"], rounding_mode="floor")
    query = r - block * c["rows"]
    if s["q_offset"] is not None:
        query = query + s["q_offset"].long()[block]
    rel = (col % c["cols"] - query).clamp(-c["reach"], c["reach"])
    return (block % c["heads"]) * c["buckets"] + s["map"].long()[rel + c["reach"]]


def _padded(s):
    """Entry numbers of each row, padded to the longest row, and which are real."""
    ro = s["ro"].long()
    at = ro[:-1, None] + torch.arange(s["longest"], device="cuda")
    return at.clamp(max=s["ci"].numel() - 1), at < ro[1:, None]


def _softmax(s, scores, at, real, r):
    """Softmax over each row's entries: row maxima and sums from the padded
    rows, the probabilities in CSR order."""
    x = scores[at].masked_fill(~real, -math.inf)
    top = x.amax(1)
    z = torch.exp(x - top[:, None]).masked_fill(~real, 0.0).sum(1)
    return torch.exp(scores - top[r]) / z[r]


def _row_sum(x, at, real):
    return x[at].masked_fill(~real, 0.0).sum(1)


def _head(s, r):
    return torch.div(r, s["case"]["rows"], rounding_mode="floor") % s["case"]["heads"]


def _plain_attention(s):
    c = s["case"]
    at, real = _padded(s)
    col = s["ci"].long()[at]
    r = torch.arange(at.shape[0], device="cuda")
    scale = c["D"] ** -0.5
    bias = s["table"].reshape(-1)[_bias_index(s, r[:, None], col)] if c["bias"] else None

    def probs(q, k):
        x = (k.float()[col] * q.float()[:, None, :]).sum(2) * scale
        x = (x if bias is None else x + bias).masked_fill(~real, -math.inf)
        top = x.amax(1, keepdim=True).clamp(min=-3e38)
        e = torch.exp(x - top)
        return e / e.sum(1, keepdim=True).clamp(min=1e-30)

    p = probs(s["Q"], s["K"])
    if c["maps"] == 2:
        p = p - s["lam"][_head(s, r)][:, None] * probs(s["Q2"], s["K2"])
    return (p[:, :, None] * s["V"].float()[col]).sum(1)


def run(s):
    if own:
        return _run_own(s)
    op, out = s["case"]["op"], _torch_dtype(s["case"])
    if op == "attention":
        return _plain_attention(s)
    r = _rows(s)
    if op == "bias":
        return s["scores"] + s["table"].reshape(-1)[_bias_index(s, r, s["ci"].long())]
    if op == "bias_grad":
        # Sums of many terms: 64 bits, spread over 256 copies of the table.
        size = s["table"].numel()
        index = _bias_index(s, r, s["ci"].long()) + torch.arange(r.numel(), device="cuda") % 256 * size
        total = torch.zeros(256 * size, dtype=torch.float64, device="cuda").index_add_(0, index, s["grad"].double())
        return total.reshape(256, *s["table"].shape).sum(0).float()
    at, real = _padded(s)
    p1 = _softmax(s, s["scores"], at, real, r)
    if op == "softmax_grad":
        return (p1 * (s["grad"] - _row_sum(p1 * s["grad"], at, real)[r])).to(out)
    p2 = _softmax(s, s["scores2"], at, real, r)
    lam = s["lam"][_head(s, r)]
    if op == "diff":
        return (p1 - lam * p2).to(out)
    c1, c2 = (_row_sum(p * s["grad"], at, real) for p in (p1, p2))
    c = s["case"]
    dlam = -c2.double().reshape(c["batch"], c["heads"], c["rows"]).sum((0, 2)).float()
    return (p1 * (s["grad"] - c1[r])).to(out), (-lam * p2 * (s["grad"] - c2[r])).to(out), dlam


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    import unstructured_sparse_matmul_gb300 as usm
    c, out = s["case"], _torch_dtype(s["case"])
    op, rows = c["op"], c["rows"]
    if op == "bias":
        return usm.rel_bias(s["ro"], s["ci"], s["scores"], s["table"], s["map"], seg_rows=rows, seg_cols=c["cols"],
                            q_offset=s["q_offset"])
    if op == "bias_grad":
        return usm.rel_bias_grad(s["ro"], s["ci"], s["grad"], c["heads"], c["buckets"], s["map"], seg_rows=rows,
                                 seg_cols=c["cols"], q_offset=s["q_offset"])
    if op == "diff":
        return usm.diff_softmax(s["ro"], s["scores"], s["scores2"], s["lam"], seg_rows=rows, out_dtype=out)
    if op == "diff_grad":
        return usm.diff_softmax_grad(s["ro"], s["scores"], s["scores2"], s["lam"], s["grad"], seg_rows=rows,
                                     out_dtype=out)
    if op == "softmax_grad":
        return usm.row_softmax_grad(s["ro"], s["scores"], s["grad"], out_dtype=out)
    extra = dict(table=s["table"], bucket_map=s["map"], seg_cols=c["cols"], q_offset=s["q_offset"]) if c["bias"] else {}
    if c["maps"] == 2:
        extra.update(Q2=s["Q2"], K2=s["K2"], lam=s["lam"])
    return usm.attention(s["ro"], s["ci"], s["Q"], s["K"], s["V"], scale=c["D"] ** -0.5, seg_rows=rows, **extra)


# ---------------------------------------------------------------------------
# Bytes and operations of one pass
# ---------------------------------------------------------------------------
def work(case):
    n = _lengths(case)
    R, nnz = n.size, int(n.sum())
    dens = nnz / (R * case["cols"])
    es = 2 if case["dtype"] == "bf16" else 4
    offsets, table = 4 * R, 4 * case["heads"] * case["buckets"]
    op = case["op"]
    if op == "bias":
        return {"bytes": nnz * 12 + offsets + table, "flops": nnz}
    if op == "bias_grad":
        return {"bytes": nnz * (4 + es) + offsets + table, "flops": nnz}
    if op == "diff":
        return {"bytes": nnz * (8 + es) + offsets, "flops": 10 * nnz}
    if op == "diff_grad":
        return {"bytes": nnz * (12 + 2 * es) + offsets, "flops": 20 * nnz}
    if op == "softmax_grad":
        return {"bytes": nnz * (8 + es) + offsets, "flops": 10 * nnz}
    D, N, maps = case["D"], case["N"], case["maps"]
    kv = case["batch"] * case["heads"] // case["group"] * case["cols"]
    touched = kv * (1 - (1 - dens) ** (case["rows"] * case["group"]))  # key rows that some query row lists
    return {"bytes": nnz * 4 + touched * (maps * D + N) * es + R * (maps * D * es + 4 * N) + offsets,
            "flops": nnz * (2 * maps * D + 2 * N)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _host(t):
    return None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy().astype(np.int64)


def exact(case, seed):
    s = prepare(case, seed)
    h = {k: _host(v) for k, v in s.items() if isinstance(v, torch.Tensor)}
    ro, ci = h["ro"], h["ci"]
    lengths = np.diff(ro)
    row = np.repeat(np.arange(lengths.size), lengths)
    block = row // case["rows"]
    head = block % case["heads"]
    some = np.flatnonzero(lengths)
    op = case["op"]

    def over_rows(f, x):
        """f (a ufunc) reduced over each row's entries, repeated for each of them."""
        return np.repeat(f.reduceat(x, ro[some]), lengths[some]) if x.size else x

    def softmax(x):
        e = np.exp(x - over_rows(np.maximum, x))
        return e / over_rows(np.add, e)

    bias = None
    if "map" in h:
        # Each key's position in its own block of keys, less the query's.
        first = np.repeat(ci[np.minimum(ro[:-1], max(ci.size - 1, 0))] // case["cols"] * case["cols"], lengths)
        query = row % case["rows"] + (h["q_offset"][block] if s["q_offset"] is not None else 0)
        far = np.minimum(np.maximum(ci - first - query, -case["reach"]), case["reach"])
        bucket = h["map"][far + case["reach"]]
        if op == "bias_grad":
            flat = np.bincount(head * case["buckets"] + bucket, h["grad"], case["heads"] * case["buckets"])
            return torch.from_numpy(flat.reshape(case["heads"], case["buckets"]))
        bias = h["table"][head, bucket]
        if op == "bias":
            return torch.from_numpy(h["scores"] + bias)
    if op == "attention":
        out = np.zeros((lengths.size, case["N"]))
        for i in some:
            here = slice(ro[i], ro[i + 1])
            keys = ci[here]
            p = 0.0
            for n, weight in (("", 1.0), ("2", -h["lam"][head[ro[i]]] if case["maps"] == 2 else 0.0))[: case["maps"]]:
                x = h["K" + n][keys] @ h["Q" + n][i] * case["D"] ** -0.5 + (0.0 if bias is None else bias[here])
                e = np.exp(x - x.max())
                p = p + weight * e / e.sum()
            out[i] = p @ h["V"][keys]
        return torch.from_numpy(out)
    p1 = softmax(h["scores"])
    if op == "softmax_grad":
        return torch.from_numpy(p1 * (h["grad"] - over_rows(np.add, p1 * h["grad"])))
    p2 = softmax(h["scores2"])
    if op == "diff":
        return torch.from_numpy(p1 - h["lam"][head] * p2)
    g1, g2 = (p * (h["grad"] - over_rows(np.add, p * h["grad"])) for p in (p1, p2))
    dlam = -np.bincount(head, p2 * h["grad"], case["heads"])
    return torch.from_numpy(g1), torch.from_numpy(-h["lam"][head] * g2), torch.from_numpy(dlam)
