"""Host-side checks of the paged-cache entry points: bad arguments are refused
before anything is launched, and empty problems are no-ops.  No compute call is
made here (the addresses are never used)."""
import ctypes

import numpy as np
import pytest

import paged_ref as R
import unstructured_sparse_matmul_gb300 as usm

A16, ODD8, ODD2 = 0x10000, 0x10008, 0x10002
INVALID, ALIGN, UNSUPPORTED, WORKSPACE = -1, -2, -3, -6
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    return usm.load()


def cache(**kw):
    """Three pages of 4 slots for 2 heads of 8 bf16 elements, two sequences."""
    f = dict(k=A16, v=A16, k_page_stride=64, k_slot_stride=16, k_head_stride=8, v_page_stride=64, v_slot_stride=16,
             v_head_stride=8, page_table=A16, lengths=A16, q_offsets=A16, dtype=1, num_pages=3, page_size=4, kv_heads=2,
             head_dim=8, num_seqs=2, table_stride=5, table_pages=5)
    f.update(kw)
    return usm.PagedCache(**f)


def tokens(data=A16, token_stride=32, head_stride=8):
    return usm.Tokens(data, token_stride, head_stride)


def ref(x):
    return None if x is None else ctypes.byref(x)


BAD_CACHE = [(dict(num_seqs=-1), INVALID), (dict(kv_heads=0), INVALID), (dict(head_dim=0), INVALID),
             (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(table_pages=-1), INVALID),
             (dict(dtype=2), INVALID), (dict(lengths=None), INVALID), (dict(page_table=None), INVALID),
             (dict(table_stride=4), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
             (dict(k_page_stride=0), INVALID), (dict(k_slot_stride=0), INVALID), (dict(k_head_stride=-8), INVALID),
             (dict(v_page_stride=7), INVALID), (dict(v_slot_stride=0), INVALID), (dict(v_head_stride=0), INVALID),
             (dict(q_offsets=None, num_seqs=4), INVALID),  # 6 tokens are no equal shares of 4
             (dict(head_dim=264), UNSUPPORTED), (dict(head_dim=12), ALIGN), (dict(k=ODD8), ALIGN), (dict(v=ODD8), ALIGN),
             (dict(k_page_stride=65), ALIGN), (dict(k_slot_stride=20), ALIGN), (dict(v_head_stride=9), ALIGN),
             (dict(lengths=ODD2), ALIGN), (dict(page_table=ODD2), ALIGN), (dict(q_offsets=ODD2), ALIGN),
             (dict(dtype=0, head_dim=6, k_head_stride=8), ALIGN)]
BAD_TOKENS = [(dict(data=None), INVALID), (dict(token_stride=-32), INVALID), (dict(head_stride=-8), INVALID),
              (dict(data=ODD8), ALIGN), (dict(token_stride=36), ALIGN), (dict(head_stride=9), ALIGN)]
OVERLAPPING = [(dict(token_stride=0), INVALID), (dict(head_stride=0), INVALID), (dict(token_stride=4), INVALID)]


def append(lib, c=None, n=6, k=None, v=None, q="in", q_out="out", q_heads=4, rope=A16, positions=9, rot=8, inter=0):
    c = cache() if c is None else c
    k, v = tokens() if k is None else k, tokens() if v is None else v
    q = tokens() if q == "in" else q
    q_out = tokens() if q_out == "out" else q_out
    return lib.paged_append(ref(c), n, ref(k), ref(v), ref(q), ref(q_out), q_heads, rope, positions, rot, inter, None)


def attention(lib, c=None, n=6, q=None, heads=4, scale=1.0, causal=1, window=0, out=None, ws=A16, wsb=1 << 40):
    c = cache() if c is None else c
    q, out = tokens() if q is None else q, tokens() if out is None else out
    return lib.paged_attention(ref(c), n, ref(q), heads, scale, causal, window, ref(out), ws, wsb, None)


def test_append_refuses(lib):
    for kw, code in BAD_CACHE:
        assert append(lib, cache(**kw)) == code, kw
    for kw, code in BAD_TOKENS:
        for name in ("k", "v", "q", "q_out"):
            assert append(lib, **{name: tokens(**kw)}) == code, (name, kw)
    for kw, code in OVERLAPPING:
        assert append(lib, q_out=tokens(**kw)) == code, kw
    for kw in (dict(n=-1), dict(q=None), dict(q_out=None), dict(q_heads=-1), dict(q_heads=0), dict(q=None, q_out=None),
               dict(rot=-2), dict(rot=7), dict(rot=10), dict(inter=2), dict(rope=None), dict(positions=0)):
        assert append(lib, **kw) == INVALID, kw
    assert append(lib, rope=ODD8) == ALIGN
    assert append(lib, n=1 << 30) == UNSUPPORTED
    assert lib.paged_append(None, 1, None, None, None, None, 0, None, 0, 0, 0, None) == INVALID


def test_attention_refuses(lib):
    for kw, code in BAD_CACHE:
        assert attention(lib, cache(**kw)) == code, kw
    for kw, code in BAD_TOKENS:
        assert attention(lib, q=tokens(**kw)) == code, kw
        assert attention(lib, out=tokens(**kw)) == code, kw
    for kw, code in OVERLAPPING:
        assert attention(lib, out=tokens(**kw)) == code, kw
    for kw in (dict(n=-1), dict(heads=0), dict(heads=3), dict(scale=-1.0), dict(scale=INF), dict(scale=NAN),
               dict(causal=2), dict(window=-1)):
        assert attention(lib, **kw) == INVALID, kw
    assert attention(lib, n=1 << 30, heads=2) == UNSUPPORTED
    assert attention(lib, ws=None) == WORKSPACE
    need = lib.paged_attention_workspace_bytes(6, 2, 4, 2, 8, 1)
    assert need > 0 and attention(lib, wsb=need - 1) == WORKSPACE
    assert attention(lib, ws=ODD8) == ALIGN


def test_empty_calls_touch_nothing(lib):
    nothing = dict(k=None, v=None, page_table=None, lengths=None, q_offsets=None)
    assert append(lib, cache(**nothing), n=0, k=tokens(None), v=tokens(None)) == 0
    assert append(lib, cache(num_seqs=0, **nothing)) == 0
    assert attention(lib, cache(**nothing), n=0, ws=None, wsb=0) == 0
    assert attention(lib, cache(num_seqs=0, **nothing), ws=None, wsb=0) == 0


def test_workspace_bytes(lib):
    f = lib.paged_attention_workspace_bytes
    for bad in ((0, 4, 4, 2, 8, 1), (4, 0, 4, 2, 8, 1), (4, 4, 0, 2, 8, 1), (4, 4, 4, 0, 8, 1), (4, 4, 3, 2, 8, 1),
                (4, 4, 4, 2, 0, 1), (4, 4, 4, 2, 257, 1), (4, 4, 4, 2, 8, 2), (1 << 30, 4, 2, 1, 8, 1)):
        assert f(*bad) == 0, bad
    assert 0 < f(1, 1, 4, 4, 64, 1) < f(64, 1, 4, 4, 64, 1) <= f(4096, 1, 32, 4, 64, 1)
    assert 0 < f(1, 1, 4, 4, 64, 0) < f(64, 1, 4, 4, 64, 0)


def test_rope_table_refuses(lib):
    f = lib.rope_table_build
    for bad in ((-1, 8, 10000.0), (4, 0, 10000.0), (4, 7, 10000.0), (4, -2, 10000.0), (4, 8, 0.0), (4, 8, -1.0),
                (4, 8, INF), (4, 8, NAN)):
        assert f(*bad, A16, None) == INVALID, bad
    assert f(4, 8, 10000.0, None, None) == INVALID
    assert f(1 << 28, 8, 10000.0, A16, None) == UNSUPPORTED
    assert f(4, 8, 10000.0, ODD2, None) == ALIGN
    assert f(0, 8, 10000.0, None, None) == 0


def test_structs_match_their_packed_form():
    c = cache()
    values = [getattr(c, name) or 0 for name, _ in usm.PagedCache._fields_]
    assert bytes(c) == usm._pack_paged(*values)
    t = tokens()
    assert bytes(t) == usm._pack_tokens(t.data, t.token_stride, t.head_stride)


def test_definition_of_attention():
    """The reference against a direct softmax on a cache of one page."""
    rng = np.random.default_rng(0)
    q, K, V = (rng.standard_normal(s) for s in ((3, 2, 4), (1, 5, 1, 4), (1, 5, 1, 4)))
    out, _ = R.attention(q, K, V, np.zeros((1, 1), int), [5], [3], [0], 0.5)
    for i in range(3):
        x = np.exp(0.5 * K[0, : 3 + i, 0] @ q[i].T)
        assert np.allclose(out[i], (x / x.sum(0)).T @ V[0, : 3 + i, 0])
    seen, _ = R.attention(q, K, V, np.zeros((1, 1), int), [5], [3], [0], 0.5, window=1)
    assert np.allclose(seen, V[0, 2:, 0][:, None])


def test_definition_of_rotation():
    """Rotating query and key by their positions leaves a product that depends on
    their distance only."""
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 8))
    table = R.rope_table(40, 6, 100.0)
    for inter in (False, True):
        dot = [float(R.rotate(q, table[p + 7], 6, inter)[0] @ R.rotate(k, table[p], 6, inter)[0]) for p in (0, 5, 32)]
        assert np.allclose(dot, dot[0])
