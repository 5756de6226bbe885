"""Host-side checks of the sparse-attention entry points: bad arguments are
refused before anything is launched, and empty problems are no-ops.  No compute
call is made here (the addresses are never used)."""
import ctypes

import numpy as np
import pytest

import attention_ref as R
import unstructured_sparse_matmul_gb300 as usm

A16, ODD4, ODD2 = 0x10000, 0x10004, 0x10002
INVALID, ALIGN, UNSUPPORTED, WORKSPACE = -1, -2, -3, -6


@pytest.fixture(scope="module")
def lib():
    return usm.load()


def bias(table=A16, table_dtype=0, num_heads=2, num_buckets=8, bucket_map=A16, max_distance=16, seg_cols=4,
         q_offset=None):
    return usm.RelBias(table, table_dtype, num_heads, num_buckets, bucket_map, max_distance, seg_cols, q_offset)


BAD_BIAS = [(dict(num_heads=0), INVALID), (dict(num_buckets=0), INVALID), (dict(max_distance=0), INVALID),
            (dict(bucket_map=None), INVALID), (dict(num_buckets=513), UNSUPPORTED),
            (dict(max_distance=8193), UNSUPPORTED), (dict(bucket_map=ODD2), ALIGN), (dict(q_offset=ODD2), ALIGN)]
BAD_TABLE = [(dict(table=None), INVALID), (dict(table_dtype=5), INVALID), (dict(table=ODD2), ALIGN)]


def rel_bias(lib, b=None, M=4, K=4, nnz=4, ro=A16, ci=A16, s=A16, seg=2, out=A16, **kw):
    b = bias(**kw) if b is None else b
    return lib.csr_rel_bias(M, K, nnz, ro, ci, s, seg, ctypes.addressof(b) if b else None, out, None)


def rel_bias_grad(lib, M=4, K=4, nnz=4, ro=A16, ci=A16, ds=A16, dt=0, seg=2, out=A16, ws=A16, wsb=1 << 20, **kw):
    b = bias(**kw)
    return lib.csr_rel_bias_grad(M, K, nnz, ro, ci, ds, dt, seg, ctypes.addressof(b), out, ws, wsb, None)


def attention(lib, b=None, **kw):
    v = dict(M=4, K=4, D=8, N=8, nnz=4, ro=A16, ci=A16, Q=A16, ldq=8, Km=A16, ldk=8, Q2=None, ldq2=0, K2=None, ldk2=0,
             V=A16, ldv=8, scale=1.0, lam=None, heads=2, seg=2, bias=ctypes.addressof(b) if b else None, C=A16, ldc=8,
             dtype=0, ws=None, wsb=0)
    v.update(kw)
    return lib.csr_attention(*v.values(), None)


@pytest.mark.parametrize("kw,code", BAD_BIAS + BAD_TABLE)
def test_bias_struct_is_checked(lib, kw, code):
    assert rel_bias(lib, **kw) == code
    assert attention(lib, bias(**kw)) == code
    if "table" not in kw and "table_dtype" not in kw:
        assert rel_bias_grad(lib, **kw) == code


def test_rel_bias_refuses(lib):
    for kw in (dict(M=-1), dict(K=-1), dict(nnz=-1), dict(K=0), dict(ro=None), dict(ci=None), dict(s=None),
               dict(out=None)):
        assert rel_bias(lib, **kw) == INVALID, kw
    assert lib.csr_rel_bias(4, 4, 4, A16, A16, A16, 2, None, A16, None) == INVALID  # no bias
    assert rel_bias(lib, s=ODD2) == ALIGN
    assert rel_bias(lib, out=ODD2) == ALIGN
    assert rel_bias(lib, M=0, ro=None) == 0
    assert rel_bias(lib, nnz=0, ci=None, s=None, out=None) == 0


def test_rel_bias_grad_refuses(lib):
    for kw in (dict(M=-1), dict(K=-1), dict(nnz=-1), dict(dt=2), dict(K=0), dict(ro=None), dict(ci=None),
               dict(ds=None), dict(out=None)):
        assert rel_bias_grad(lib, **kw) == INVALID, kw
    assert rel_bias_grad(lib, out=ODD2) == ALIGN
    assert rel_bias_grad(lib, ds=ODD2) == ALIGN
    assert rel_bias_grad(lib, ds=0x10001, dt=1) == ALIGN
    need = lib.csr_rel_bias_grad_workspace_bytes(4, 4, 2, 2, 8)
    assert need > 0
    assert rel_bias_grad(lib, ws=None) == WORKSPACE
    assert rel_bias_grad(lib, wsb=need - 1) == WORKSPACE
    assert rel_bias_grad(lib, ws=ODD4) == ALIGN
    assert lib.csr_rel_bias_grad_workspace_bytes(0, 4, 2, 2, 8) == 0
    assert lib.csr_rel_bias_grad_workspace_bytes(4, 0, 2, 2, 8) == 0


def test_bucket_build_refuses(lib):
    f = lib.rel_bucket_build
    for args in ((1, 16, 1, A16), (3, 16, 0, A16), (2, 16, 0, A16), (32, 16, 1, A16), (32, 8, 0, A16), (32, 128, 2, A16),
                 (32, 128, 0, None), (32, 0, 0, A16)):
        assert f(*args, None) == INVALID, args
    assert f(514, 8000, 0, A16, None) == UNSUPPORTED
    assert f(32, 8193, 0, A16, None) == UNSUPPORTED
    assert f(32, 128, 0, ODD2, None) == ALIGN


def test_maps_refuse(lib):
    names = ["M", "nnz", "ro", "s1", "s2", "lam", "heads", "seg", "out", "dt"]
    ok = dict(zip(names, [4, 4, A16, A16, A16, A16, 2, 2, A16, 0]))
    f = lambda **kw: lib.csr_diff_softmax(*{**ok, **kw}.values(), None)
    for kw in (dict(M=-1), dict(nnz=-1), dict(heads=0), dict(dt=2), dict(ro=None), dict(s1=None), dict(s2=None),
               dict(lam=None), dict(out=None)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(s1=ODD2), dict(s2=ODD2), dict(lam=ODD2), dict(out=ODD2), dict(out=0x10001, dt=1)):
        assert f(**kw) == ALIGN, kw
    assert f(M=0, ro=None) == 0
    assert f(nnz=0, s1=None, out=None) == 0

    names = ["M", "nnz", "ro", "s1", "s2", "lam", "heads", "seg", "dout", "din", "g1", "g2", "dt", "dlam", "ws", "wsb"]
    okg = dict(zip(names, [4, 4, A16, A16, A16, A16, 2, 2, A16, 0, A16, A16, 0, A16, A16, 1 << 20]))
    g = lambda **kw: lib.csr_diff_softmax_grad(*{**okg, **kw}.values(), None)
    for kw in (dict(M=-1), dict(nnz=-1), dict(heads=0), dict(din=2), dict(dt=2), dict(ro=None), dict(s1=None),
               dict(s2=None), dict(lam=None), dict(dout=None), dict(g1=None), dict(g2=None)):
        assert g(**kw) == INVALID, kw
    for kw in (dict(s1=ODD2), dict(s2=ODD2), dict(lam=ODD2), dict(dout=ODD2), dict(g1=ODD2), dict(g2=ODD2),
               dict(dlam=ODD2), dict(ws=ODD4)):
        assert g(**kw) == ALIGN, kw
    assert lib.csr_diff_softmax_grad_workspace_bytes(4) >= 16
    assert g(ws=None) == WORKSPACE
    assert g(wsb=3) == WORKSPACE
    assert g(M=0, ro=None, dlam=None) == 0
    assert g(nnz=0, s1=None, dlam=None) == 0

    names = ["M", "nnz", "ro", "s", "dout", "din", "g", "dt"]
    oks = dict(zip(names, [4, 4, A16, A16, A16, 0, A16, 0]))
    h = lambda **kw: lib.csr_row_softmax_grad(*{**oks, **kw}.values(), None)
    for kw in (dict(M=-1), dict(nnz=-1), dict(din=3), dict(dt=3), dict(ro=None), dict(s=None), dict(dout=None),
               dict(g=None)):
        assert h(**kw) == INVALID, kw
    for kw in (dict(s=ODD2), dict(dout=ODD2), dict(g=ODD2)):
        assert h(**kw) == ALIGN, kw
    assert h(M=0, ro=None) == 0


def test_attention_refuses(lib):
    two = dict(lam=A16, Q2=A16, ldq2=8, K2=A16, ldk2=8)
    for kw in (dict(M=-1), dict(K=-1), dict(D=-1), dict(N=-1), dict(nnz=-1), dict(heads=0), dict(dtype=2),
               dict(ro=None), dict(ci=None), dict(Q=None), dict(Km=None), dict(V=None), dict(C=None), dict(ldc=4),
               dict(ldq=4), dict(ldk=4), dict(ldv=4), dict(K=0), dict(lam=A16), dict(Q2=A16), dict(K2=A16),
               dict(two, ldq2=4), dict(two, ldk2=4), dict(two, Q2=None)):
        assert attention(lib, **kw) == INVALID, kw
    for kw in (dict(Q=ODD4), dict(Km=ODD4), dict(V=ODD4), dict(C=ODD4), dict(ldc=10), dict(ldq=9), dict(ldk=9),
               dict(ldv=9), dict(two, Q2=ODD4), dict(two, K2=ODD4), dict(two, ldq2=9), dict(two, ldk2=9),
               dict(two, lam=ODD2), dict(dtype=1, ldq=12)):
        assert attention(lib, **kw) == ALIGN, kw
    assert attention(lib, D=257, ldq=260, ldk=260) == UNSUPPORTED
    assert attention(lib, N=260, ldv=260, ldc=260) == UNSUPPORTED
    assert attention(lib, D=513, ldq=520, ldk=520, dtype=1) == UNSUPPORTED
    assert attention(lib, bias(num_heads=3)) == INVALID  # heads disagree
    big = dict(M=64, nnz=1 << 20, K=1 << 20)
    need = lib.csr_attention_workspace_bytes(64, 1 << 20, 8, 8, 1 << 20, 0, 0)
    assert need > 0 and lib.csr_attention_workspace_bytes(4, 4, 8, 8, 4, 0, 0) == 0
    assert attention(lib, **big) == WORKSPACE
    assert attention(lib, **big, ws=A16, wsb=need - 1) == WORKSPACE
    assert attention(lib, **big, ws=ODD4, wsb=need) == ALIGN
    assert attention(lib, M=0, ro=None, C=None) == 0
    assert attention(lib, N=0, C=None) == 0


@pytest.mark.parametrize("heads,buckets", [(2**31 - 1, 1), (2**31 - 456, 2), (10**9, 512), (457, 32), (1, 1)])
def test_workspace_of_many_heads(lib, heads, buckets):
    """Each head has a part of the sum at least, whatever their number."""
    parts = heads * buckets * 4
    need = lib.csr_rel_bias_grad_workspace_bytes(1 << 20, 1 << 20, 1, heads, buckets)
    assert need >= parts and need % parts == 0
    assert need // parts <= -(-456 // heads)


def test_binding_refuses_without_gpu():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    with pytest.raises(RuntimeError, match="no CUDA device"):
        usm.rel_bias(None, None, None, None, None)
    with pytest.raises(RuntimeError, match="no CUDA device"):
        usm.attention(None, None, None, None, None)


# ---------------------------------------------------------------------------
# The 64-bit definitions' own checks: gradients against central differences.
# ---------------------------------------------------------------------------
def _small():
    rng = np.random.default_rng(7)
    ro = np.array([0, 3, 3, 4, 9])
    return rng, ro, rng.standard_normal(9), rng.standard_normal(9), rng.standard_normal(9)


def _difference(f, x, h=1e-6):
    g = np.zeros(x.size)
    for i in range(x.size):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


def test_definitions_of_gradients_match_differences():
    rng, ro, s1, s2, w = _small()
    lam, heads = np.array([0.3, 0.8]), R.head_of_rows(4, 2, 2)
    f = lambda a, b, l: np.sum(w * R.diff_map(ro, a, b, l[heads]))
    g1, g2, gl = R.diff_grad(ro, s1, s2, lam[heads], w, 2, heads)
    # Central differences: truncation h^2/6 times third derivatives of order
    # one, and rounding 2^-52/h of sums of order ten: below 1e-8.
    assert np.allclose(g1, _difference(lambda x: f(x, s2, lam), s1), atol=1e-8)
    assert np.allclose(g2, _difference(lambda x: f(s1, x, lam), s2), atol=1e-8)
    assert np.allclose(gl, _difference(lambda x: f(s1, s2, x), lam), atol=1e-8)
    gs, _, _ = R.softmax_grad(ro, s1, w)
    assert np.allclose(gs, _difference(lambda x: np.sum(w * R.row_softmax(ro, x)), s1), atol=1e-8)


def test_definition_of_buckets():
    # 32 buckets, reach 128, both directions: e = 8, boundaries 8·16^(i/8).
    f = lambda d: R.log_bucket(d, 32, 128, False)
    assert [f(-n) for n in (0, 1, 7, 8, 11, 12, 15, 16, 22, 23, 31, 32, 45, 46, 63, 64, 90, 91, 128, 5000)] == \
        [0, 1, 7, 8, 8, 9, 9, 10, 10, 11, 11, 12, 12, 13, 13, 14, 14, 15, 15, 15]
    assert f(1) == 17 and f(128) == 31
    g = lambda d: R.log_bucket(d, 32, 128, True)
    assert g(5) == 0 and g(-15) == 15 and g(-16) == 16 and g(-128) == 31
