"""Refusals and sizes of the packed-sequence and paged-cache calls, found on
the host before anything is enqueued (no GPU needed)."""
import ctypes

import pytest

from int4_quantized_attention_b200 import api, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.lib()


A = 1 << 20   # an aligned address that no call below gets to use


def packed(**kw):
    base = dict(n_seqs=2, Hq=8, Hkv=2, d=128, dtype=0, causal=1, total_q=50, total_k=60, scale=0.0, q_token=1024,
                q_head=128, k_token=256, k_head=128, v_token=256, v_head=128, o_token=1024, o_head=128)
    base.update(kw)
    return api.Packed(**base)


def call_packed(lib, p, q=A, k=A, v=A, cq=A, ck=A, o=A, lse=None, ws=A, size=1 << 40):
    return lib.ra_packed_attention_fwd(ctypes.byref(p) if p is not None else None, q, k, v, cq, ck, o, lse, ws, size,
                                       None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=64), api.RA_ERR_UNSUPPORTED), (dict(Hq=7), api.RA_ERR_INVALID_ARG), (dict(Hq=0), api.RA_ERR_INVALID_ARG),
    (dict(Hkv=0), api.RA_ERR_INVALID_ARG), (dict(Hq=258), api.RA_ERR_UNSUPPORTED),
    (dict(n_seqs=0), api.RA_ERR_INVALID_ARG), (dict(dtype=2), api.RA_ERR_INVALID_ARG),
    (dict(causal=2), api.RA_ERR_INVALID_ARG), (dict(total_q=-1), api.RA_ERR_INVALID_ARG),
    (dict(total_k=1 << 30 | 1), api.RA_ERR_UNSUPPORTED), (dict(scale=-1.0), api.RA_ERR_INVALID_ARG),
    (dict(scale=1e-60), api.RA_ERR_INVALID_ARG), (dict(total_q=1 << 29, Hq=4096, Hkv=4096, q_token=4096 * 128,
                                                       o_token=4096 * 128), api.RA_ERR_UNSUPPORTED),
    (dict(scale=float("nan")), api.RA_ERR_INVALID_ARG), (dict(scale=float("inf")), api.RA_ERR_INVALID_ARG),
    (dict(q_token=1020), api.RA_ERR_INVALID_ARG), (dict(k_head=0), api.RA_ERR_INVALID_ARG),
    (dict(v_token=0), api.RA_ERR_INVALID_ARG), (dict(o_token=512), api.RA_ERR_INVALID_ARG),
    (dict(o_head=0), api.RA_ERR_INVALID_ARG),
])
def test_packed_problem_refusals(lib, kw, status):
    p = packed(**kw)
    assert api.packed_workspace_bytes(p) == 0
    assert call_packed(lib, p) == status
    assert lib.ra_last_error_detail()


def test_packed_pointer_refusals(lib):
    p = packed()
    need = api.packed_workspace_bytes(p)
    assert need > 256
    for kw in (dict(q=None), dict(k=A + 2), dict(v=None), dict(cq=None), dict(ck=A + 1), dict(o=A + 8), dict(ws=None),
               dict(ws=A + 16), dict(lse=A + 2)):
        assert call_packed(lib, p, **kw) == api.RA_ERR_INVALID_ARG, kw
    assert call_packed(lib, p, size=need - 1) == api.RA_ERR_WORKSPACE
    assert call_packed(lib, None) == api.RA_ERR_INVALID_ARG


def test_packed_layouts_accepted(lib):
    # head-major tensors, and anything for the stride of a dimension of one entry
    assert api.packed_workspace_bytes(packed(q_token=128, q_head=6400, o_token=128, o_head=6400)) > 0
    assert api.packed_workspace_bytes(packed(Hq=1, Hkv=1, q_head=0, k_head=1, v_head=3, o_head=0)) > 0
    assert api.packed_workspace_bytes(packed(total_q=1, q_token=0, o_token=0)) > 0


def cache(**kw):
    base = dict(layers=2, n_pages=10, page_size=16, Hkv=2, d=128, dtype=1, max_seqs=4, max_pages=5)
    base.update(kw)
    return api.CacheProblem(**base)


C = api.Cache(A, A, A, A, A)


@pytest.mark.parametrize("kw,status", [
    (dict(d=96), api.RA_ERR_UNSUPPORTED), (dict(page_size=8), api.RA_ERR_UNSUPPORTED),
    (dict(page_size=48), api.RA_ERR_UNSUPPORTED), (dict(page_size=256), api.RA_ERR_UNSUPPORTED),
    (dict(layers=0), api.RA_ERR_INVALID_ARG), (dict(n_pages=0), api.RA_ERR_INVALID_ARG),
    (dict(Hkv=0), api.RA_ERR_INVALID_ARG), (dict(max_seqs=0), api.RA_ERR_INVALID_ARG),
    (dict(max_pages=0), api.RA_ERR_INVALID_ARG), (dict(dtype=7), api.RA_ERR_INVALID_ARG),
    (dict(max_seqs=1 << 20, max_pages=1 << 11), api.RA_ERR_UNSUPPORTED),
    (dict(page_size=128, max_pages=1 << 23), api.RA_ERR_UNSUPPORTED),
    (dict(n_pages=1 << 23, layers=200, page_size=128), api.RA_ERR_UNSUPPORTED),
])
def test_cache_problem_refusals(lib, kw, status):
    p = cache(**kw)
    assert api.cache_validate(p) == status
    assert api.cache_pool_bytes(p) == api.cache_state_bytes(p) == api.cache_workspace_bytes(p) == 0
    assert lib.ra_cache_compact(ctypes.byref(p), ctypes.byref(C), A, 1 << 40, None) == status


def test_cache_sizes_and_binding(lib):
    p = cache()
    assert api.cache_pool_bytes(p) == 2 * 2 * 10 * 2 * 16 * 256
    assert api.cache_state_bytes(p) == 3 * 256                       # 40, 16 and 80 bytes, each on 256
    out = api.Cache()
    args = (ctypes.byref(p), A, api.cache_pool_bytes(p), 2 * A, api.cache_state_bytes(p))
    assert lib.ra_cache_bind(*args, ctypes.byref(out)) == api.RA_OK
    assert (out.k, out.v, out.refs, out.lens, out.table) == (A, A + 2 * 10 * 2 * 16 * 256, 2 * A, 2 * A + 256, 2 * A + 512)
    assert lib.ra_cache_bind(args[0], A, args[2] - 1, 2 * A, args[4], ctypes.byref(out)) == api.RA_ERR_INVALID_ARG
    assert lib.ra_cache_bind(args[0], A, args[2], 2 * A, args[4] - 1, ctypes.byref(out)) == api.RA_ERR_INVALID_ARG
    assert lib.ra_cache_bind(args[0], A + 16, args[2], 2 * A, args[4], ctypes.byref(out)) == api.RA_ERR_INVALID_ARG
    assert lib.ra_cache_bind(*args, None) == api.RA_ERR_INVALID_ARG


def test_cache_call_refusals(lib):
    p, size = ctypes.byref(cache()), 1 << 40
    c = ctypes.byref(C)
    bad = ctypes.byref(api.Cache(A, A, A, None, A))
    inv = api.RA_ERR_INVALID_ARG
    assert lib.ra_cache_extend(p, bad, A, A, 1, A, size, None) == inv
    assert lib.ra_cache_extend(p, None, A, A, 1, A, size, None) == inv
    assert lib.ra_cache_extend(p, c, A, A, 5, A, size, None) == inv           # more rows than the table has
    assert lib.ra_cache_extend(p, c, A, None, 1, A, size, None) == inv
    assert lib.ra_cache_extend(p, c, A, A, -1, A, size, None) == inv
    assert lib.ra_cache_extend(p, c, A, A, 1, A + 16, size, None) == inv
    assert lib.ra_cache_extend(p, c, A, A, 1, A, 256, None) == api.RA_ERR_WORKSPACE
    assert lib.ra_cache_extend(p, c, None, None, 0, A, size, None) == api.RA_OK
    assert lib.ra_cache_fork(p, c, A, None, 1, A, size, None) == inv
    assert lib.ra_cache_free(p, c, None, 1, A, size, None) == inv
    w = lambda layer=0, n=2, total=2, cu=None, k=A, kt=256, kh=128: lib.ra_cache_write(   # noqa: E731
        p, c, layer, A, cu, n, total, k, A, kt, kh, 256, 128, A, size, None)
    assert w(layer=2) == inv and w(layer=-1) == inv and w(total=3) == inv and w(n=0, total=1, cu=A) == inv
    assert w(k=None) == inv and w(kt=100) == inv and w(kh=0) == inv and w(total=-1, cu=A) == inv
    assert w(n=0, total=0) == api.RA_OK


def attn(**kw):
    base = dict(n_seqs=2, Hq=8, total_q=2, layer=0, shared=0, scale=0.0, q_token=1024, q_head=128, o_token=1024, o_head=128)
    base.update(kw)
    return api.CacheAttn(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=7), api.RA_ERR_INVALID_ARG), (dict(Hq=512), api.RA_ERR_UNSUPPORTED), (dict(n_seqs=0), api.RA_ERR_INVALID_ARG),
    (dict(total_q=-2), api.RA_ERR_INVALID_ARG), (dict(layer=2), api.RA_ERR_INVALID_ARG),
    (dict(shared=8), api.RA_ERR_INVALID_ARG), (dict(shared=-16), api.RA_ERR_INVALID_ARG),
    (dict(shared=96), api.RA_ERR_INVALID_ARG), (dict(scale=-2.0), api.RA_ERR_INVALID_ARG),
    (dict(q_head=4), api.RA_ERR_INVALID_ARG), (dict(o_token=128), api.RA_ERR_INVALID_ARG),
])
def test_cache_attention_refusals(lib, kw, status):
    p, a = cache(), attn(**kw)
    assert api.cache_attention_workspace_bytes(p, a) == 0
    f = lib.ra_cache_attention_fwd
    assert f(ctypes.byref(p), ctypes.byref(C), ctypes.byref(a), A, A, None, A, None, A, 1 << 40, None) == status


def test_cache_attention_pointer_refusals(lib):
    p, a, inv = cache(), attn(), api.RA_ERR_INVALID_ARG
    f = lambda q=A, seqs=A, cu=None, o=A, lse=None, ws=A, size=1 << 40, c=C, a=a: lib.ra_cache_attention_fwd(   # noqa: E731
        ctypes.byref(p), ctypes.byref(c), ctypes.byref(a), q, seqs, cu, o, lse, ws, size, None)
    assert f(q=None) == inv and f(seqs=None) == inv and f(cu=A + 2) == inv and f(o=A + 4) == inv
    assert f(lse=A + 1) == inv and f(ws=A + 64) == inv and f(c=api.Cache(A, A, A, A, None)) == inv
    assert f(a=attn(total_q=3)) == inv                                # single tokens: one row each
    assert f(size=api.cache_attention_workspace_bytes(p, a) - 1) == api.RA_ERR_WORKSPACE
