"""The entry points of svgemm_layer.h: exported as declared, and refusing bad
arguments on the host with the documented status codes.  No GPU: every call
here fails a check (or is an empty call) before anything could be enqueued, so
no pointer passed is ever dereferenced."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "svgemm_layer.h")

A = 0x10000      # aligned, never dereferenced
MIS = 0x10002    # 2-byte aligned


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^svg_status\s+(\w+)\s*\(", text, flags=re.M)))


@pytest.fixture(scope="module")
def svg():
    import speculative_verify_gemm_amd as svg
    return svg


def test_every_declared_call_is_exported_and_bound(svg):
    assert "add_rmsnorm_quant_i8" in declared()
    for name in declared():
        fn = getattr(svg.lib, name)
        assert ctypes.cast(fn, ctypes.c_void_p).value and fn.argtypes, name


def norm(svg, **kw):
    a = dict(x=A, xt=0, res=A, w=A, wt=0, eps=1e-6, M=4, K=128, signs=A, block=32, y=None, xq=A, xs=A)
    a.update(kw)
    return svg.lib.add_rmsnorm_quant_i8(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(signs=None), 1), (dict(xq=None), 1), (dict(xs=None), 1),
    (dict(M=-1), 1), (dict(K=0), 1), (dict(eps=0.0), 1), (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1),
    (dict(xt=3), 2), (dict(wt=-1), 2), (dict(block=16), 2), (dict(K=48), 2), (dict(K=96, block=64), 2),
    (dict(K=32800), 2), (dict(M=(1 << 24) + 1), 2),
    (dict(x=MIS), 3), (dict(res=MIS), 3), (dict(w=MIS), 3), (dict(y=MIS), 3), (dict(xq=MIS), 3), (dict(xs=MIS), 3),
    (dict(signs=MIS), 3),
])
def test_norm_refusals(svg, kw, code):
    assert norm(svg, **kw) == code
    assert svg.last_error().startswith("add_rmsnorm_quant_i8:")


def test_empty_norm(svg):
    assert norm(svg, M=0) == 0 and svg.last_error() == ""
    assert norm(svg, M=0, res=None, y=None) == 0


# ---------------------------------------------------------------- the cache
def cache(svg, **kw):
    f = dict(k=A, v=A, type=1, heads=2, dim=64, page=32, n_pages=8, n_layers=2, n_slots=2, width=4, table=A, pages=A,
             len=A, refs=A)
    f.update(kw)
    return svg.layer.KVCacheC(*f.values())


CACHE_CALLS = {
    "kv_append": lambda L, c: L.kv_append(c, 0, A, 128, A, 128, 1, None, None),
    "kv_commit": lambda L, c: L.kv_commit(c, 4, A, A, A + 64, None),
    "kv_fork": lambda L, c: L.kv_fork(c, A, A + 64, A + 64, A + 64, None),
    "kv_reserve": lambda L, c: L.kv_reserve(c, A, A, A, None),
    "kv_copy_pages": lambda L, c: L.kv_copy_pages(c, A, A, 1, None),
    "tree_attention": lambda L, c: L.tree_attention(c, 0, A, 512, 8, A, 4, None, None, 0.1, A, A, None),
    "tree_attention_workspace": lambda L, c: L.tree_attention_workspace(c, 8, 4, ctypes.byref(ctypes.c_uint64())),
}
NO_TABLES = {"kv_copy_pages"}


def cache_refusals():
    bad = [(dict(k=None), 1), (dict(v=None), 1), (dict(type=0), 2), (dict(type=3), 2), (dict(dim=96), 2), (dict(page=16), 2),
           (dict(heads=0), 2), (dict(heads=1025), 2), (dict(n_pages=0), 2), (dict(n_pages=(1 << 20) + 1), 2),
           (dict(n_layers=0), 2), (dict(n_layers=65536), 2), (dict(k=MIS), 3), (dict(v=MIS), 3)]
    tables = [(dict(n_slots=-1), 1), (dict(width=-1), 1), (dict(n_slots=1025), 2), (dict(width=1 << 26), 2),
              (dict(table=None), 1), (dict(pages=MIS + 1), 3), (dict(len=None), 1)]
    return [(call, kw, code) for call in CACHE_CALLS for kw, code in bad + ([] if call in NO_TABLES else tables)]


@pytest.mark.parametrize("call,kw,code", cache_refusals())
def test_cache_refusals(svg, call, kw, code):
    assert CACHE_CALLS[call](svg.lib, ctypes.byref(cache(svg, **kw))) == code
    assert svg.last_error().startswith(call + ":")
    assert CACHE_CALLS[call](svg.lib, None) == 1


@pytest.mark.parametrize("call", [c for c in CACHE_CALLS if c not in NO_TABLES])
def test_no_slots_is_an_empty_call(svg, call):
    c = cache(svg, n_slots=0, width=0, table=None, pages=None, len=None, refs=None)
    assert CACHE_CALLS[call](svg.lib, ctypes.byref(c)) == 0


def test_cache_call_refusals(svg):
    L, c = svg.lib, ctypes.byref(cache(svg))
    for args, code in (((2, A, 128, A, 128, 1, None), 1), ((-1, A, 128, A, 128, 1, None), 1), ((0, None, 128, A, 128, 1, None), 1),
                       ((0, A, 128, None, 128, 1, None), 1), ((0, A, 128, A, 128, 0, None), 1), ((0, A, 124, A, 128, 1, None), 2),
                       ((0, A, 130, A, 128, 1, None), 2), ((0, A, 128, A, 1 << 31, 1, None), 2), ((0, A, 128, A, 128, 1 << 30, None), 2),
                       ((0, MIS, 128, A, 128, 1, None), 3), ((0, A, 128, MIS, 128, 1, None), 3), ((0, A, 128, A, 128, 1, MIS), 3)):
        assert L.kv_append(c, *args, None) == code, args
    for args, code in (((0, A, A, A), 1), ((33, A, A, A), 2), ((4, None, A, A), 1), ((4, A, None, A), 1), ((4, A, A, None), 1),
                       ((4, MIS, A, A), 3), ((4, A, MIS, A), 3), ((4, A, A, MIS), 3)):
        assert L.kv_commit(c, *args, None) == code, args
    B = A + 64
    for args, code in (((None, B, B, B), 1), ((A, None, B, B), 1), ((A, A, B, B), 1), ((A, B, A, B), 1), ((A, B, B, A), 1),
                       ((MIS, B, B, B), 3), ((A, B, B, MIS), 3)):
        assert L.kv_fork(c, *args, None) == code, args
    assert L.kv_fork(ctypes.byref(cache(svg, refs=None)), A, B, B, B, None) == 1
    for args, code in (((None, A, A), 1), ((A, None, A), 1), ((A, A, None), 1), ((A, A, A + 4), 3), ((MIS, A, A), 3)):
        assert L.kv_reserve(c, *args, None) == code, args
    for args, code in (((A, A, -1), 1), ((None, A, 1), 1), ((A, None, 1), 1), ((MIS, A, 1), 3), ((None, None, 0), 0)):
        assert L.kv_copy_pages(c, *args, None) == code, args


def attention(svg, c=None, **kw):
    a = dict(layer=0, q=A, ld=512, heads=8, parent=A, T=4, n=None, shared=None, scale=0.1, out=A, ws=A)
    a.update(kw)
    return svg.lib.tree_attention(ctypes.byref(c or cache(svg)), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(layer=2), 1), (dict(layer=-1), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(T=0), 1),
    (dict(heads=0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(T=33), 2), (dict(heads=7), 2),
    (dict(heads=4098, ld=1 << 20), 2), (dict(ld=508), 2), (dict(ld=514), 2), (dict(ld=1 << 31), 2), (dict(q=MIS), 3),
    (dict(out=MIS), 3), (dict(ws=A + 128), 3), (dict(parent=MIS), 3), (dict(n=MIS), 3), (dict(shared=MIS), 3),
])
def test_attention_refusals(svg, kw, code):
    assert attention(svg, **kw) == code
    assert svg.last_error().startswith("tree_attention:")


def test_attention_workspace_sizes(svg):
    n = ctypes.c_uint64()

    def size(heads, T, **kw):
        assert svg.lib.tree_attention_workspace(ctypes.byref(cache(svg, **kw)), heads, T, ctypes.byref(n)) == 0
        return n.value

    # a partial for each of 512 workgroups at least: one row tile of 16 rows, dim + 2 values
    assert size(2, 1, n_slots=1) >= 512 * 16 * 66 * 4
    assert size(8, 32, n_slots=8) > size(8, 1, n_slots=8) > size(8, 1, n_slots=1)
    assert size(8, 4, n_slots=0) == 0
    assert svg.lib.tree_attention_workspace(ctypes.byref(cache(svg)), 8, 4, None) == 1
