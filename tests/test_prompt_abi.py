"""The entry points of svgemm_prompt.h: exported as declared, and refusing bad
arguments on the host with the documented status codes.  No GPU: every call here
fails a check (or is an empty call) before anything could be enqueued, so no
pointer passed is ever dereferenced."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "svgemm_prompt.h")

A = 0x10000      # aligned, never dereferenced
MIS = 0x10002    # 2-byte aligned


@pytest.fixture(scope="module")
def svg():
    import speculative_verify_gemm_amd as svg
    return svg


def test_every_declared_call_is_exported_and_bound(svg):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^svg_status\s+(\w+)\s*\(", text, flags=re.M)))
    assert len(names) == 7
    for name in names:
        fn = getattr(svg.lib, name)
        assert ctypes.cast(fn, ctypes.c_void_p).value and fn.argtypes, name
        if not name.endswith("_workspace"):
            assert callable(getattr(svg, name))


def cache(svg, **kw):
    f = dict(k=A, v=A, type=1, heads=2, dim=64, page=32, n_pages=8, n_layers=2, n_slots=2, width=4, table=A, pages=A,
             len=A, refs=A)
    f.update(kw)
    return svg.layer.KVCacheC(*f.values())


def call(svg, name, defaults, c=None, **kw):
    a = dict(defaults)
    a.update(kw)
    first = [] if c is False else [ctypes.byref(c or cache(svg))]
    return getattr(svg.lib, name)(*first, *a.values(), None)


MAP = dict(n_new=A, parent=None, T=0, n_rows=10, start=A, count=A, slot=None, pos=A, place=A)


@pytest.mark.parametrize("kw,code", [
    (dict(n_new=None), 1), (dict(start=None), 1), (dict(count=None), 1), (dict(pos=None), 1), (dict(place=None), 1), (dict(T=-1), 1),
    (dict(n_rows=-1), 1), (dict(T=4), 1), (dict(parent=A), 1), (dict(parent=A, T=33, n_rows=66), 2), (dict(T=1 << 30), 2),
    (dict(n_new=MIS), 3), (dict(parent=MIS, T=5), 3), (dict(start=MIS), 3), (dict(count=MIS), 3), (dict(slot=MIS), 3), (dict(pos=MIS), 3),
    (dict(place=MIS), 3),
])
def test_row_map_refusals(svg, kw, code):
    assert call(svg, "kv_row_map", MAP, **kw) == code
    assert svg.last_error().startswith("kv_row_map:")


class RopeArgs(dict):
    pass


ROPE = dict(layer=0, rope=None, q=A, ld_q=256, heads=4, k=A, ld_k=128, v=A, ld_v=128, xt=0, n_rows=3, pos=A, place=A, q_out=A, qt=0)


def rope(svg, freq=A, rot=64, inter=0, amp=1.0, c=None, **kw):
    a = dict(ROPE, rope=ctypes.byref(svg.prompt.RopeC(freq, rot, inter, amp)))
    a.update(kw)
    return svg.lib.rope_append(ctypes.byref(c or cache(svg)), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(rope=None), 1), (dict(layer=2), 1), (dict(layer=-1), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(pos=None), 1),
    (dict(place=None), 1), (dict(q_out=None), 1), (dict(freq=None), 1), (dict(n_rows=-1), 1), (dict(heads=-1), 1),
    (dict(amp=float("nan")), 1), (dict(amp=float("inf")), 1),
    (dict(rot=0), 2), (dict(rot=24), 2), (dict(rot=80), 2), (dict(xt=3), 2), (dict(xt=-1), 2), (dict(qt=2), 2), (dict(heads=4097, ld_q=1 << 20), 2),
    (dict(ld_q=255), 2), (dict(ld_k=127), 2), (dict(ld_v=64), 2), (dict(ld_k=1 << 31), 2),
    (dict(q=MIS), 3), (dict(k=MIS), 3), (dict(v=MIS), 3), (dict(q_out=MIS), 3), (dict(ld_q=258), 3), (dict(ld_k=132, xt=1), 3), (dict(ld_v=130), 3),
    (dict(freq=A + 4), 3), (dict(pos=MIS), 3), (dict(place=MIS), 3),
])
def test_rope_refusals(svg, kw, code):
    assert rope(svg, **kw) == code
    assert svg.last_error().startswith("rope_append:")


def test_empty_calls(svg):
    none = cache(svg, n_slots=0, width=0, table=None, pages=None, len=None, refs=None)
    assert call(svg, "kv_row_map", MAP, c=none, n_rows=0, n_new=None, start=None, count=None, pos=None, place=None) == 0
    assert rope(svg, n_rows=0, q=None, k=None, v=None, pos=None, place=None, q_out=None) == 0
    assert call(svg, "prompt_attention", ATT, c=none) == 0 and call(svg, "prompt_attention", ATT, n_rows=0, q=None, out=None) == 0
    assert call(svg, "w8a8_prompt_linear", W8, c=False, M=0, xq=None) == 0 and call(svg, "w8a8_prompt_linear", W8, c=False, N=0, wq=None) == 0
    assert call(svg, "w4a8_prompt_linear", W4, c=False, M=0, y=None) == 0
    assert call(svg, "gated_quant_i8", GATE, c=False, M=0, x=None) == 0
    assert svg.last_error() == ""


ATT = dict(layer=0, q=A, ld=512, heads=8, n_rows=5, start=A, count=A, scale=0.1, out=A, ws=A)


@pytest.mark.parametrize("kw,code", [
    (dict(layer=2), 1), (dict(layer=-1), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(start=None), 1), (dict(count=None), 1),
    (dict(n_rows=-1), 1), (dict(heads=0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(heads=7), 2),
    (dict(heads=4098, ld=1 << 20), 2), (dict(ld=511), 2), (dict(ld=1 << 31), 2), (dict(n_rows=1 << 28), 2), (dict(q=MIS), 3), (dict(ld=516), 3),
    (dict(out=MIS), 3), (dict(ws=A + 128), 3), (dict(start=MIS), 3), (dict(count=MIS), 3),
])
def test_attention_refusals(svg, kw, code):
    assert call(svg, "prompt_attention", ATT, **kw) == code
    assert svg.last_error().startswith("prompt_attention:")


def cache_refusals():
    bad = [(dict(k=None), 1), (dict(v=None), 1), (dict(type=0), 2), (dict(dim=96), 2), (dict(page=16), 2), (dict(heads=0), 2), (dict(n_pages=0), 2),
           (dict(n_layers=0), 2), (dict(k=MIS), 3)]
    tables = [(dict(n_slots=-1), 1), (dict(n_slots=1025), 2), (dict(width=1 << 26), 2), (dict(table=None), 1), (dict(pages=MIS + 1), 3),
              (dict(len=None), 1)]
    return [(n, kw, code) for n in ("kv_row_map", "rope_append", "prompt_attention") for kw, code in bad + ([] if n == "rope_append" else tables)]


@pytest.mark.parametrize("name,kw,code", cache_refusals())
def test_cache_refusals(svg, name, kw, code):
    c = cache(svg, **kw)
    got = rope(svg, c=c) if name == "rope_append" else call(svg, name, MAP if name == "kv_row_map" else ATT, c=c)
    assert got == code
    assert svg.last_error().startswith(name + ":")


def test_attention_workspace(svg):
    n = ctypes.c_uint64()

    def size(heads, rows, **kw):
        assert svg.lib.prompt_attention_workspace(ctypes.byref(cache(svg, **kw)), heads, rows, ctypes.byref(n)) == 0
        return n.value

    assert size(8, 5, dim=128) > size(8, 5) > 128 * 64 * 4
    assert size(8, 0) == 0 and size(8, 5, n_slots=0) == 0
    assert svg.lib.prompt_attention_workspace(ctypes.byref(cache(svg)), 8, 5, None) == 1
    assert svg.lib.prompt_attention_workspace(ctypes.byref(cache(svg)), 7, 5, ctypes.byref(n)) == 2


W8 = dict(xq=A, xs=A, M=40, K=128, wq=A, ws=A, N=48, y=A, yt=0)
W4 = dict(xq=A, xs=A, M=40, K=128, wq=A, ws=A, wz=A, fmt=1, group=64, N=48, y=A, yt=0)
LINEAR = [
    (dict(xq=None), 1), (dict(xs=None), 1), (dict(wq=None), 1), (dict(ws=None), 1), (dict(y=None), 1), (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=0), 1),
    (dict(K=-32), 1), (dict(yt=3), 2), (dict(K=48), 2), (dict(K=131072 + 32), 2), (dict(M=(1 << 24) + 1), 2), (dict(M=1 << 24, K=65536), 2),
    (dict(M=1 << 24, N=1 << 16, K=32 * 32), 2), (dict(xq=MIS), 3), (dict(wq=MIS), 3), (dict(xs=MIS), 3), (dict(ws=MIS), 3), (dict(y=MIS), 3),
]


@pytest.mark.parametrize("kw,code", LINEAR)
def test_linear_refusals(svg, kw, code):
    assert call(svg, "w8a8_prompt_linear", W8, c=False, **kw) == code
    assert svg.last_error().startswith("w8a8_prompt_linear:")
    assert call(svg, "w4a8_prompt_linear", W4, c=False, **kw) == code
    assert svg.last_error().startswith("w4a8_prompt_linear:")


@pytest.mark.parametrize("kw,code", [(dict(fmt=2), 2), (dict(fmt=3), 2), (dict(group=16), 2), (dict(K=96), 2), (dict(K=64, group=128), 2),
                                     (dict(wz=None), 1), (dict(wz=MIS), 3)])
def test_w4_refusals(svg, kw, code):
    assert call(svg, "w4a8_prompt_linear", W4, c=False, **kw) == code


GATE = dict(x=A, ld_x=256, gate=A, ld_g=256, xt=1, M=40, K=128, signs=A, block=32, xq=A, xs=A)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(signs=None), 1), (dict(xq=None), 1), (dict(xs=None), 1), (dict(M=-1), 1), (dict(K=0), 1), (dict(xt=3), 2), (dict(block=16), 2),
    (dict(K=48), 2), (dict(K=96, block=64), 2), (dict(K=32800, ld_x=40000, ld_g=40000), 2), (dict(M=(1 << 24) + 1), 2), (dict(ld_x=127), 2),
    (dict(ld_g=64), 2), (dict(ld_x=1 << 31), 2), (dict(x=MIS), 3), (dict(gate=MIS), 3), (dict(ld_x=252), 3), (dict(ld_g=260), 3), (dict(xq=MIS), 3),
    (dict(signs=MIS), 3), (dict(xs=MIS), 3),
])
def test_gate_refusals(svg, kw, code):
    assert call(svg, "gated_quant_i8", GATE, c=False, **kw) == code
    assert svg.last_error().startswith("gated_quant_i8:")
