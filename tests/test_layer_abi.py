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
