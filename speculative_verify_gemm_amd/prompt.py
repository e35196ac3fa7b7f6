"""Python binding of include/svgemm_prompt.h: a prompt's pass through a decoder
layer.  Argument marshalling only, as in the package's other modules: every
function checks devices, dtypes and shapes and calls the C entry point of the
same name on the current stream of the tensors' device (or the stream given)."""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from .layer import _FLOATS, _call, _device, _slots, _tensor, KVCacheC

_lib = None  # the library, once the package has loaded it (_bind)
_I32 = torch.int32


class RopeC(ctypes.Structure):
    """svg_rope (include/svgemm_prompt.h)."""
    _fields_ = [("freq", ctypes.c_void_p), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int), ("amplitude", ctypes.c_float)]


def _bind(lib):
    global _lib
    _lib = lib
    vp, i, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    kv, rope = ctypes.POINTER(KVCacheC), ctypes.POINTER(RopeC)
    lib.kv_row_map.argtypes = [kv, vp, vp, i, i, vp, vp, vp, vp, vp, vp]
    lib.rope_append.argtypes = [kv, i, rope, vp, i64, i, vp, i64, vp, i64, i, i, vp, vp, vp, i, vp]
    lib.prompt_attention_workspace.argtypes = [kv, i, i, ctypes.POINTER(ctypes.c_uint64)]
    lib.prompt_attention.argtypes = [kv, i, vp, i64, i, i, vp, vp, ctypes.c_float, vp, vp, vp]
    lib.w4a8_prompt_linear.argtypes = [vp, vp, i, i, vp, vp, vp, i, i, i, vp, i, vp]
    lib.w8a8_prompt_linear.argtypes = [vp, vp, i, i, vp, vp, i, vp, i, vp]
    lib.gated_quant_i8.argtypes = [vp, i64, vp, i64, i, i, i, vp, i, vp, vp, vp]
    for fn in (lib.kv_row_map, lib.rope_append, lib.prompt_attention_workspace, lib.prompt_attention, lib.w4a8_prompt_linear,
               lib.w8a8_prompt_linear, lib.gated_quant_i8):
        fn.restype = ctypes.c_int


def _float_rows(t, name, dev, dtype, width=None):
    """Rows [n, ...] of contiguous values of a float type (dtype, or any): (address, row stride, n, type number)."""
    kind = _FLOATS.get(t.dtype)
    if kind is None or (dtype is not None and t.dtype is not dtype):
        raise TypeError(f"{name} must be {dtype or 'float32, float16 or bfloat16'}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        ok = (width is None or shape[1] * shape[2] == width) and stride[2] == 1 and (stride[1] == shape[2] or shape[1] == 1)
        wide = shape[1] * shape[2]
    else:
        ok = len(shape) == 2 and (width is None or shape[1] == width) and (stride[1] == 1 or shape[1] == 1)
        wide = shape[-1]
    if not ok:
        raise ValueError(f"{name} must be [n, {'width' if width is None else width}] or [n, heads, dim] with contiguous rows")
    n = shape[0]
    return t.data_ptr(), (stride[0] if n > 1 else wide), n, kind


# ------------------------------------------------------------------ row map
class RowMap:
    """Where a step's rows belong (kv_row_map writes it, rope_append and
    prompt_attention read it): start and count int32 [n_slots], pos and place
    int32 [n_rows], and, if wanted, slot int32 [n_rows].  The object keeps the
    tensors; without pos and place (n_rows given) only prompt_attention takes it.
    The tensors may be set to others of the same shape and device (calls that a
    graph has captured go on with the ones they were made with)."""

    def __init__(self, start, count, pos=None, place=None, slot=None, n_rows=None):
        dev = _device(start, "start")
        if start.dim() != 1 or count.shape != start.shape:
            raise ValueError("start and count must be [n_slots]")
        if (pos is None) != (place is None) or (pos is None and n_rows is None):
            raise ValueError("need pos and place, or n_rows")
        if pos is not None and (pos.dim() != 1 or place.shape != pos.shape or (slot is not None and slot.shape != pos.shape)):
            raise ValueError("pos, place and slot must be [n_rows]")
        if pos is not None and n_rows is not None and n_rows != pos.shape[0]:
            raise ValueError("n_rows must be the length of pos")
        self._t = dict(start=start, count=count, slot=slot, pos=pos, place=place)
        self.device, self.n_slots = dev, start.shape[0]
        self.n_rows = pos.shape[0] if pos is not None else int(n_rows)
        self._p = [None if t is None else _tensor(t, name, _I32, dev) for name, t in self._t.items()]

    def _set(self, name, t):
        now = self._t[name]
        if now is None:
            raise ValueError(f"rows has no {name}")
        if t is None or t.shape != now.shape:
            raise ValueError(f"{name} must have shape {list(now.shape)}")
        self._p[list(self._t).index(name)] = _tensor(t, name, _I32, self.device)
        self._t[name] = t

    @classmethod
    def empty(cls, cache, n_rows):
        """Buffers for `n_rows` rows of the cache's slots (a row of no slot in all of them)."""
        none = lambda n: torch.full((n,), -1, dtype=_I32, device=cache.device)  # noqa: E731
        zero = lambda: torch.zeros(cache.n_slots, dtype=_I32, device=cache.device)  # noqa: E731
        return cls(zero(), zero(), none(n_rows), none(n_rows), none(n_rows))


for _name in ("start", "count", "slot", "pos", "place"):
    setattr(RowMap, _name, property(lambda self, n=_name: self._t[n], lambda self, t, n=_name: self._set(n, t)))


def kv_row_map(cache, n_new, rows, T=0, parent=None, stream=None):
    """Fill `rows` (a RowMap) for a step in which slot s has n_new[s] new rows
    (int32 [n_slots]): packed one slot after another (T = 0), or T a slot, chains
    or draft trees (parent int32 [n_slots, T]).  Behind kv_reserve; once for all layers."""
    if rows.device != cache.device or rows.n_slots != cache.n_slots:
        raise ValueError("rows must be a RowMap of the cache's device and number of slots")
    if rows._p[3] is None:
        raise ValueError("rows has no pos and place")
    pp = None if parent is None else _slots(parent, "parent", cache, T)
    _call(_lib.kv_row_map, cache.device, stream, cache._ref, _slots(n_new, "n_new", cache), pp, T, rows.n_rows, *rows._p)


# --------------------------------------------------------------------- rope
class Rope:
    """Rotary positions: the angle of pair i at position p is p * freq[i], freq
    float64 [rot / 2] on the device; pairs (2 i, 2 i + 1) if interleaved, else
    (i, i + rot / 2); cosines and sines are multiplied by amplitude.  The object
    keeps freq, which may be set to another tensor of its shape and device, as
    interleaved and amplitude may be set anew (calls that a graph has captured go on
    with what they were made with)."""

    def __init__(self, freq, interleaved=False, amplitude=1.0):
        dev = _device(freq, "freq")
        if freq.dim() != 1:
            raise ValueError("freq must be [rot / 2]")
        self.device, self.rot = dev, 2 * freq.shape[0]
        self._c = RopeC(None, self.rot)
        self._ref = ctypes.byref(self._c)
        self.freq, self.interleaved, self.amplitude = freq, interleaved, amplitude

    @property
    def freq(self):
        return self._freq

    @freq.setter
    def freq(self, t):
        if t.shape != (self.rot // 2,):
            raise ValueError(f"freq must have shape {[self.rot // 2]}")
        self._c.freq = _tensor(t, "freq", torch.float64, self.device)
        self._freq = t

    @property
    def interleaved(self):
        return bool(self._c.interleaved)

    @interleaved.setter
    def interleaved(self, v):
        self._c.interleaved = int(bool(v))

    @property
    def amplitude(self):
        return self._amplitude

    @amplitude.setter
    def amplitude(self, v):
        self._c.amplitude = self._amplitude = float(v)

    @classmethod
    def make(cls, rot, base=10000.0, interleaved=False, scaling=None, factor=1.0, trained=None, bounds=(32.0, 1.0), amplitude=None,
             device="cuda"):
        """freq[i] = base^(-2 i / rot), for contexts `factor` times the trained
        ones bent by `scaling`: "linear" (positions divided by factor), "base"
        (base times factor^(rot / (rot - 2)): the slowest pair as with "linear",
        the fastest as it was) or "bands" (YaRN's interpolation by parts: pairs that
        turn more than bounds[0] times over the `trained` positions as they were,
        those that turn less than bounds[1] times divided by factor, a ramp in the
        pair's index between them; amplitude 0.1 ln(factor) + 1 unless given).  The ramp's ends are
        whole numbers, rounded outward and kept to 0 and rot - 1, as models trained with it have them."""
        if rot < 2 or rot % 2:
            raise ValueError("rot must be even")
        if not factor > 0 or not base > 1:
            raise ValueError("need factor > 0 and base > 1")
        e = torch.arange(0, rot, 2, dtype=torch.float64) / rot
        if scaling is None or scaling == "linear":
            freq = base ** -e / (factor if scaling else 1.0)
        elif scaling == "base":
            if rot < 4:
                raise ValueError("\"base\" needs rot >= 4")
            freq = (base * factor ** (rot / (rot - 2))) ** -e
        elif scaling == "bands":
            if not trained or trained <= 0 or not bounds[0] > bounds[1] > 0:
                raise ValueError("\"bands\" needs the trained positions, and bounds[0] > bounds[1] > 0")
            freq = base ** -e
            # the pair (a real number) that turns n times over the trained positions
            low, high = (rot * math.log(trained / (2 * math.pi * n)) / (2 * math.log(base)) for n in bounds)
            low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
            ramp = ((torch.arange(rot // 2, dtype=torch.float64) - low) / max(high - low, 1)).clamp(0, 1)  # (one whole number: a step)
            freq = freq * (1 - ramp) + freq / factor * ramp
            if amplitude is None:
                amplitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
        else:
            raise ValueError("scaling must be None, \"linear\", \"base\" or \"bands\"")
        return cls(freq.to(device), interleaved, 1.0 if amplitude is None else amplitude)


def rope_append(cache, layer, rows, rope, q, k, v, q_out=None, stream=None):
    """Rotate the rows' queries into q_out and write their rotated keys and their
    values into the pages of one layer: q [n_rows, q_heads, dim] (None: keys
    and values alone), k, v [n_rows, heads * dim] (or [.., heads, dim]; all of one
    float type, rows may lie apart, as in the output of a fused projection); rows a RowMap; q_out
    [n_rows, q_heads, dim] fp32 or the cache's type."""
    dev, D = cache.device, cache.dim
    width = cache.heads * D
    pk, lk, n, kind = _float_rows(k, "k", dev, None, width)
    pv, lv, nv, _ = _float_rows(v, "v", dev, k.dtype, width)
    if rows._p[3] is None:
        raise ValueError("rows has no pos and place")
    if n != rows.n_rows or nv != n:
        raise ValueError("k and v must have n_rows rows")
    if rows.device != dev or rope.device != dev:
        raise ValueError(f"rows and rope must be on {dev}")
    pq, lq, heads, po, ko = None, 0, 0, None, _FLOATS[cache.k.dtype]
    if q is not None:
        if q.dim() != 3 or q.shape[2] != D:
            raise ValueError("q must be [n_rows, q_heads, dim]")
        heads = q.shape[1]
        pq, lq, nq, _ = _float_rows(q, "q", dev, k.dtype, heads * D)
        if q_out is None or q_out.shape != q.shape or nq != n:
            raise ValueError("q must have n_rows rows, and q_out its shape")
        if q_out.dtype is not torch.float32 and q_out.dtype is not cache.k.dtype:
            raise TypeError(f"q_out must be torch.float32 or {cache.k.dtype}, got {q_out.dtype}")
        po, ko = _tensor(q_out, "q_out", q_out.dtype, dev), _FLOATS[q_out.dtype]
    _call(_lib.rope_append, dev, stream, cache._ref, layer, rope._ref, pq, lq, heads, pk, lk, pv, lv, kind, n, rows._p[3],
          rows._p[4], po, ko)


# ---------------------------------------------------------------- attention
def prompt_attention_workspace(cache, q_heads, n_rows):
    """A workspace for prompt_attention calls (one for each stream that makes them)."""
    n = ctypes.c_uint64()
    status = _lib.prompt_attention_workspace(cache._ref, q_heads, n_rows, ctypes.byref(n))
    if status:
        from . import SvgError, last_error
        raise SvgError(status, last_error())
    return torch.empty(max(n.value, 1), dtype=torch.uint8, device=cache.device)


def prompt_attention(cache, layer, rows, q, out, workspace, scale=None, stream=None):
    """Causal attention of a step's rows over the cache, in one layer: q
    [n_rows, q_heads, dim] of the cache's type (rows may lie apart), rows a RowMap,
    out of q's shape and type, workspace from prompt_attention_workspace(); scale defaults to
    1 / sqrt(dim).  Rows of no slot are left as they were."""
    dev, D = cache.device, cache.dim
    if q.dim() != 3 or q.shape[2] != D:
        raise ValueError("q must be [n_rows, q_heads, dim]")
    heads = q.shape[1]
    pq, ld, n, _ = _float_rows(q, "q", dev, cache.k.dtype, heads * D)
    if rows.device != dev or rows.n_slots != cache.n_slots:
        raise ValueError("rows must be a RowMap of the cache's device and number of slots")
    if n != rows.n_rows:
        raise ValueError("q must have n_rows rows")
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    key = ("prompt", heads, n > 0)
    need = cache._attn_bytes.get(key)
    if need is None:
        b = ctypes.c_uint64()
        if _lib.prompt_attention_workspace(cache._ref, heads, n, ctypes.byref(b)) == 0:
            need = cache._attn_bytes[key] = b.value
    if need is not None and workspace.numel() * workspace.element_size() < need:
        raise ValueError("workspace is smaller than prompt_attention_workspace(cache, q_heads, n_rows)")
    _call(_lib.prompt_attention, dev, stream, cache._ref, layer, pq, ld, heads, n, rows._p[0], rows._p[1],
          D ** -0.5 if scale is None else scale, _tensor(out, "out", q.dtype, dev), _tensor(workspace, "workspace", torch.uint8, dev))


# ------------------------------------------------------------------ linears
def _linear_args(xq, x_scale, N, y):
    dev = _device(xq, "xq")
    shape = xq.shape
    if len(shape) != 2:
        raise ValueError("xq must be [M, K]")
    M, K = shape
    if x_scale.shape != (M,) or y.shape != (M, N):
        raise ValueError("y must be [M, N] and x_scale [M]")
    kind = _FLOATS.get(y.dtype)
    if kind is None:
        raise TypeError(f"y must be float32, float16 or bfloat16, got {y.dtype}")
    return dev, M, K, _tensor(xq, "xq", torch.int8, dev), _tensor(x_scale, "x_scale", torch.float32, dev), _tensor(y, "y", y.dtype, dev), kind


@functools.lru_cache(maxsize=4096)
def _sizes(N, K, f, group):
    """Values that the weight storage has at least: codes (bytes), scales, zeros (bytes of 4-bit ones, fp16 values)."""
    from . import W4_Z4, weight_sizes
    codes, scales, zeros = weight_sizes(N, K, f, group) if N > 0 else (0, 0, 0)
    return codes, scales // 2, zeros if f == W4_Z4 else zeros // 2


def _large(t, name, dtype, dev, least):
    at = _tensor(t, name, dtype, dev)
    if t.numel() < least:
        raise ValueError(f"{name} is too small: need {least} values")
    return at


def w4a8_prompt_linear(xq, x_scale, wq, w_scale, w_zero, fmt, group, N, y, stream=None):
    """y[M, N] = dequantized (xq . W^T) for any number of rows: xq [M, K] in 32-row
    slab buffers, tiled W4 weights of N rows, y fp32, fp16 or bf16."""
    from . import FORMATS, W4_Z4
    f = FORMATS[fmt] if isinstance(fmt, str) else int(fmt)
    dev, M, K, px, ps, py, kind = _linear_args(xq, x_scale, N, y)
    codes, scales, zeros = _sizes(N, K, f, group)
    if w_zero is None:
        raise ValueError("W4 formats need w_zero")
    _call(_lib.w4a8_prompt_linear, dev, stream, px, ps, M, K, _large(wq, "wq", torch.uint8, dev, codes),
          _large(w_scale, "w_scale", torch.float16, dev, scales),
          _large(w_zero, "w_zero", torch.uint8 if f == W4_Z4 else torch.float16, dev, zeros), f, group, N, py, kind)


def w8a8_prompt_linear(xq, x_scale, wq, w_scale, N, y, stream=None):
    """y[M, N] = dequantized (xq . W^T) for any number of rows: xq [M, K] in 32-row
    slab buffers, tiled W8 weights of N rows, y fp32, fp16 or bf16."""
    dev, M, K, px, ps, py, kind = _linear_args(xq, x_scale, N, y)
    codes, scales, _ = _sizes(N, K, 2, 0)  # (SVG_W8_SYM)
    _call(_lib.w8a8_prompt_linear, dev, stream, px, ps, M, K, _large(wq, "wq", torch.int8, dev, codes),
          _large(w_scale, "w_scale", torch.float16, dev, scales), N, py, kind)


def gated_quant_i8(x, gate, signs, xq, x_scale, block=32, stream=None):
    """x * silu(gate) (x alone without a gate), rotation and int8 quantization in
    one launch: x, gate [M, K] fp32 / fp16 / bf16 (rows may lie apart, as halves of
    one product's); outputs xq (M * K codes, one slab buffer per 32 rows) and x_scale [M]."""
    dev = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    px, lx, _, kind = _float_rows(x, "x", dev, None, K)
    pg, lg = None, 0
    if gate is not None:
        pg, lg, mg, _ = _float_rows(gate, "gate", dev, x.dtype, K)
        if mg != M:
            raise ValueError("gate must have x's shape")
    if signs.numel() != K or xq.numel() != M * K or x_scale.numel() != M:
        raise ValueError("need signs [K], xq of M * K codes and x_scale [M]")
    _call(_lib.gated_quant_i8, dev, stream, px, lx, pg, lg, kind, M, K, _tensor(signs, "signs", torch.int8, dev), block,
          _tensor(xq, "xq", torch.int8, dev), _tensor(x_scale, "x_scale", torch.float32, dev))
