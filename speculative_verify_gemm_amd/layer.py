"""Python binding of include/svgemm_layer.h: the steps of a decoder layer around
the quantized linears.  Argument marshalling only, as in the package's main
module: every function checks devices, dtypes and shapes and calls the C entry
point of the same name on the current stream of the tensors' device (or the
stream given)."""
from __future__ import annotations

import ctypes

import torch

_lib = None  # the library, once the package has loaded it (_bind)
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream

_FP32 = torch.float32
_FLOATS = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _bind(lib):
    global _lib
    _lib = lib
    vp, i, d = ctypes.c_void_p, ctypes.c_int, ctypes.c_double
    lib.add_rmsnorm_quant_i8.argtypes = [vp, i, vp, vp, i, d, i, i, vp, i, vp, vp, vp, vp]
    lib.add_rmsnorm_quant_i8.restype = ctypes.c_int
    kv, i64 = ctypes.POINTER(KVCacheC), ctypes.c_int64
    lib.kv_append.argtypes = [kv, i, vp, i64, vp, i64, i, vp, vp]
    lib.kv_commit.argtypes = [kv, i, vp, vp, vp, vp]
    lib.kv_fork.argtypes = [kv, vp, vp, vp, vp, vp]
    lib.kv_reserve.argtypes = [kv, vp, vp, vp, vp]
    lib.kv_copy_pages.argtypes = [kv, vp, vp, i, vp]
    lib.tree_attention_workspace.argtypes = [kv, i, i, ctypes.POINTER(ctypes.c_uint64)]
    lib.tree_attention.argtypes = [kv, i, vp, i64, i, vp, i, vp, vp, ctypes.c_float, vp, vp, vp]
    for fn in (lib.tree_attention_workspace, lib.tree_attention, lib.kv_append, lib.kv_commit, lib.kv_fork, lib.kv_reserve, lib.kv_copy_pages):
        fn.restype = ctypes.c_int


class KVCacheC(ctypes.Structure):
    """svg_kv_cache (include/svgemm_layer.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v")]
                + [(n, ctypes.c_int) for n in ("type", "heads", "dim", "page", "n_pages", "n_layers", "n_slots", "width")]
                + [(n, ctypes.c_void_p) for n in ("table", "pages", "len", "refs")])


def _bad(t, name, dtype, dev):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _tensor(t, name, dtype, dev):
    """A contiguous tensor of dtype on dev: its address."""
    if t.dtype is dtype and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    _bad(t, name, dtype, dev)


def _float_tensor(t, name, dev):
    """As _tensor, of any of the element types: (address, type number)."""
    dtype = t.dtype
    kind = _FLOATS.get(dtype)
    if kind is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {dtype}")
    return _tensor(t, name, dtype, dev), kind


def _device(t, name):
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")
    return dev


def _call(fn, dev, stream, *args):
    """fn(*args, stream) with dev as the current device."""
    if stream is None:
        stream = _raw_stream(dev.index)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if _current_device() == dev.index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        from . import SvgError, last_error
        raise SvgError(status, last_error())


def add_rmsnorm_quant_i8(x, residual, weight, eps, signs, xq, x_scale, y=None, block=32, stream=None):
    """residual += x (x alone without a residual), root-mean-square norm by
    weight, rotation and int8 quantization in one launch: x [M, K] fp32 / fp16
    / bf16, residual fp32 [M, K] or None, weight [K]; outputs xq (M * K codes,
    one slab buffer per 32 rows), x_scale [M] and, if given, the normalised
    rows y fp32 [M, K]."""
    dev = _device(x, "x")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [M, K]")
    M, K = shape
    px, kx = _float_tensor(x, "x", dev)
    pw, kw = _float_tensor(weight, "weight", dev)
    pr = None if residual is None else _tensor(residual, "residual", torch.float32, dev)
    py = None if y is None else _tensor(y, "y", torch.float32, dev)
    ps = _tensor(signs, "signs", torch.int8, dev)
    pq = _tensor(xq, "xq", torch.int8, dev)
    pc = _tensor(x_scale, "x_scale", torch.float32, dev)
    if ((residual is not None and residual.shape != shape) or (y is not None and y.shape != shape)
            or weight.numel() != K or signs.numel() != K or xq.numel() != M * K or x_scale.numel() != M):
        raise ValueError("need residual and y [M, K], weight and signs [K], xq of M * K codes and x_scale [M]")
    _call(_lib.add_rmsnorm_quant_i8, dev, stream, px, kx, pr, pw, kw, eps, M, K, ps, block, py, pq, pc)


# ------------------------------------------------------------------ the cache
class KVCache:
    """A paged key/value cache and the slots that use it (svg_kv_cache of
    include/svgemm_layer.h): k, v fp16 or bf16 [n_layers, n_pages, heads, page *
    dim]; table int32 [n_slots, width], pages and len [n_slots], refs [n_pages]
    (without them only kv_copy_pages takes the cache).  The object keeps the
    tensors; their contents are read by the calls on the device only.  k, v and
    the tables may be set to other tensors of the same shape, type and device
    (calls that a graph has captured go on with the ones they were made with)."""

    def __init__(self, k, v, table=None, pages=None, len=None, refs=None, *, dim, page):
        dev = _device(k, "k")
        if k.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError(f"k must be float16 or bfloat16, got {k.dtype}")
        if k.dim() != 4 or k.shape != v.shape or k.shape[3] != page * dim:
            raise ValueError("k and v must be [n_layers, n_pages, heads, page * dim]")
        L, P, H, _ = k.shape
        c = KVCacheC(_tensor(k, "k", k.dtype, dev), _tensor(v, "v", k.dtype, dev), _FLOATS[k.dtype], H, dim, page, P, L)
        if table is not None:
            if table.dim() != 2:
                raise ValueError("table must be [n_slots, width]")
            S, c.width = table.shape
            c.n_slots = S
            c.table = _tensor(table, "table", torch.int32, dev)
            for name, t, n in (("pages", pages, S), ("len", len, S), ("refs", refs, P)):
                if t is None or t.shape != (n,):
                    raise ValueError(f"{name} must have shape [{n}]")
                setattr(c, name, _tensor(t, name, torch.int32, dev))
        self._t = dict(k=k, v=v, table=table, pages=pages, len=len, refs=refs)
        self.dim, self.page, self.heads, self.device = dim, page, H, dev
        self.n_layers, self.n_pages = L, P
        self.n_slots, self.width = c.n_slots, c.width
        self._c = c
        self._ref = ctypes.byref(c)
        self._attn_bytes = {}  # workspace sizes by (q_heads, T)

    def _set(self, name, t):
        now = self._t[name]
        if now is None:
            raise ValueError(f"the cache has no {name}")
        if t is None or t.shape != now.shape:
            raise ValueError(f"{name} must have shape {list(now.shape)}")
        setattr(self._c, name, _tensor(t, name, now.dtype, self.device))
        self._t[name] = t

    @classmethod
    def empty(cls, n_layers, n_pages, heads, dim, page, n_slots, width, dtype=torch.float16, device="cuda"):
        """A cache of free pages and empty slots (the pages' contents are not set)."""
        shape = (n_layers, n_pages, heads, page * dim)
        zeros = lambda n: torch.zeros(n, dtype=torch.int32, device=device)  # noqa: E731
        return cls(torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device),
                   torch.full((n_slots, width), -1, dtype=torch.int32, device=device), zeros(n_slots), zeros(n_slots),
                   zeros(n_pages), dim=dim, page=page)

    def other_tables(self):
        """The same pages and counts with tables of their own (empty slots): what kv_fork writes to."""
        return KVCache(self.k, self.v, torch.full_like(self.table, -1), torch.zeros_like(self.pages),
                       torch.zeros_like(self.len), self.refs, dim=self.dim, page=self.page)


for _name in ("k", "v", "table", "pages", "len", "refs"):
    setattr(KVCache, _name, property(lambda self, n=_name: self._t[n], lambda self, t, n=_name: self._set(n, t)))


def _rows(t, name, cache, width):
    """fp32 rows [n, ...] of `width` values each, a row contiguous: (address, row stride, n)."""
    if t.dtype is not _FP32:
        raise TypeError(f"{name} must be torch.float32, got {t.dtype}")
    if t.device != cache.device:
        raise ValueError(f"{name} must be on {cache.device}, got {t.device}")
    shape, stride = t.shape, t.stride()  # (each look at a tensor costs as much as the rest of the check)
    if len(shape) == 3:
        ok = shape[1] * shape[2] == width and stride[2] == 1 and (stride[1] == shape[2] or shape[1] == 1)
    else:
        ok = len(shape) == 2 and shape[1] == width and stride[1] == 1
    if not ok:
        raise ValueError(f"{name} must be [n, {width}] or [n, heads, dim] with contiguous rows")
    n = shape[0]
    return t.data_ptr(), (stride[0] if n > 1 else width), n


def _slots(t, name, cache, *more):
    """An int32 tensor of one entry (or a row of `more`) for each slot."""
    if t.shape != (cache.n_slots, *more):
        raise ValueError(f"{name} must have shape {[cache.n_slots, *more]}")
    return _tensor(t, name, torch.int32, cache.device)


def kv_append(cache, layer, k, v, T, n_rows=None, stream=None):
    """Write T new tokens of each slot behind its committed ones, in one layer:
    k, v fp32 [n_slots * T, heads * dim] (or [.., heads, dim]; rows may lie apart,
    as in the output of a fused projection); n_rows int32 [n_slots]: fewer of them.
    Rows without a page, or in one that other slots hold too, are passed over."""
    pk, lk, nk = _rows(k, "k", cache, cache.heads * cache.dim)
    pv, lv, nv = _rows(v, "v", cache, cache.heads * cache.dim)
    if nk != cache.n_slots * T or nv != nk:
        raise ValueError("k and v must have n_slots * T rows")
    pn = None if n_rows is None else _slots(n_rows, "n_rows", cache)
    _call(_lib.kv_append, cache.device, stream, cache._ref, layer, pk, lk, pv, lv, T, pn)


def kv_commit(cache, path, n_emit, len_out=None, stream=None):
    """Move the accepted path of each slot's tree behind its root, in every
    layer: path int32 [n_slots, T] and n_emit [n_slots] as tree_accept_greedy
    writes them; the new lengths go to len_out (None: into the cache's own). A
    slot whose path has no pages of its own keeps its tokens and length."""
    if path.dim() != 2:
        raise ValueError("path must be [n_slots, T]")
    T = path.shape[1]
    out = cache.len if len_out is None else len_out
    _call(_lib.kv_commit, cache.device, stream, cache._ref, T, _slots(path, "path", cache, T),
          _slots(n_emit, "n_emit", cache), _slots(out, "len_out", cache))


def kv_fork(cache, src, out, stream=None):
    """Every slot s of `out` (a KVCache over the same pages and counts, with
    tables of its own: cache.other_tables()) becomes a fork of slot src[s] of
    `cache`, keeps it (src[s] == s) or is freed (-1).  Afterwards `cache`'s tables are spent."""
    if out.k.data_ptr() != cache.k.data_ptr() or out.refs.data_ptr() != cache.refs.data_ptr():
        raise ValueError("out must be a cache over the same pages and counts")
    if out.table.shape != cache.table.shape:
        raise ValueError("out needs tables of the same shape")
    _call(_lib.kv_fork, cache.device, stream, cache._ref, _slots(src, "src", cache), out._c.table, out._c.pages,
          out._c.len)


def kv_workspace(cache):
    """A workspace for kv_reserve."""
    return torch.empty(2 * cache.n_slots + 4, dtype=torch.int32, device=cache.device)


def kv_reserve(cache, need, status, workspace, stream=None):
    """Room for need[s] more tokens of each slot, in pages of its own; status
    int32 [n_slots]: 0 done, 1 not enough free pages, 2 does not fit the table. A
    slot with 1 or 2 is left as it was and takes no part in a step until it has room."""
    pw = _tensor(workspace, "workspace", torch.int32, cache.device)
    if workspace.numel() < 2 * cache.n_slots + 4:
        raise ValueError("workspace is smaller than kv_workspace(cache)")
    _call(_lib.kv_reserve, cache.device, stream, cache._ref, _slots(need, "need", cache),
          _slots(status, "status", cache), pw)


def kv_copy_pages(cache, src, dst, stream=None):
    """Copy pages src (int32 [n]) to pages dst in every layer."""
    if src.dim() != 1 or src.shape != dst.shape:
        raise ValueError("src and dst must be [n]")
    _call(_lib.kv_copy_pages, cache.device, stream, cache._ref, _tensor(src, "src", torch.int32, cache.device),
          _tensor(dst, "dst", torch.int32, cache.device), src.shape[0])


# -------------------------------------------------------------- attention
def tree_attention_workspace(cache, q_heads, T):
    """A workspace for tree_attention calls of these sizes (one for each stream that makes them)."""
    n = ctypes.c_uint64()
    status = _lib.tree_attention_workspace(cache._ref, q_heads, T, ctypes.byref(n))
    if status:
        from . import SvgError, last_error
        raise SvgError(status, last_error())
    return torch.empty(max(n.value, 1), dtype=torch.uint8, device=cache.device)


def tree_attention(cache, layer, q, parent, out, workspace, scale=None, n_nodes=None, shared=None, stream=None):
    """Attention of every slot's draft tree over the cache, in one layer: q fp32
    [n_slots * T, q_heads, dim] (rows may lie apart, as in the output of a fused
    projection), parent int32 [n_slots, T] (None: chains; T is then q's rows per
    slot), out fp32 of q's shape, workspace from tree_attention_workspace();
    scale defaults to 1 / sqrt(dim); n_nodes int32 [n_slots]: nodes of each tree;
    shared int32 [1]: leading tokens that are the same pages in every slot. Nodes
    without a place of their own in the cache give NaN rows."""
    S, D = cache.n_slots, cache.dim
    heads = q.shape[1] if q.dim() == 3 else q.shape[-1] // D
    pq, ld, n = _rows(q, "q", cache, heads * D)
    T = n // S if S else (1 if parent is None or parent.dim() < 2 else parent.shape[1])  # (no slots: an empty call)
    if n != S * T:
        raise ValueError("q must have n_slots * T rows")
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    need = cache._attn_bytes.get((heads, T))
    if need is None:
        b = ctypes.c_uint64()
        if _lib.tree_attention_workspace(cache._ref, heads, T, ctypes.byref(b)) == 0:
            need = cache._attn_bytes[(heads, T)] = b.value
    if need is not None and workspace.numel() * workspace.element_size() < need:
        raise ValueError("workspace is smaller than tree_attention_workspace(cache, q_heads, T)")
    pp = None if parent is None else _slots(parent, "parent", cache, T)
    pn = None if n_nodes is None else _slots(n_nodes, "n_nodes", cache)
    if shared is not None and shared.numel() < 1:
        raise ValueError("shared needs 1 element")
    ps = None if shared is None else _tensor(shared, "shared", torch.int32, cache.device)
    _call(_lib.tree_attention, cache.device, stream, cache._ref, layer, pq, ld, heads, pp, T, pn, ps,
          D ** -0.5 if scale is None else scale, _tensor(out, "out", torch.float32, cache.device),
          _tensor(workspace, "workspace", torch.uint8, cache.device))
