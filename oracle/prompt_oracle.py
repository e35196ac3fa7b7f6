"""A prompt's pass through a decoder layer: the plain CPU oracle, fp64, one row at a
time.

TEST INFRASTRUCTURE.  Only tests/ and __graft_entry__.smoke() may import this
module; the HIP library shares no code with it.

  M1. Packed rows follow one another slot after slot (n_new below 1: none) and end at n_rows; dense ones
      are T a slot, of which min(max(n_new, 0), T) are in use.
  M2. Row i of slot s has position len + i, in a tree len + the depth of node i; its place is position
      len + i's in the pages, if the slot may write there.
  R1. The pair (a, b) becomes (a c - b s, b c + a s), c and s of pos * freq[i] (one fp64 product), times
      the amplitude.
  A1. Row i of slot s attends to the positions 0 .. len + i; softmax of scale q . k.
  G1. u = x * gate / (1 + exp(-gate)) rounded once to fp32, then svg_oracle.quant_acts.
"""
import numpy as np

from . import attention_oracle as AO
from . import cache_oracle as CO
from . import svg_oracle as O


def row_map(c, n_new, T, n_rows, parent=None):
    """(start, count, slot, pos, place)."""
    S = len(c["len"])
    start, count = np.zeros(S, np.int64), np.zeros(S, np.int64)
    slot, pos, place = (np.full(n_rows, -1, np.int64) for _ in range(3))
    at = 0
    for s in range(S):
        n = max(int(n_new[s]), 0)
        if T:
            at, n = s * T, min(n, T)
        start[s], count[s] = at, min(n, n_rows - at)
        for i in range(count[s]):
            r = at + i
            slot[r] = s
            path = AO.root_path(None if parent is None else parent[s], i)
            length = int(c["len"][s])
            if path is None or length < 0 or length + len(path) - 1 > 2 ** 31 - 1:
                continue
            pos[r] = length + len(path) - 1
            page = CO.own_page_of(c, s, length + i)
            if page is not None:
                place[r] = page * c["page"] + (length + i) % c["page"]
        at = min(at + n, n_rows)
    return start, count, slot, pos, place


def pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rope(x, pos, freq, interleaved, amplitude):
    """x [R, heads, dim]: (rotated fp64, the sum of the products' sizes of each value)."""
    a, b = pairs(2 * len(freq), interleaved)
    angle = pos.astype(np.float64)[:, None] * freq
    c, s = (f(angle)[:, None, :] * amplitude for f in (np.cos, np.sin))
    x = x.astype(np.float64)
    y, size = x.copy(), np.zeros_like(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
    size[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, size


def write(c, layer, place, k, v):
    """Rows of patterns [R, H, dim] to their places (those below 0 passed over)."""
    d = np.arange(c["dim"])
    for r in np.flatnonzero(place >= 0):
        p, t = int(place[r]) // c["page"], int(place[r]) % c["page"]
        c["k"][layer, p][:, CO.key_at(t, d, c["dim"])] = k[r]
        c["v"][layer, p][:, CO.value_at(t, d, c["dim"])] = v[r]


def attention(c, wide, layer, q, start, count, scale):
    """q [R, A, dim] -> (out fp64, NaN where the row is not defined; whether a row is some slot's; per row and head the largest
    |scale| sum |q k|, the largest |v| and the mean |v| by weight)."""
    R, A, dim = q.shape
    H = c["k"].shape[2]
    out, mine = np.full((R, A, dim), np.nan), np.zeros(R, bool)
    size = np.zeros((R, A, 3))
    for s in range(len(c["len"])):
        if not 0 <= start[s] < R:
            continue
        n, length = min(int(count[s]), R - int(start[s])), int(c["len"][s])
        if n <= 0:
            continue
        mine[start[s]:start[s] + n] = True
        held = int(c["pages"][s])
        if length < 0 or not 0 <= held <= c["table"].shape[1] or length + n > held * c["page"]:
            continue
        at = np.arange(length + n)
        pg = c["table"][s][at // c["page"]].astype(np.int64)
        fine = (pg >= 0) & (pg < len(c["refs"]))
        fine[fine] &= (at[fine] < length) | (c["refs"][pg[fine]] <= 1)
        seen = int(np.argmin(fine)) if not fine.all() else length + n      # positions before the first bad one
        pg = np.where((pg >= 0) & (pg < len(c["refs"])), pg, 0)
        t, d = (at % c["page"])[:, None], np.arange(dim)[None, :]
        for a in range(A):
            h = a // (A // H)
            K = wide(c["k"][layer, pg, h][np.arange(len(at))[:, None], CO.key_at(t, d, dim)])
            V = wide(c["v"][layer, pg, h][np.arange(len(at))[:, None], CO.value_at(t, d, dim)])
            for i in range(n):
                L = length + i + 1
                if L > seen:
                    break
                x = q[start[s] + i, a].astype(np.float64)
                sc = scale * (K[:L] @ x)
                p = np.exp(sc - sc.max())
                p /= p.sum()
                out[start[s] + i, a] = p @ V[:L]
                size[start[s] + i, a] = (abs(scale) * (np.abs(K[:L]) @ np.abs(x)).max(), np.abs(V[:L]).max(),
                                         (p @ np.abs(V[:L])).max())
    return out, mine, size


def gated(x, gate):
    """fp32 rows."""
    if gate is None:
        return x.astype(np.float32)
    g = gate.astype(np.float64)
    with np.errstate(over="ignore"):
        return (x.astype(np.float64) * (g / (1.0 + np.exp(-g)))).astype(np.float32)


def gated_quant(x, gate, signs, block):
    """(codes [M, K] int8, scales [M])."""
    return O.quant_acts(gated(x, gate), signs, block)
