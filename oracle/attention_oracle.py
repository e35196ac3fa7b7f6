"""Attention of draft trees over a paged cache: the plain CPU oracle, fp64, one
row at a time.

TEST INFRASTRUCTURE.  Only tests/ and __graft_entry__.smoke() may import this
module; the HIP library shares no code with it.

  A1. Node i of slot s reads the positions 0 .. len - 1 and len + j for the nodes
      j on its root path, itself included.
  A2. Query head a reads key/value head a / (q_heads / heads).
  A3. o = sum softmax(scale q . k) v.
A path that is no path to the root, or that meets a node in a page which several
slots hold (no token could be written there), gives a NaN row.
"""
import numpy as np

from . import cache_oracle as CO


def root_path(parent, i):
    """Nodes from the root to i, or None."""
    if parent is None:
        return list(range(i + 1))
    if parent[0] != -1:
        return None
    path = [i]
    while i:
        p = int(parent[i])
        if not 0 <= p < i:
            return None
        path.append(p)
        i = p
    return path[::-1]


def positions(length, parent, i):
    path = root_path(parent, i)
    return None if path is None else list(range(length)) + [length + j for j in path]


def attention(c, wide, layer, q, parent, T, n_nodes, scale):
    """c: the cache's dict (16-bit patterns); wide: patterns -> float64; q [S, T, A, dim];
    parent [S, T] or None.  Returns (out [S, T, A, dim] fp64, NaN where there is
    no row, and the bound below for each (row, head))."""
    S, A, dim = len(c["len"]), q.shape[2], q.shape[3]
    H = c["k"].shape[2]
    G = A // H
    out = np.full((S, T, A, dim), np.nan)
    spread = np.zeros((S, T, A, 2))  # largest sum |q k| scale, largest |v|
    for s in range(S):
        n = T if n_nodes is None else min(max(int(n_nodes[s]), 0), T)
        length = int(c["len"][s])
        if n == 0:
            continue
        at = np.arange(length + n)
        pg = c["table"][s][at // c["page"]]
        t, d = (at % c["page"])[:, None], np.arange(dim)[None, :]
        for h in range(H):
            K = wide(c["k"][layer, pg, h][np.arange(len(at))[:, None], CO.key_at(t, d, dim)])
            V = wide(c["v"][layer, pg, h][np.arange(len(at))[:, None], CO.value_at(t, d, dim)])
            for i in range(n):
                pos = positions(length, None if parent is None else parent[s], i)
                if pos is None or any(CO.own_page_of(c, s, x) is None for x in pos[length:]):
                    continue
                k, v = K[pos], V[pos]
                for a in range(h * G, h * G + G):
                    x = q[s, i, a].astype(np.float64)
                    sc = scale * (k @ x)
                    p = np.exp(sc - sc.max())
                    out[s, i, a] = (p @ v) / p.sum()
                    spread[s, i, a] = abs(scale) * (np.abs(k) @ np.abs(x)).max(), np.abs(v).max()
    return out, spread
