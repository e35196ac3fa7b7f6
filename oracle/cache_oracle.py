"""The paged key/value cache: the plain CPU oracle, one slot and one value at a
time, on numpy arrays.

TEST INFRASTRUCTURE.  Only tests/ and __graft_entry__.smoke() may import this
module; the HIP library shares no code with it.

A cache is a dict: k, v [L, P, H, page * dim] (any 16-bit type), table [S, W],
pages [S], len [S], refs [P] (int), dim, page.

  P1. A page is free where refs is 0; a page taken is the lowest free one.
  P2. reserve serves the slots in order: a slot gets all it asks for or nothing.
      Its partly filled last page is replaced by a copy if more than one slot
      holds it at that moment; then pages are added.
  P3. fork: slot s holds the pages of slot src[s]'s committed tokens; all slots
      change at once.
  P4. commit: node path[j]'s token moves to position len + 1 + j.
  P5. a page that several slots hold is not written: append passes over its rows,
      commit keeps a slot with a position of its path there.
"""
import numpy as np


def key_at(t, d, dim):
    return ((t // 16) * (dim // 32) + d // 32) * 512 + (16 * ((d % 32) // 8) + t % 16) * 8 + d % 8


def value_at(t, d, dim):
    return (((t // 32) * (dim // 16) + d // 16) * 512 + (16 * ((t % 16) // 4) + d % 16) * 8
            + 4 * ((t % 32) // 16) + t % 4)


def page_of(c, s, pos):
    """The page that holds position pos of slot s, or None."""
    i = pos // c["page"]
    if pos < 0 or not 0 <= c["pages"][s] <= c["table"].shape[1] or i >= c["pages"][s]:
        return None
    p = int(c["table"][s, i])
    return p if 0 <= p < c["refs"].shape[0] else None


def own_page_of(c, s, pos):
    """The same, None also where another slot holds the page."""
    p = page_of(c, s, pos)
    return None if p is None or c["refs"][p] > 1 else p


def token(c, layer, s, pos):
    """(key [H, dim], value [H, dim]) of one position."""
    p, t, d = page_of(c, s, pos), pos % c["page"], np.arange(c["dim"])
    return c["k"][layer, p][:, key_at(t, d, c["dim"])], c["v"][layer, p][:, value_at(t, d, c["dim"])]


def put(c, layer, s, pos, key, value):
    p, t, d = page_of(c, s, pos), pos % c["page"], np.arange(c["dim"])
    c["k"][layer, p][:, key_at(t, d, c["dim"])] = key
    c["v"][layer, p][:, value_at(t, d, c["dim"])] = value


def append(c, layer, k, v, T, n_rows=None):
    """k, v [S, T, H, dim], in the cache's type already."""
    for s in range(len(c["len"])):
        n = T if n_rows is None else min(max(int(n_rows[s]), 0), T)
        for i in range(n):
            pos = int(c["len"][s]) + i
            if c["len"][s] >= 0 and own_page_of(c, s, pos) is not None:
                put(c, layer, s, pos, k[s, i], v[s, i])


def commit(c, path, n_emit):
    """Moves the tokens; returns the new lengths."""
    new = c["len"].copy()
    T = path.shape[1]
    for s in range(len(new)):
        n, base = int(n_emit[s]), int(c["len"][s])
        if not 1 <= n <= T:
            continue
        p = [0] + [int(x) for x in path[s, :n - 1]]
        if any(b <= a or b >= T for a, b in zip(p, p[1:])):
            continue
        if base < 0 or own_page_of(c, s, base) is None or own_page_of(c, s, base + p[-1]) is None:
            continue
        for layer in range(c["k"].shape[0]):
            rows = [tuple(np.array(x) for x in token(c, layer, s, base + x)) for x in p[1:]]
            for j, (key, value) in enumerate(rows):
                put(c, layer, s, base + 1 + j, key, value)
        new[s] = base + n
    return new


def fork(c, src):
    """The cache after the fork: new tables; refs is updated in place."""
    S, W = c["table"].shape
    out = dict(c, table=np.full_like(c["table"], -1), pages=np.zeros_like(c["pages"]), len=np.zeros_like(c["len"]))
    for s in range(S):
        f = int(src[s])
        if not -1 <= f < S:
            f = s
        if f < 0:
            held = []
        elif f == s:
            held = c["table"][s, :c["pages"][s]].tolist()
        else:
            held = c["table"][f, :min(-(-int(c["len"][f]) // c["page"]), int(c["pages"][f]))].tolist()
        if f >= 0:
            out["len"][s] = c["len"][f]
        out["pages"][s] = len(held)
        out["table"][s, :len(held)] = held
        if f != s:
            for p in held:
                c["refs"][p] += 1
            for p in c["table"][s, :c["pages"][s]]:
                c["refs"][p] -= 1
    return out


def reserve(c, need):
    """Makes room in place; returns the status of each slot."""
    S, W = c["table"].shape
    PS, P = c["page"], c["refs"].shape[0]
    status = np.zeros(S, np.int32)
    # pages given back by a copy in this call are not taken again in it (their count stays above 0)
    for s in range(S):
        if need[s] < 1:
            continue
        n, held = int(c["len"][s]), int(c["pages"][s])
        total = -(-(n + int(need[s])) // PS)
        if n < 0 or not 0 <= held <= W or n > held * PS or total > W:
            status[s] = 2
            continue
        part = int(c["table"][s, n // PS]) if n % PS else None
        if part is not None and not 0 <= part < P:
            status[s] = 2
            continue
        copy = part is not None and c["refs"][part] > 1
        want = max(total - held, 0) + copy
        free = np.flatnonzero(c["refs"] == 0)
        if want > len(free):
            status[s] = 1
            continue
        taken = [int(x) for x in free[:want]]
        for p in taken:
            c["refs"][p] = 1
        if copy:
            p = taken.pop(0)
            c["refs"][part] -= 1
            c["table"][s, n // PS] = p
            c["k"][:, p] = c["k"][:, part]
            c["v"][:, p] = c["v"][:, part]
        c["table"][s, held:held + len(taken)] = taken
        c["pages"][s] = held + len(taken)
    return status


def copy_pages(c, src, dst):
    P = c["k"].shape[1]
    for a, b in zip(src, dst):
        if 0 <= a < P and 0 <= b < P:
            c["k"][:, b] = c["k"][:, a]
            c["v"][:, b] = c["v"][:, a]


def holders(c):
    """Slots that hold each page (what refs has to say)."""
    n = np.zeros(c["refs"].shape[0], np.int64)
    for s in range(c["table"].shape[0]):
        for p in c["table"][s, :c["pages"][s]]:
            n[p] += 1
    return n
