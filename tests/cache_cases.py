"""Shared plumbing of the cache tests: a cache of seeded contents as the oracle's
dict (16-bit patterns) and as the library's object."""
import numpy as np
import torch

from oracle import cache_oracle as CO

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def bits(t):
    """A 16-bit tensor's patterns on the host."""
    return t.contiguous().view(torch.int16).cpu().numpy().copy()


def make(seed, lens, room, L=1, H=2, dim=64, page=32, spare=4, shuffle=True, width=None):
    """Slots of the given lengths with `room` tokens of space behind them."""
    rng = np.random.default_rng(seed)
    held = [-(-(n + room) // page) for n in lens]
    P = sum(held) + spare
    W = width or max(held + [1]) + 2
    ids = rng.permutation(P) if shuffle else np.arange(P)
    table = np.full((len(lens), W), -1, np.int32)
    at = 0
    for s, h in enumerate(held):
        table[s, :h] = ids[at:at + h]
        at += h
    refs = np.zeros(P, np.int32)
    refs[ids[:at]] = 1
    shape = (L, P, H, page * dim)
    # normal 16-bit numbers of either type (exponent bits away from the ends)
    word = lambda: (rng.integers(0x3000, 0x4000, shape) | (rng.integers(0, 2, shape) << 15)).astype(np.uint16).view(np.int16)  # noqa: E731
    return dict(k=word(), v=word(), table=table, pages=np.array(held, np.int32), len=np.array(lens, np.int32), refs=refs,
                dim=dim, page=page)


def copy_of(c):
    return {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in c.items()}


def to_library(svg, c, kind="fp16", dev="cuda"):
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    return svg.KVCache(t(c["k"]).view(TYPES[kind]), t(c["v"]).view(TYPES[kind]), t(c["table"]), t(c["pages"]), t(c["len"]),
                       t(c["refs"]), dim=c["dim"], page=c["page"])


def same(cache, c, what=("k", "v", "table", "pages", "len", "refs")):
    torch.cuda.synchronize()
    for name in what:
        t = getattr(cache, name)
        got = bits(t) if name in ("k", "v") else t.cpu().numpy()
        assert np.array_equal(got, c[name]), name
