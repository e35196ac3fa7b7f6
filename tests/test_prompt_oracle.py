"""The oracle of a prompt's pass against definitions written another way, and the
frequencies of Rope.make (CPU)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache_oracle as CO
from oracle import prompt_oracle as PO
import cache_cases as K


def test_row_map_by_hand():
    c = K.make(3, [5, 40, 31, 7], 0, page=32, spare=9, width=4, shuffle=False)
    c["pages"][:] = [1, 2, 1, 1]
    start, count, slot, pos, place = PO.row_map(c, [3, -2, 4, 2], 0, 8)
    assert list(start) == [0, 3, 3, 7] and list(count) == [3, 0, 4, 1]
    assert list(slot) == [0, 0, 0, 2, 2, 2, 2, 3] and list(pos) == [5, 6, 7, 31, 32, 33, 34, 7]
    p0, p2, p3 = c["table"][0, 0], c["table"][2, 0], c["table"][3, 0]
    assert list(place) == [p0 * 32 + 5, p0 * 32 + 6, p0 * 32 + 7, p2 * 32 + 31, -1, -1, -1, p3 * 32 + 7]
    parent = np.array([[-1, 0, 0, 1], [0, 0, 1, 2], [-1, 0, 5, 2], [-1, 0, 1, 2]])
    start, count, slot, pos, place = PO.row_map(c, [4, 9, 4, 1], 4, 16, parent)
    assert list(start) == [0, 4, 8, 12] and list(count) == [4, 4, 4, 1]
    assert list(pos[:4]) == [5, 6, 6, 7] and list(place[:4]) == [p0 * 32 + 5 + i for i in range(4)]
    assert list(pos[4:8]) == [-1] * 4 and list(pos[8:12]) == [31, 32, -1, -1] and list(pos[12:]) == [7, -1, -1, -1]
    assert list(slot[12:]) == [3, -1, -1, -1]


def test_rope_turns_pairs():
    freq, pos = np.array([1.0, 0.25]), np.array([3, 100001])
    x = np.random.default_rng(0).standard_normal((2, 3, 6))
    for interleaved in (False, True):
        y, size = PO.rope(x, pos, freq, interleaved, 1.0)
        a, b = PO.pairs(4, interleaved)
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[:, None, None] * freq)
        assert np.allclose(y[..., a], z.real, atol=1e-12) and np.allclose(y[..., b], z.imag, atol=1e-12)
        assert np.array_equal(y[..., 4:], x[..., 4:]) and np.all(size[..., :4] >= np.abs(y[..., :4]) - 1e-12)


def test_attention_is_softmax():
    c = K.make(1, [3, 0], 4, H=1, dim=64, page=32)
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 7, 64)).astype(np.float16)
    for s, n in ((0, 7), (1, 4)):
        for t in range(n):
            CO.put(c, 0, s, t, k[t].view(np.int16)[None], v[t].view(np.int16)[None])
    q = rng.standard_normal((6, 2, 64)).astype(np.float16)
    wide = lambda a: np.ascontiguousarray(a).view(np.float16).astype(np.float64)  # noqa: E731
    out, mine, size = PO.attention(c, wide, 0, q, [0, 4], [4, 1], 0.125)
    assert list(mine) == [True] * 5 + [False]
    for r, L in ((0, 4), (3, 7), (4, 1)):
        p = np.exp(0.125 * k[:L].astype(np.float64) @ q[r, 1].astype(np.float64))
        assert np.allclose(out[r, 1], p @ v[:L].astype(np.float64) / p.sum(), atol=1e-12)
    assert np.isnan(out[5]).all()
    c["refs"][c["table"][0, 0]] = 2      # its own positions in a page that others hold too
    assert np.isnan(PO.attention(c, wide, 0, q, [0, 4], [4, 1], 0.125)[0][:4]).all()
    c["refs"][c["table"][0, 0]] = 1
    c["pages"][1] = 0
    out = PO.attention(c, wide, 0, q, [0, 4], [4, 1], 0.125)[0]
    assert np.isnan(out[4]).all() and not np.isnan(out[:4]).any()


def test_gated_rows():
    x, g = np.array([[2.0, -1.0, 3.0, 1.0]], np.float32), np.array([[0.0, 1.0, -800.0, 90.0]], np.float32)
    want = [0.0, -1.0 / (1 + math.exp(-1.0)), 0.0, 90.0]
    assert np.array_equal(PO.gated(x, g), np.array([want], np.float32))
    assert np.array_equal(PO.gated(x, None), x)


class _Host:
    """Rope.make's frequencies without a device."""

    def __init__(self, freq, interleaved=False, amplitude=1.0):
        self.freq, self.amplitude = freq, amplitude


def test_rope_frequencies():
    import speculative_verify_gemm_amd as svg
    make = lambda *a, **k: svg.Rope.make.__func__(_Host, *a, device="cpu", **k)  # noqa: E731
    plain = make(64).freq
    assert plain.dtype == torch.float64 and plain.shape == (32,) and plain[0] == 1 and math.isclose(plain[16], 10000.0 ** -0.5)
    assert torch.allclose(make(64, scaling="linear", factor=4.0).freq, plain / 4)
    base = make(64, scaling="base", factor=8.0).freq
    assert base[0] == 1 and math.isclose(base[-1], plain[-1] / 8, rel_tol=1e-12)
    bands = make(64, scaling="bands", factor=4.0, trained=4096)
    turns = 4096 * plain / (2 * math.pi)
    fast, slow = turns > 64, turns < 0.5
    assert fast.any() and slow.any()
    assert torch.equal(bands.freq[fast], plain[fast]) and torch.allclose(bands.freq[slow], plain[slow] / 4)
    assert bool((bands.freq[1:] < bands.freq[:-1]).all()) and math.isclose(bands.amplitude, 0.1 * math.log(4) + 1)
    for bad in (dict(scaling="bands"), dict(scaling="other"), dict(factor=0.0, scaling="linear"), dict(base=1.0)):
        with pytest.raises(ValueError):
            make(64, **bad)
    with pytest.raises(ValueError):
        make(7)
