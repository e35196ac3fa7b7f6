"""Pins of the oracles of the steps around the linears (CPU): the page layout, the norm, the cache's bookkeeping and
attention, against closed forms and independent formulations; and the binding's checks of its arguments."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import attention_oracle as AO
from oracle import cache_oracle as CO
from oracle import norm_oracle as N


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [32, 64, 128])
def test_page_layout_is_a_bijection_of_16_byte_pieces(dim, page):
    t, d = np.meshgrid(np.arange(page), np.arange(dim), indexing="ij")
    for at in (CO.key_at, CO.value_at):
        x = at(t, d, dim)
        assert np.array_equal(np.sort(x.ravel()), np.arange(page * dim))
    # a lane's eight keys are consecutive values of one token, its eight values two runs of four tokens of one column
    k, v = CO.key_at(t, d, dim), CO.value_at(t, d, dim)
    assert np.array_equal(k[:, 0::8] + 7, k[:, 7::8])
    assert np.array_equal(v[0::4] + 3, v[3::4])
    assert np.array_equal(v[0] + 4, v[16])
    # 16 tokens of 32 values, and 32 tokens of 16, fill one KiB
    assert set((k[:16, :32] // 512).ravel()) == {0} and set((v[:32, :16] // 512).ravel()) == {0}


def test_norm_of_a_constant_row_is_the_weight():
    w = np.arange(1, 65, dtype=np.float32)
    x = np.full((1, 64), 3.0, np.float32)
    assert np.allclose(N.norm_f64(x, None, w, 1e-12)[0], w, rtol=1e-12)
    h, u = N.norm_rows(x, -x / 2, w, 1e-12)
    assert np.array_equal(h, x / 2) and np.allclose(u[0], w, rtol=1e-6)


def test_norm_steps_are_near_the_64_bit_norm():
    rng = np.random.default_rng(1)
    x, r, w = rng.standard_normal((5, 256)), rng.standard_normal((5, 256)) * 30, rng.standard_normal(256)
    x, r, w = (a.astype(np.float32) for a in (x, r, w))
    _h, u = N.norm_rows(x, r, w, 1e-6)
    # one rounding each of the sum (relative to h), r and two products: four half steps of 2^-24, and a little
    ref = N.norm_f64(x, r, w, 1e-6)
    assert np.all(np.abs(u - ref) <= 4.01 * 2.0 ** -24 * np.abs(ref))


def test_slab_codes_of_more_than_32_rows():
    q = np.arange(35 * 64, dtype=np.int64).reshape(35, 64).astype(np.int8)
    s = N.slab_codes(q)
    assert np.array_equal(s[:32], q[0, :32]) and np.array_equal(s[32:64], q[1, :32])
    assert np.array_equal(s[32 * 64:32 * 64 + 32], q[32, :32]) and np.array_equal(s[32 * 64 + 3 * 32:32 * 64 + 4 * 32], q[32, 32:])


def cache(lens, room, dim=64, page=32, spare=6, seed=0):
    from cache_cases import make
    return make(seed, lens, room, H=1, dim=dim, page=page, spare=spare)


def test_counts_stay_the_holders_through_random_steps():
    """Forks, frees, growth and shortages: refs is the number of holders, no slot's writable page is held by another,
    and tokens keep their contents."""
    rng = np.random.default_rng(3)
    c = cache([20, 50, 3, 32], 0, spare=5)
    seen = set()
    for _ in range(40):
        before = [[CO.token(c, 0, s, p)[0].copy() for p in range(int(c["len"][s]))] for s in range(4)]
        src = [int(x) for x in np.where(rng.random(4) < 0.5, np.arange(4), rng.integers(-1, 4, 4))]
        c = CO.fork(c, src)
        assert np.array_equal(CO.holders(c), c["refs"])
        need = rng.integers(0, 40, 4)
        st = CO.reserve(c, need)
        seen |= set(st.tolist())
        assert np.array_equal(CO.holders(c), c["refs"])
        for s in range(4):
            old = before[src[s]] if src[s] >= 0 else []
            for p, key in enumerate(old):
                assert np.array_equal(CO.token(c, 0, s, p)[0], key)
            if st[s] == 0 and need[s] > 0:
                for p in range(int(c["len"][s]), int(c["len"][s]) + int(need[s])):
                    assert c["refs"][CO.page_of(c, s, p)] == 1
                    CO.put(c, 0, s, p, rng.integers(-99, 99, 64), rng.integers(-99, 99, 64))
                c["len"][s] += int(need[s])
        for s in range(4):               # now and then a slot has grown enough
            if c["len"][s] > 70:
                c = CO.fork(c, [x if x != s else -1 for x in range(4)])
    assert seen >= {0, 1}


def test_commit_by_hand():
    c = cache([30], 8, dim=64)
    rows = {p: tuple(x.copy() for x in CO.token(c, 0, 0, p)) for p in range(38)}
    new = CO.commit(c, np.array([[2, 5, 7, -1, -1, -1, -1, -1]]), [4])
    assert list(new) == [34]
    for at, was in ((29, 29), (30, 30), (31, 32), (32, 35), (33, 37), (34, 34)):
        assert all(np.array_equal(a, b) for a, b in zip(CO.token(c, 0, 0, at), rows[was]))


def test_attention_of_a_chain_is_causal_attention():
    """Against torch's softmax over a causal mask."""
    rng = np.random.default_rng(4)
    c = cache([11], 6)
    q = rng.standard_normal((1, 6, 3, 64))
    as_value = lambda a: a.astype(np.float64) / 9000  # noqa: E731
    out, _ = AO.attention(c, as_value, 0, q, None, 6, None, 0.125)
    k = np.stack([as_value(CO.token(c, 0, 0, p)[0][0]) for p in range(17)])
    v = np.stack([as_value(CO.token(c, 0, 0, p)[1][0]) for p in range(17)])
    sc = torch.from_numpy(np.einsum("iad,td->ait", q[0], k) * 0.125)
    mask = torch.tril(torch.ones(6, 17, dtype=torch.bool), diagonal=11)
    p = torch.softmax(sc.masked_fill(~mask, -float("inf")), -1).numpy()
    assert np.allclose(out[0], np.einsum("ait,td->iad", p, v), rtol=1e-12, atol=1e-12)


def test_a_tree_row_is_the_chain_of_its_root_path():
    rng = np.random.default_rng(5)
    c = cache([9], 5)
    q = rng.standard_normal((1, 5, 1, 64))
    wide = lambda a: a.astype(np.float64) / 9000  # noqa: E731
    parent = np.array([[-1, 0, 0, 2, 1]])
    out, _ = AO.attention(c, wide, 0, q, parent, 5, None, 0.2)
    for i, path in ((3, [0, 2, 3]), (4, [0, 1, 4])):
        d = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in c.items()}
        for j, n in enumerate(path):
            CO.put(d, 0, 0, 9 + j, *(x.copy() for x in CO.token(c, 0, 0, 9 + n)))
        one, _ = AO.attention(d, wide, 0, np.repeat(q[:, i:i + 1], 3, 1), None, 3, None, 0.2)
        assert np.allclose(one[0, 2], out[0, i], rtol=1e-12, atol=1e-12)
    assert AO.root_path(np.array([-1, 0, 5]), 2) is None and AO.root_path(np.array([0, 0]), 1) is None


def test_binding_refuses_tensors_of_the_host():
    import speculative_verify_gemm_amd as svg
    f = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="device tensor"):
        svg.add_rmsnorm_quant_i8(f, None, f[0], 1e-6, f[0].to(torch.int8), f.to(torch.int8), f[:, 0])
    k = torch.zeros((1, 4, 2, 32 * 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="device tensor"):
        svg.KVCache(k, k, dim=64, page=32)
