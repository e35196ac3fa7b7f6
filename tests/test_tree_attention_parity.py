"""tree_attention against the fp64 oracle (oracle/attention_oracle.py).

Tolerance, from the number formats.  Write u for half a step of the cache's type
(fp16 2^-11, bf16 2^-8).  A score is a sum of products of exact 16-bit keys with q
in parts that leave u^2 (fp16, two parts) or u^3 (bf16, three) of it, added up in
fp32 by at most dim additions and rounded a few times more: with
B = scale * sum |q k| it is off by at most e = B * (u_q + (dim + 8) 2^-24).  A probability is then
off by e relative (and 2^-20 for the exponential, its argument and the lift), plus u^2 for its two
parts; numerator and denominator are both off by that, each at most max |v| (or 1) times it, and the
fp32 sums over the tiles add (tiles + 64) 2^-24 each.  So
  |out - exact| <= max|v| * 2 * (e + 2^-20 + u^2 + (tiles + 64) 2^-24)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import attention_oracle as AO
from oracle import cache_oracle as CO

pytestmark = pytest.mark.gpu

U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    global C, K, svg
    import svg_cases as C  # noqa: F401
    import cache_cases as K  # noqa: F401
    import speculative_verify_gemm_amd as svg


def wide(kind):
    return lambda a: torch.from_numpy(np.ascontiguousarray(a)).view(K.TYPES[kind]).double().numpy()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=C.DEV)


def trees(rng, S, T):
    """Random trees, the first one a chain."""
    parent = np.full((S, T), -1, np.int32)
    for s in range(S):
        for i in range(1, T):
            parent[s, i] = i - 1 if s == 0 else rng.integers(0, i)
    return parent


def fill(c, rng, kind, spread=1.0):
    """Ordinary keys and values over the whole pool."""
    for name in ("k", "v"):
        x = torch.from_numpy(rng.standard_normal(c[name].shape).astype(np.float32) * np.float32(spread))
        c[name] = K.bits(x.to(K.TYPES[kind]))


def queries(rng, S, T, A, dim, size=1.0):
    """Rows as slices of a wider matrix (numpy [S, T, A, dim], device view)."""
    rows = rng.standard_normal((S * T, (A + 2) * dim)).astype(np.float32) * np.float32(size)
    rows[:, :A * dim] *= np.repeat(np.linspace(0.3, 3.0, A), dim).astype(np.float32)
    d = C.to_dev(rows)
    return rows[:, :A * dim].reshape(S, T, A, dim), d[:, :A * dim].unflatten(1, (A, dim))


def bound(c, kind, spread, most):
    u, dim = U[kind], c["dim"]
    uq = u ** 2 if kind == "fp16" else u ** 3
    e = spread[..., 0] * (uq + (dim + 8) * 2.0 ** -24)
    return spread[..., 1] * 2 * (e + 2.0 ** -20 + u ** 2 + (most / 32 + 64) * 2.0 ** -24)


def close(got, ref, tol):
    """Every row within its bound; a row that has no exact value is NaN."""
    bad = np.isnan(ref)
    assert np.array_equal(np.isnan(got), bad)
    err = np.where(bad, 0, np.abs(got - np.where(bad, 0, ref))).max(-1)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())


def run(cache, q, parent, T, n_nodes=None, shared=None, scale=None, layer=0, workspace=None):
    S, A = cache.n_slots, q.shape[1]
    guard = 256
    buf = torch.full((S * T * A * cache.dim + 2 * guard,), 7.0, device=C.DEV)
    out = buf[guard:-guard].view(S * T, A, cache.dim)
    ws = workspace if workspace is not None else svg.tree_attention_workspace(cache, A, T).fill_(0xFF)
    svg.tree_attention(cache, layer, q, None if parent is None else i32(parent), out, ws, scale=scale,
                       n_nodes=None if n_nodes is None else i32(n_nodes), shared=None if shared is None else i32([shared]))
    assert bool((buf[:guard] == 7).all()) and bool((buf[-guard:] == 7).all())
    return C.host(out).reshape(S, T, A, cache.dim).astype(np.float64)


CASES = [  # lens, T, H, G, dim, page, kind
    ([0], 1, 1, 1, 64, 32, "fp16"), ([1], 1, 2, 4, 128, 64, "bf16"), ([31], 2, 1, 3, 64, 32, "bf16"),
    ([32], 1, 1, 8, 256, 32, "fp16"), ([33], 16, 2, 1, 128, 32, "fp16"), ([1000], 1, 8, 4, 128, 64, "fp16"),
    ([257], 32, 2, 4, 128, 128, "bf16"), ([2049], 32, 1, 8, 64, 64, "fp16"), ([700], 7, 2, 8, 256, 32, "bf16"),
    ([5, 0, 64, 333], 3, 2, 2, 128, 64, "bf16"), ([100] * 9, 1, 1, 5, 64, 32, "fp16"), ([63, 65, 64], 32, 1, 2, 256, 64, "fp16"),
    ([4100, 3, 900], 5, 3, 7, 128, 128, "fp16"), ([40], 17, 1, 16, 128, 32, "bf16"), ([90, 20], 32, 2, 12, 64, 32, "bf16"),
    ([300] * 40, 2, 4, 1, 64, 32, "fp16"), ([513, 31], 8, 2, 4, 128, 64, "fp16"), ([100, 1], 5, 2, 4, 64, 32, "bf16"),
    ([1290], 4, 3, 8, 128, 32, "bf16"), ([(7 * s) % 90 for s in range(300)], 2, 1, 2, 64, 32, "bf16"), ([3] * 1024, 1, 1, 1, 64, 32, "fp16"),
]


@pytest.mark.parametrize("lens,T,H,G,dim,page,kind", CASES)
def test_matches_the_oracle(lens, T, H, G, dim, page, kind):
    C.say(f"tree_attention lens={lens[:5]} T={T} H={H} G={G} dim={dim} page={page} {kind}")
    rng = np.random.default_rng(T * 31 + dim + len(lens))
    S = len(lens)
    c = K.make(T + dim, lens, T, L=2, H=H, dim=dim, page=page)
    fill(c, rng, kind)
    cache = K.to_library(svg, c, kind)
    parent = trees(rng, S, T)
    q, qd = queries(rng, S, T, H * G, dim)
    ref, spread = AO.attention(c, wide(kind), 1, q, parent, T, None, dim ** -0.5)
    close(run(cache, qd, parent, T, layer=1), ref, bound(c, kind, spread, max(lens) + T))
    # chains, unequal trees and idle slots: rows behind a slot's nodes stay as they were
    n = [(s * 5 + T - 1) % (T + 1) for s in range(S)]
    n[0] = T
    got = run(cache, qd, None, T, n_nodes=n)
    ref, spread = AO.attention(c, wide(kind), 0, q, None, T, n, dim ** -0.5)
    for s in range(S):
        assert np.all(got[s, n[s]:] == 7.0)
        close(got[s, :n[s]], ref[s, :n[s]], bound(c, kind, spread, max(lens) + T)[s, :n[s]])


def share(c, first, tokens):
    """The slots' leading pages replaced by slot `first`'s."""
    n = tokens // c["page"]
    c["table"][:, :n] = c["table"][first, :n]


@pytest.mark.parametrize("lens,common,T,H,G,dim,page,kind", [
    ([300, 257, 256], 256, 1, 2, 4, 128, 64, "fp16"), ([64, 65, 130, 64], 64, 5, 1, 8, 64, 32, "bf16"),
    ([1500] * 3 + [1400] * 20, 1280, 1, 2, 2, 128, 128, "bf16"), ([520, 513], 512, 32, 1, 4, 256, 32, "fp16"),
    ([96] * 33, 96, 4, 2, 1, 64, 32, "fp16"), ([777, 5000, 640], 640, 3, 1, 4, 128, 64, "fp16"),
])
def test_a_shared_prefix(lens, common, T, H, G, dim, page, kind):
    C.say(f"tree_attention shared {common} of lens={lens[:4]} T={T} H={H} G={G} dim={dim} {kind}")
    rng = np.random.default_rng(common + T)
    S = len(lens)
    c = K.make(common, lens, T, H=H, dim=dim, page=page)
    fill(c, rng, kind)
    share(c, 0, common)
    cache = K.to_library(svg, c, kind)
    parent = trees(rng, S, T)
    q, qd = queries(rng, S, T, H * G, dim)
    n = [T] * S
    n[0] = 0                         # the first slot idle: another one's row names the pages
    ref, spread = AO.attention(c, wide(kind), 0, q, parent, T, n, dim ** -0.5)
    tol = bound(c, kind, spread, max(lens) + T)
    for said in (common, common + 10 ** 6, common - 31, common // 2 + 1, 31, 0, -5):
        if said > common and min(lens[1:]) > common:
            continue                 # (more than is shared, and not cut by a length)
        got = run(cache, qd, parent, T, n_nodes=n, shared=said)
        assert np.all(got[0] == 7.0)
        close(got[1:], ref[1:], tol[1:])


def test_scores_of_any_size():
    """Queries from 1e-30 to 1e30, zero rows, one-hot attention, a negative and a zero scale."""
    rng = np.random.default_rng(3)
    for kind in ("fp16", "bf16"):
        c = K.make(5, [200], 4, H=1, dim=64)
        fill(c, rng, kind)
        cache = K.to_library(svg, c, kind)
        q, _ = queries(rng, 1, 4, 8, 64)
        q = q.copy()
        q[0, 0] *= np.float32(1e-30)
        q[0, 1, 0] = 0
        q[0, 1, 1:] *= np.float32(1e4)
        q[0, 2] *= np.float32(60)
        q[0, 3, :4] *= np.float32(1e30)
        qd = C.to_dev(q.reshape(4, 8, 64))
        for scale in (0.125, -0.125, 0.0, 1e-3):
            ref, spread = AO.attention(c, wide(kind), 0, q, None, 4, None, scale)
            tol = bound(c, kind, spread, 204)
            got = run(cache, qd, None, 4, scale=scale)
            one = tol > 0.1          # scores so far apart that their rounding decides: a value of some token
            assert np.isfinite(got).all()
            assert np.all(np.abs(got[one]).max(-1) <= spread[one][:, 1] * 1.001) if one.any() else True
            close(np.where(one[..., None], 0, got), np.where(one[..., None], 0, ref), tol)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_what_a_row_does_not_see_never_reaches_it(kind):
    """NaN, infinities and the largest numbers in keys and values of siblings, of places behind
    the last token and of other pages; a value that is not finite reaches the rows that see it, as NaN or infinity."""
    rng = np.random.default_rng(8)
    T, dim = 6, 128
    lens = [70, 32]
    c = K.make(2, lens, T, H=2, dim=dim, page=64, spare=3)
    fill(c, rng, kind)
    parent = np.array([[-1, 0, 0, 1, 2, 3], [-1, 0, 1, 1, 1, 4]], np.int32)
    q, qd = queries(rng, 2, T, 4, dim)
    inf, nan = (0x7C00, 0x7E00) if kind == "fp16" else (0x7F80, 0x7FC0)
    pats = np.array([nan, inf, inf | 0x8000, inf - 1, 0xFFFF], np.uint16).view(np.int16)
    clean, _ = AO.attention(c, wide(kind), 0, q, parent, T, None, dim ** -0.5)
    spread = AO.attention(c, wide(kind), 0, q, parent, T, None, dim ** -0.5)[1]
    dirty = K.copy_of(c)
    # behind the last token, and pages nobody holds
    for s in range(2):
        for pos in range(lens[s] + T, int(c["pages"][s]) * 64):
            CO.put(dirty, 0, s, pos, pats[pos % 5], pats[(pos + 2) % 5])
    for p in np.flatnonzero(c["refs"] == 0):
        dirty["k"][:, p] = pats[0]
        dirty["v"][:, p] = pats[1]
    got = run(K.to_library(svg, dirty, kind), qd, parent, T)
    tol = bound(c, kind, spread, 80)
    close(got, clean, tol)
    # node 2 of the first tree (seen by nodes 2 and 4): its key, then its value
    for which in ("key", "value"):
        for pat in pats:
            d2 = K.copy_of(dirty)
            key, value = (np.array(x) for x in CO.token(d2, 0, 0, 72))
            if which == "key":
                key[:] = pat
            else:
                value[0, 5:9] = pat
            CO.put(d2, 0, 0, 72, key, value)
            got = run(K.to_library(svg, d2, kind), qd, parent, T)
            for i in (0, 1, 3, 5):
                close(got[0, i], clean[0, i], tol[0, i])
            close(got[1], clean[1], tol[1])
            if which == "value" and not np.isfinite(wide(kind)(np.array([pat]))[0]):
                assert not np.isfinite(got[0, [2, 4], :2, 5:9]).any()
                assert np.isfinite(got[0, [2, 4], 2:]).all() and np.isfinite(got[0, [2, 4], :2, 9:]).all()


def test_broken_trees_pages_and_slots_give_nan_rows_only_there():
    rng = np.random.default_rng(9)
    T, dim, lens = 5, 64, [70, 40, 50, 100, 33, 20, 64]
    c = K.make(4, lens, T, H=1, dim=dim, page=32)
    fill(c, rng, "fp16")
    parent = np.tile(np.array([-1, 0, 1, 1, 0], np.int32), (7, 1))
    q, qd = queries(rng, 7, T, 2, dim)
    ref, spread = AO.attention(c, wide("fp16"), 0, q, parent, T, None, dim ** -0.5)
    tol = bound(c, "fp16", spread, 110)
    parent[0, 1] = 3                 # nodes 1, 2, 3 hang off it
    parent[1, 0] = 0                 # no root
    parent[2, 4] = -1                # a second root
    d = K.copy_of(c)
    d["table"][3, 1] = 10 ** 9       # a page outside the cache
    d["table"][4, 0] = -1
    d["pages"][5] = 0                # no pages
    d["len"][6] = -1
    got = run(K.to_library(svg, d), qd, parent, T)
    for s, nodes in ((0, [1, 2, 3]), (1, range(T)), (2, [4]), (3, range(T)), (4, range(T)), (5, range(T)), (6, range(T))):
        ref[s, list(nodes)] = np.nan
    close(got, ref, tol)
    d["pages"][2] = 99               # more than the row has
    d["len"][0] = 10 ** 8            # more than its pages hold
    ref[[0, 2]] = np.nan
    close(run(K.to_library(svg, d), qd, parent, T), ref, tol)


def test_pages_beyond_four_gib():
    """A pool whose pages start beyond 2^32 bytes (and 2^31 elements)."""
    dim, page, H, P = 256, 128, 8, 9000   # 512 KiB a page: 4.6 GB for the keys, as much for the values
    k = torch.empty((1, P, H, page * dim), dtype=torch.float16, device=C.DEV)
    v = torch.empty_like(k)
    rng = np.random.default_rng(1)
    ids = [P - 1, 3, P - 2]
    c = K.make(1, [300], 4, H=H, dim=dim, page=page, spare=0)
    fill(c, rng, "fp16")
    src = c["table"][0, :3].copy()
    for a, b in zip(src, ids):
        k[0, b] = C.to_dev(c["k"][0, a]).view(torch.float16)
        v[0, b] = C.to_dev(c["v"][0, a]).view(torch.float16)
    cache = svg.KVCache(k, v, i32([ids + [-1]]), i32([3]), i32([300]), torch.zeros(P, dtype=torch.int32, device=C.DEV),
                        dim=dim, page=page)
    q, qd = queries(rng, 1, 4, 16, dim)
    ref, spread = AO.attention(c, wide("fp16"), 0, q, None, 4, None, dim ** -0.5)
    close(run(cache, qd, None, 4), ref, bound(c, "fp16", spread, 304))


def test_the_same_bits_every_time_and_in_a_captured_graph():
    """Two eager runs, and a graph replayed over growing lengths: equal bits each."""
    rng = np.random.default_rng(2)
    lens, T = [500, 64], 8
    c = K.make(6, lens, 200, H=2, dim=128, page=64)
    fill(c, rng, "fp16")
    cache = K.to_library(svg, c)
    parent = i32(trees(rng, 2, T))
    _q, qd = queries(rng, 2, T, 8, 128)
    ws, ws2 = (svg.tree_attention_workspace(cache, 8, T) for _ in range(2))
    out, eager = torch.zeros((2 * T, 8, 128), device=C.DEV), torch.zeros((2 * T, 8, 128), device=C.DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        svg.tree_attention(cache, 0, qd, parent, out, ws)
    side.synchronize()
    svg.tree_attention(cache, 0, qd, parent, eager, ws2)
    assert np.array_equal(C.host(out), C.host(eager))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svg.tree_attention(cache, 0, qd, parent, out, ws)
    for turn in range(4):
        cache.len += i32([40, 1])
        out.zero_()
        g.replay()
        svg.tree_attention(cache, 0, qd, parent, eager, ws2)
        assert np.array_equal(C.host(out), C.host(eager))


def test_two_streams_with_their_own_workspaces():
    rng = np.random.default_rng(4)
    c = K.make(7, [900], 8, H=4, dim=64)
    fill(c, rng, "bf16")
    cache = K.to_library(svg, c, "bf16")
    _q, qd = queries(rng, 1, 8, 8, 64)
    outs = [torch.zeros((8, 8, 64), device=C.DEV) for _ in range(2)]
    wss = [svg.tree_attention_workspace(cache, 8, 8) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o, w in zip(streams, outs, wss):
            svg.tree_attention(cache, 0, qd, None, o, w, stream=s)
    torch.cuda.synchronize()
    ref = torch.zeros((8, 8, 64), device=C.DEV)
    svg.tree_attention(cache, 0, qd, None, ref, wss[0])
    assert all(np.array_equal(C.host(o), C.host(ref)) for o in outs)


def test_the_binding_checks_its_tensors():
    """What the C call cannot see: devices, types, shapes, strides, the workspace's size."""
    c = K.make(1, [5, 9], 4, H=2, dim=64)
    cache = K.to_library(svg, c)
    q = torch.zeros((8, 4, 64), device=C.DEV)
    out, ws, par = torch.zeros_like(q), svg.tree_attention_workspace(cache, 4, 4), i32(np.zeros((2, 4)))
    ok = dict(q=q, parent=par, out=out, workspace=ws)
    svg.tree_attention(cache, 0, **ok)
    for kw, err in ((dict(q=q.half()), TypeError), (dict(q=q[:7]), ValueError), (dict(q=q.cpu()), ValueError),
                    (dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), ValueError), (dict(out=out[:, :2]), ValueError),
                    (dict(out=out.double()), TypeError), (dict(workspace=ws[:-1]), ValueError), (dict(parent=par.long()), TypeError),
                    (dict(parent=par[:1]), ValueError), (dict(n_nodes=i32([1])), ValueError),
                    (dict(shared=torch.zeros(0, dtype=torch.int32, device=C.DEV)), ValueError)):
        with pytest.raises(err):
            svg.tree_attention(cache, 0, **{**ok, **kw})
    with pytest.raises(svg.SvgError):
        svg.tree_attention(cache, 1, **ok)
    with pytest.raises(svg.SvgError):    # rows that do not begin on 16 bytes
        svg.tree_attention(cache, 0, **{**ok, "q": torch.zeros((8, 257), device=C.DEV)[:, 1:].unflatten(1, (4, 64))})
    k = torch.zeros((8, 2, 64), device=C.DEV)
    with pytest.raises(ValueError):
        svg.kv_append(cache, 0, k, k[:4], 4)
    with pytest.raises(ValueError):
        svg.kv_commit(cache, i32(np.zeros((3, 4))), i32([1, 1]))
    with pytest.raises(ValueError):
        svg.kv_fork(cache, i32([0, 0]), K.to_library(svg, c))
    with pytest.raises(svg.SvgError):
        svg.kv_fork(cache, i32([0, 0]), cache)
    with pytest.raises(ValueError):
        svg.kv_reserve(cache, i32([1, 1]), i32([0, 0]), svg.kv_workspace(cache)[:-1])


@pytest.mark.parametrize("lens,common,T,H,G,dim,page,kind", [
    ([(5 * s) % 70 for s in range(64)], 0, 1, 8, 4, 128, 64, "fp16"),         # a row tile, tokens in one to three tiles
    ([(7 * s) % 50 for s in range(300)], 0, 1, 8, 2, 64, 32, "bf16"),         # more heads of slots than the device has waves
    ([(11 * s) % 120 for s in range(40)], 0, 5, 8, 4, 128, 32, "bf16"),       # two row tiles
    ([(3 * s) % 90 for s in range(64)], 0, 2, 4, 8, 256, 32, "bf16"),
    ([130 + s for s in range(32)], 128, 1, 8, 1, 64, 32, "fp16"),             # branches with the prefix in the same launch
    ([64 + s % 3 for s in range(70)], 64, 2, 4, 4, 128, 64, "fp16"),          # and in a launch of its own
    ([2500] + [3] * 63, 0, 1, 4, 4, 64, 128, "fp16"),                         # one long slot among short ones
    ([0] * 256, 0, 1, 1, 8, 128, 32, "fp16"),
])
def test_many_slots_of_few_tokens(lens, common, T, H, G, dim, page, kind):
    C.say(f"tree_attention {len(lens)} slots, shared {common} T={T} H={H} G={G} dim={dim} {kind}")
    rng = np.random.default_rng(dim + T + len(lens))
    S = len(lens)
    c = K.make(S, lens, T, H=H, dim=dim, page=page)
    fill(c, rng, kind)
    share(c, 1, common)
    parent = trees(rng, S, T)
    q, qd = queries(rng, S, T, H * G, dim)
    n = [T - (s % 3 if s % 4 == 2 else 0) for s in range(S)]
    n = [max(x, 0) for x in n]
    n[7] = 0
    ref, spread = AO.attention(c, wide(kind), 0, q, parent, T, n, dim ** -0.5)
    tol = bound(c, kind, spread, max(lens) + T)
    d = K.copy_of(c)
    d["pages"][3] = 0                                # a slot without pages, one with a page outside the cache
    ref[3] = np.nan
    last = (lens[9] + n[9] - 1) // page
    d["table"][9, last] = 10 ** 8
    ref[9, :n[9]] = np.nan
    if T > 1:
        parent[10, 1] = 1
        ref[10, [i for i in range(T) if i == 1 or path_has(parent[10], i, 1)]] = np.nan
    cache = K.to_library(svg, d, kind)
    ws = svg.tree_attention_workspace(cache, H * G, T).fill_(0xFF)
    for _ in range(2):                               # the second time over the first one's workspace
        got = run(cache, qd, parent, T, n_nodes=n, shared=common or None, workspace=ws)
        for s in range(S):
            assert np.all(got[s, n[s]:] == 7.0), s
            close(got[s, :n[s]], ref[s, :n[s]], tol[s, :n[s]])


def path_has(parent, i, node):
    """Whether node i's path meets `node` before it ends."""
    for _ in range(len(parent)):
        if i == node:
            return True
        if i < 0 or parent[i] >= i:
            return False
        i = parent[i]
    return False


@pytest.mark.parametrize("lens,common,T,H,G,dim,page,kind", [
    ([12000], 0, 1, 1, 4, 128, 128, "fp16"), ([9500], 0, 2, 1, 8, 256, 64, "bf16"), ([5000], 0, 16, 2, 8, 128, 64, "bf16"),
    ([9100, 9000, 9300, 40], 0, 1, 1, 1, 64, 64, "fp16"), ([4200, 4101, 4300], 4096, 9, 1, 4, 256, 32, "fp16"),
])
def test_long_lists_of_partials(lens, common, T, H, G, dim, page, kind):
    """Few heads and many tokens: every workgroup of the device holds a part of the same rows."""
    C.say(f"tree_attention lens={lens} shared {common} T={T} H={H} G={G} dim={dim} {kind}")
    rng = np.random.default_rng(dim + T)
    c = K.make(dim, lens, T, H=H, dim=dim, page=page)
    fill(c, rng, kind)
    share(c, 0, common)
    parent = trees(rng, len(lens), T)
    q, qd = queries(rng, len(lens), T, H * G, dim)
    ref, spread = AO.attention(c, wide(kind), 0, q, parent, T, None, dim ** -0.5)
    tol = bound(c, kind, spread, max(lens) + T)
    cache = K.to_library(svg, c, kind)
    close(run(cache, qd, parent, T, shared=common or None), ref, tol)
    if len(lens) > 1:
        n = [T] * len(lens)
        n[1], c["len"][2] = 0, -1
        got = run(K.to_library(svg, c, kind), qd, parent, T, n_nodes=n, shared=common or None)
        assert np.all(got[1] == 7.0) and np.isnan(got[2]).all()
        close(got[0], ref[0], tol[0])


@pytest.mark.parametrize("lens,common,T,H,G,dim,page,kind", [
    ([500, 390, 420, 385], 384, 5, 2, 4, 128, 64, "bf16"),                # two row tiles of own tokens
    ([260 + s % 40 for s in range(70)], 256, 5, 4, 4, 64, 32, "fp16"),    # and many such slots
    ([700, 650, 641, 900, 640], 640, 2, 2, 4, 256, 64, "fp16"),
    ([200 + s for s in range(66)], 192, 1, 4, 8, 256, 64, "bf16"),
    ([64] * 3, 64, 7, 1, 3, 128, 64, "fp16"),                             # no own token but the nodes
    ([70 + s % 9 for s in range(140)], 64, 1, 2, 2, 64, 32, "fp16"),
    ([129] * 128, 128, 1, 1, 2, 64, 32, "bf16"), ([129] * 129, 128, 1, 1, 2, 64, 32, "bf16"),
])
def test_a_prefix_of_many_rows_beside_slots_of_few(lens, common, T, H, G, dim, page, kind):
    C.say(f"tree_attention {len(lens)} slots behind {common} T={T} H={H} G={G} dim={dim} {kind}")
    rng = np.random.default_rng(common + dim)
    S = len(lens)
    c = K.make(common, lens, T, H=H, dim=dim, page=page)
    fill(c, rng, kind)
    share(c, 0, common)
    parent = trees(rng, S, T)
    q, qd = queries(rng, S, T, H * G, dim)
    n = [T] * S
    n[2] = max(T - 2, 0)
    ref, spread = AO.attention(c, wide(kind), 0, q, parent, T, n, dim ** -0.5)
    tol = bound(c, kind, spread, max(lens) + T)
    cache = K.to_library(svg, c, kind)
    for said in (common, 33):
        got = run(cache, qd, parent, T, n_nodes=n, shared=said)
        assert np.all(got[2, n[2]:] == 7.0)
        for s in range(S):
            close(got[s, :n[s]], ref[s, :n[s]], tol[s, :n[s]])


@pytest.mark.parametrize("common", [0, 64])
def test_one_captured_graph_from_short_slots_to_long_ones(common):
    """Which workgroups work on what is decided on the device: a graph captured over slots of few tokens serves long and
    unequal ones, and short ones again, with the bits of an eager call each time."""
    rng = np.random.default_rng(11)
    S, T = 64, 2
    c = K.make(3, [70 + s % 5 for s in range(S)], 900, H=4, dim=64, page=64)
    fill(c, rng, "fp16")
    share(c, 0, common)
    cache = K.to_library(svg, c)
    _q, qd = queries(rng, S, T, 16, 64)
    shared = i32([common]) if common else None
    ws, ws2 = (svg.tree_attention_workspace(cache, 16, T) for _ in range(2))
    out, eager = torch.zeros((S * T, 16, 64), device=C.DEV), torch.zeros((S * T, 16, 64), device=C.DEV)
    short = cache.len.clone()
    svg.tree_attention(cache, 0, qd, None, out, ws, shared=shared)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svg.tree_attention(cache, 0, qd, None, out, ws, shared=shared)
    for turn, lens in enumerate((short, short + 400, short + 10 * torch.arange(S, dtype=torch.int32, device=C.DEV), short + 820, short)):
        cache.len.copy_(lens)
        out.zero_()
        g.replay()
        svg.tree_attention(cache, 0, qd, None, eager, ws2, shared=shared)
        assert np.array_equal(C.host(out), C.host(eager)), turn
        assert np.isfinite(C.host(eager)).all()
    c["len"] = (short + 10 * torch.arange(S, dtype=torch.int32, device=C.DEV)).cpu().numpy()
    cache.len.copy_(i32(c["len"]))
    g.replay()
    q = C.host(qd).reshape(S, T, 16, 64)
    ref, spread = AO.attention(c, wide("fp16"), 0, q, None, T, None, 64 ** -0.5)
    close(C.host(out).reshape(S, T, 16, 64).astype(np.float64), ref, bound(c, "fp16", spread, 1000))
