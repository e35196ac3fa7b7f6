"""What svgemm_layer.h says of the calls' edges: slots that were refused, pages
that several slots hold, rows far from ordinary, sizes at the limits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import attention_oracle as AO
from oracle import cache_oracle as CO


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    global A, C, K, svg
    import cache_cases as K  # noqa: F401
    import svg_cases as C  # noqa: F401
    import test_tree_attention_parity as A  # noqa: F401
    import speculative_verify_gemm_amd as svg
    A.svg, A.C, A.K = svg, C, K


# ------------------------------------------------- pages of several holders
def refused_forks(kind="fp16", dim=64):
    """Slots 1 and 2, forks of one another in the middle of a page, that kv_reserve had no pages left for; slot 0 took
    them.  The oracle's cache and the library's."""
    c = K.make(11, [10, 40, 70], 0, L=2, H=2, dim=dim, page=32, spare=0, width=6)
    A.fill(c, np.random.default_rng(3), kind)
    a = K.to_library(svg, c, kind)
    b = a.other_tables()
    svg.kv_fork(a, A.i32([0, 1, 1]), b)
    c = CO.fork(c, [0, 1, 1])
    status = A.i32([9, 9, 9])
    svg.kv_reserve(b, A.i32([118, 8, 8]), status, svg.kv_workspace(b))
    assert list(CO.reserve(c, [118, 8, 8])) == list(C.host(status)) == [0, 1, 1]
    K.same(b, c)
    assert c["refs"][c["table"][1, 1]] == 2 and c["table"][1, 1] == c["table"][2, 1]
    return c, b


def rows(seed, S, T, kind="fp16", dim=64):
    """fp32 rows of keys and values on the device, and their patterns."""
    x = torch.randn((2, S * T, 2 * dim), generator=torch.Generator().manual_seed(seed))
    pat = K.bits(x.to(K.TYPES[kind])).reshape(2, S, T, 2, dim)
    return x[0].to(C.DEV), x[1].to(C.DEV), pat[0], pat[1]


def test_the_oracle_leaves_pages_of_several_holders():
    z = np.zeros((1, 3, 1, 32 * 64), np.int16)
    c = dict(k=z.copy(), v=z.copy(), table=np.array([[0, 1], [0, 2]], np.int32), pages=np.array([2, 2], np.int32),
             len=np.array([30, 32], np.int32), refs=np.array([2, 1, 1], np.int32), dim=64, page=32)
    new = np.arange(2 * 4 * 64, dtype=np.int16).reshape(2, 4, 1, 64) + 1
    CO.append(c, 0, new, new, 4)
    assert not c["k"][0, 0].any() and not c["v"][0, 0].any()
    assert np.array_equal(CO.token(c, 0, 0, 32)[0], new[0, 2]) and np.array_equal(CO.token(c, 0, 1, 35)[1], new[1, 3])
    path = np.array([[2, -1, -1, -1], [2, -1, -1, -1]])
    assert list(CO.commit(c, path, [1, 1])) == [30, 33] and list(CO.commit(c, path, [2, 2])) == [30, 34]
    assert np.array_equal(CO.token(c, 0, 1, 33)[0], new[1, 2]) and not c["k"][0, 0].any()


@pytest.mark.gpu
def test_append_and_commit_leave_pages_of_several_holders(gpu):
    T = 8
    c, cache = refused_forks()
    k, v, kp, vp = rows(1, 3, T)
    for n in ([T, T, 0], [0, 0, T], [T, T, T]):  # one of the refused slots, the other, both
        svg.kv_append(cache, 1, k, v, T, n_rows=A.i32(n))
        CO.append(c, 1, kp, vp, T, n)
        K.same(cache, c)
    # the path of a refused slot stays where it is: moves, and the root alone
    path = np.full((3, T), -1, np.int32)
    path[:, :2] = [2, 5]
    for n in ([3, 3, 1], [1, 1, 3]):
        out = torch.zeros(3, dtype=torch.int32, device=C.DEV)
        svg.kv_commit(cache, A.i32(path), A.i32(n), out)
        new = CO.commit(c, path, n)
        assert list(new) == list(C.host(out)) == [10 + n[0], 40, 40]
        K.same(cache, c)
    # one of them given up: the page is the other's own, and takes its rows
    b = cache.other_tables()
    svg.kv_fork(cache, A.i32([0, 1, -1]), b)
    c = CO.fork(c, [0, 1, -1])
    svg.kv_append(b, 0, k, v, T)
    CO.append(c, 0, kp, vp, T)
    svg.kv_commit(b, A.i32(path), A.i32([1, 3, 0]))
    c["len"] = CO.commit(c, path, [1, 3, 0])
    assert list(c["len"]) == [11, 43, 0]
    K.same(b, c)


@pytest.mark.gpu
def test_a_path_that_reaches_into_a_page_of_several_holders(gpu):
    """The root's page is the slot's own and the next one is not: what lies in the first is written, and nothing committed."""
    c = K.make(5, [30, 30], 8, L=1, H=1, dim=64, page=32)
    A.fill(c, np.random.default_rng(4), "fp16")
    c["table"][1, 1] = c["table"][0, 1]
    c["refs"] = CO.holders(c).astype(np.int32)
    cache = K.to_library(svg, c)
    x = torch.randn((2, 16, 64), generator=torch.Generator().manual_seed(2))
    pat = K.bits(x.half()).reshape(2, 2, 8, 1, 64)
    svg.kv_append(cache, 0, x[0].to(C.DEV), x[1].to(C.DEV), 8)
    CO.append(c, 0, pat[0], pat[1], 8)
    K.same(cache, c)
    path = np.full((2, 8), -1, np.int32)
    path[:, 0] = [1, 2]                  # inside the first page; in the second
    out = torch.zeros(2, dtype=torch.int32, device=C.DEV)
    svg.kv_commit(cache, A.i32(path), A.i32([2, 2]), out)
    assert list(CO.commit(c, path, [2, 2])) == list(C.host(out)) == [32, 30]
    K.same(cache, c)


@pytest.mark.gpu
def test_attention_of_refused_slots_is_nan(gpu):
    """The rows that kv_append has passed over are never read as if they were the slot's."""
    T, A_, dim = 8, 4, 64
    c, cache = refused_forks()
    k, v, kp, vp = rows(1, 3, T)
    svg.kv_append(cache, 1, k, v, T)
    CO.append(c, 1, kp, vp, T)
    q, qd = A.queries(np.random.default_rng(7), 3, T, A_, dim)
    ref, spread = AO.attention(c, A.wide("fp16"), 1, q, None, T, None, dim ** -0.5)
    assert np.isnan(ref[1:]).all() and np.isfinite(ref[0]).all()
    A.close(A.run(cache, qd, None, T, layer=1), ref, A.bound(c, "fp16", spread, 80))
    n = [T, 0, 0]                        # as such slots are to be called: they take no part
    got = A.run(cache, qd, None, T, layer=1, n_nodes=n)
    assert (got[1:] == 7.0).all()
    A.close(got[:1], ref[:1], A.bound(c, "fp16", spread, 80)[:1])


@pytest.mark.gpu
@pytest.mark.parametrize("S,common,T,H,G,dim,page,kind", [
    (3, 0, 7, 2, 2, 64, 32, "fp16"), (3, 0, 32, 2, 8, 128, 32, "bf16"), (4, 0, 6, 1, 8, 256, 64, "fp16"),
    (40, 0, 3, 8, 2, 128, 32, "bf16"), (20, 64, 4, 2, 4, 128, 64, "fp16"), (70, 64, 2, 4, 4, 64, 64, "bf16"),
])
def test_attention_of_trees_that_reach_into_a_page_of_several_holders(gpu, S, common, T, H, G, dim, page, kind):
    """Every way over the tiles: some slots' trees begin in a page of their own and go on in one that others hold."""
    C.say(f"tree_attention, shared tree pages: S={S} common={common} T={T} H={H} G={G} dim={dim} {kind}")
    rng = np.random.default_rng(S + T)
    lens = [common + page - 1 - s % 3 for s in range(S)]
    c = K.make(S, lens, max(T, 4), H=H, dim=dim, page=page)
    A.fill(c, rng, kind)
    A.share(c, 0, common)
    two = 1 + common // page
    for s in range(1, S, 3):             # the page behind: the first slot's
        c["table"][s, two] = c["table"][0, two]
    c["refs"] = CO.holders(c).astype(np.int32)
    parent = A.trees(rng, S, T)
    parent[-1] = -1
    parent[-1, 1:] = 0                   # siblings: those behind the page's end are alone in it
    q, qd = A.queries(rng, S, T, H * G, dim)
    ref, spread = AO.attention(c, A.wide(kind), 0, q, parent, T, None, dim ** -0.5)
    assert np.isnan(ref).any() and np.isfinite(ref).any()
    got = A.run(K.to_library(svg, c, kind), qd, parent, T, shared=common or None)
    A.close(got, ref, A.bound(c, kind, spread, max(lens) + T))


# -------------------------------------------------------- rows far from ordinary
@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,T,G", [(128, 1, 2), (64, 16, 3), (256, 5, 8)])
@pytest.mark.parametrize("above", [2.0 ** 11, 2.0 ** 16, 2.0 ** 20])
def test_one_channel_of_q_far_above_the_others(gpu, kind, dim, T, G, above):
    """The keys hardly use the large channel, so the small ones decide: they keep their bits.  Beside the bound of the
    ordinary rows, a value of q is off by 2^-38 of its row's largest at most (fp16 parts end at 2^-24, half a step of
    which is 2^-25, and the largest is at least 2^13): a score by 2^-38 scale max|q| sum|k|."""
    rng = np.random.default_rng(dim + T)
    c = K.make(7, [1000], T, H=1, dim=dim, page=64)
    A.fill(c, rng, kind)
    cols = [3, dim - 2]
    t = np.arange(64)
    for d in cols:                       # 0 in the large channels
        c["k"][0, :, 0, CO.key_at(t, d, dim)] = 0
    q, _ = A.queries(rng, 1, T, G, dim)
    q = q.copy()
    q[..., cols] = np.float32(above) * np.sign(q[..., cols])
    qd = C.to_dev(q.reshape(T, G, dim))
    ref, spread = AO.attention(c, A.wide(kind), 0, q, None, T, None, dim ** -0.5)
    tol = A.bound(c, kind, spread, 1000 + T)
    if kind == "fp16":
        most = np.abs(A.wide(kind)(c["k"][0, :, 0])).reshape(-1, 64 // 16, dim // 32, 4, 16, 8).sum((2, 3, 5)).max()
        tol = tol + spread[..., 1] * 2 * 2.0 ** -38 * dim ** -0.5 * above * most
    A.close(A.run(K.to_library(svg, c, kind), qd, None, T), ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("low", [31.5, 33.5, 35.5, 39.5])
def test_a_long_tail_of_small_probabilities(gpu, kind, low):
    """One token and 2^18 others, each of them 2^-low of it: together 2^(18 - low).  256 slots over the same pages, so
    that a workgroup has a slot and its waves an eighth of the tokens (thin) or half of them (thick).  A probability's two
    fp16 parts lose up to 2^-36 of the largest that the wave has seen: 2^-36 for each token of a wave, which the others'
    sums do not see.  Beside it stands the ordinary bound, relative to what it is the bound of: a score of one product
    (q in parts; q's factor and the exponent rounded), the exponential, p in two parts, and sums of one sign over a
    wave's tiles, eight rounded ones a tile."""
    S, dim, page, N = 256, 64, 128, 1 << 18
    k = torch.zeros((N, dim))
    v = torch.zeros((N, dim))
    at = 177777                          # the large one: not the first to be seen
    k[at, 0] = 32.0
    v[:, 1] = 1.0
    v[at, 1] = 0.0
    v[at, 2] = 1.0
    P = N // page
    pool = lambda: torch.zeros((1, P + S, 1, page * dim), dtype=K.TYPES[kind], device=C.DEV)  # noqa: E731
    kp, vp = pool(), pool()
    refs = torch.ones(P + S, dtype=torch.int32, device=C.DEV)
    pages = torch.arange(P, dtype=torch.int32, device=C.DEV)
    first = svg.KVCache(kp, vp, pages[None].contiguous(), A.i32([P]), A.i32([0]), refs, dim=dim, page=page)
    svg.kv_append(first, 0, k.to(C.DEV), v.to(C.DEV), N)
    own = torch.arange(P, P + S, dtype=torch.int32, device=C.DEV)[:, None]   # for the tree's token: a zero key and value
    refs[:P] = S
    cache = svg.KVCache(kp, vp, torch.cat((pages.expand(S, P), own), 1).contiguous(), A.i32([P + 1] * S), A.i32([N] * S), refs,
                        dim=dim, page=page)
    for G, part in ((1, N // 8), (40, N // 2)):
        q = np.zeros((S, G, dim), np.float32)
        q[:, :, 0] = low * np.log(2.0) / 32.0
        got = A.run(cache, C.to_dev(q), None, 1, scale=1.0)[:, 0]
        x = 32.0 * float(q[0, 0, 0])     # the large one's score; all others have 0
        e = np.exp(-x)
        total = 1 + N * e                # (N - 1 others and the tree's own)
        u = 2.0 ** -11 if kind == "fp16" else 2.0 ** -8
        score = x * ((u ** 2 if kind == "fp16" else u ** 3) + 3 * 2.0 ** -24)
        tol = 2 * (score + 2.0 ** -20 + u ** 2 + (8 * part / 32 + 64) * 2.0 ** -24)
        lost = part * 2.0 ** -36 if kind == "fp16" else 0.0
        tail = (N - 1) * e / total
        err = np.abs(got[:, :, 1] - tail).max()
        print(f"{kind} 2^-{low} G={G}: tail {tail:.3e}, off by {err:.3e} of {tail * tol + lost:.3e}", flush=True)
        assert err <= tail * tol + lost
        assert np.abs(got[:, :, 2] - 1 / total).max() <= tol + lost
        assert (got[:, :, 3:] == 0).all() and (got[:, :, 0] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("T,G,common", [(1, 4, 0), (3, 2, 64), (32, 8, 0), (20, 3, 64)])
def test_committed_keys_and_values_that_are_not_finite(gpu, kind, T, G, common):
    """A committed key of +-infinity or NaN: the rows of its head are NaN, or those of the definition (a score of
    -infinity leaves the token out); a value: its own element is not finite.  No other head, slot or element has them."""
    rng = np.random.default_rng(T + G)
    S, H, dim, page = 2, 2, 64, 32
    lens = [common + 40, common + 3]
    c = K.make(3, lens, T, H=H, dim=dim, page=page)
    A.fill(c, rng, kind)
    A.share(c, 0, common)
    q, qd = A.queries(rng, S, T, H * G, dim)
    clean, spread = AO.attention(c, A.wide(kind), 0, q, None, T, None, dim ** -0.5)
    tol = A.bound(c, kind, spread, max(lens) + T)
    inf, nan = (0x7C00, 0x7E00) if kind == "fp16" else (0x7F80, 0x7FC0)
    for pos in (5, lens[0] - 1):         # in a whole tile, and in the tile where the tree begins
        hit = [0, 1] if pos < common else [0]
        for pat in np.array([nan, inf, inf | 0x8000], np.uint16).view(np.int16):
            d = K.copy_of(c)
            key, value = (np.array(x) for x in CO.token(d, 0, 0, pos))
            key[0, 7] = pat
            CO.put(d, 0, 0, pos, key, value)
            got = A.run(K.to_library(svg, d, kind), qd, None, T, shared=common or None)
            with np.errstate(invalid="ignore"):
                ref, _ = AO.attention(d, A.wide(kind), 0, q, None, T, None, dim ** -0.5)
            for s in range(S):
                for a in range(H * G):
                    if s in hit and a < G:
                        out = np.isnan(got[s, :, a]).all(-1)
                        assert out[np.isnan(ref[s, :, a]).all(-1)].all()
                        A.close(got[s, ~out, a], ref[s, ~out, a], tol[s, ~out, a])
                    else:
                        A.close(got[s, :, a], clean[s, :, a], tol[s, :, a])
            d = K.copy_of(c)
            key, value = (np.array(x) for x in CO.token(d, 0, 0, pos))
            value[1, 9] = pat
            CO.put(d, 0, 0, pos, key, value)
            got = A.run(K.to_library(svg, d, kind), qd, None, T, shared=common or None)
            assert not np.isfinite(got[hit][:, :, G:, 9]).any()
            got[hit, :, G:, 9] = clean[hit, :, G:, 9]
            A.close(got, clean, tol)


# ------------------------------------------------------------ sizes at the limits
@pytest.mark.gpu
@pytest.mark.parametrize("M", [1 << 20, (1 << 20) + 1, (1 << 24) - 33, 1 << 24])
def test_norm_of_as_many_rows_as_it_takes(gpu, M):
    """Up to 2^24 rows, past what one dimension of a grid holds: the codes of the same rows in calls of 2^18."""
    K_, part = 32, 1 << 18
    g = torch.Generator(device=C.DEV).manual_seed(M)
    x = torch.randn((M, K_), device=C.DEV, dtype=torch.float16, generator=g)
    w = torch.randn(K_, device=C.DEV, generator=g)
    signs = (torch.randint(0, 2, (K_,), device=C.DEV, generator=g) * 2 - 1).to(torch.int8)
    new = lambda: (torch.zeros((M, K_), dtype=torch.int8, device=C.DEV), torch.zeros(M, device=C.DEV))  # noqa: E731
    (xq, xs), (pq, ps) = new(), new()
    svg.add_rmsnorm_quant_i8(x, None, w, 1e-5, signs, xq, xs)
    for a in range(0, M, part):
        b = min(a + part, M)
        svg.add_rmsnorm_quant_i8(x[a:b], None, w, 1e-5, signs, pq[a:b], ps[a:b])
    assert torch.equal(xq, pq) and torch.equal(xs, ps) and bool((xs > 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1 << 28, (1 << 31) - 1])
def test_append_of_more_rows_than_any_table_holds(gpu, T):
    """T itself is not limited by the table: rows without a place are passed over, however many there could be.  (The C
    call: n_rows says that only the first rows are there.)"""
    c = K.make(9, [5], 40, H=1, dim=64, page=32)
    cache = K.to_library(svg, c)
    x = torch.randn((2, 70, 64), generator=torch.Generator().manual_seed(1))
    d, n = x.to(C.DEV), A.i32([70])
    stream = torch.cuda.current_stream().cuda_stream
    assert svg.lib.kv_append(cache._ref, 0, d[0].data_ptr(), 64, d[1].data_ptr(), 64, T, n.data_ptr(), stream) == 0
    pat = K.bits(x.half()).reshape(2, 1, 70, 1, 64)
    CO.append(c, 0, pat[0], pat[1], 70, [70])
    K.same(cache, c)


# ------------------------------------------------------------------ the binding
@pytest.mark.gpu
def test_the_caches_tensors_may_be_replaced(gpu):
    """Lengths that alternate between two tensors, as a program keeps them that commits into the other one; tables
    and pages likewise."""
    T, lens = 4, [10, 33]
    c = K.make(2, lens, 40, H=1, dim=64, page=32)
    cache = K.to_library(svg, c)
    other = torch.zeros_like(cache.len)
    path = np.full((2, T), -1, np.int32)
    path[:, 0] = 2
    for turn in range(3):
        k, v, kp, vp = rows(turn, 2, T)
        k, v, kp, vp = k[:, :64].contiguous(), v[:, :64].contiguous(), kp[:, :, :1], vp[:, :, :1]
        svg.kv_append(cache, 0, k, v, T)
        CO.append(c, 0, kp, vp, T)
        svg.kv_commit(cache, A.i32(path), A.i32([2, 2]), other)
        c["len"] = CO.commit(c, path, [2, 2])
        cache.len, other = other, cache.len
        K.same(cache, c)
    cache.len += A.i32([1, 0])           # in place: the same tensor
    c["len"][0] += 1
    table = cache.table.clone()
    cache.table.fill_(-1)                # the old one is not looked at any more
    cache.table = table
    cache.k, cache.v = cache.k.clone(), cache.v.clone()
    k, v, kp, vp = rows(7, 2, T)
    svg.kv_append(cache, 0, k[:, :64].contiguous(), v[:, :64].contiguous(), T)
    CO.append(c, 0, kp[:, :, :1], vp[:, :, :1], T)
    K.same(cache, c)
    for name, t, err in (("len", torch.zeros(3, dtype=torch.int32, device=C.DEV), ValueError), ("len", cache.len.long(), TypeError),
                         ("len", cache.len.cpu(), ValueError), ("refs", None, ValueError), ("k", cache.k.bfloat16(), TypeError),
                         ("table", table.t().contiguous().t(), ValueError)):
        with pytest.raises(err):
            setattr(cache, name, t)
    K.same(cache, c)
    with pytest.raises(ValueError):
        svg.KVCache(cache.k, cache.v, dim=64, page=32).len = cache.len


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5])
def test_no_slots_are_empty_calls(gpu, T):
    """A cache of no slots: every call of the binding is a call of nothing, whatever the trees' size."""
    cache = svg.KVCache.empty(1, 4, 2, 64, 32, 0, 3, device=C.DEV)
    none = lambda *s: torch.zeros((0, *s), dtype=torch.int32, device=C.DEV)  # noqa: E731
    q = torch.zeros((0, 4, 64), device=C.DEV)
    ws = svg.tree_attention_workspace(cache, 4, T)
    svg.tree_attention(cache, 0, q, none(T), torch.zeros_like(q), ws)
    svg.tree_attention(cache, 0, q, none(T), torch.zeros_like(q), ws, n_nodes=none(), shared=A.i32([32]))
    svg.tree_attention(cache, 0, q, None, torch.zeros_like(q), ws)
    with pytest.raises(ValueError):
        svg.tree_attention(cache, 0, q, A.i32(np.zeros((1, T))), torch.zeros_like(q), ws)
    kv = torch.zeros((0, 2, 64), device=C.DEV)
    svg.kv_append(cache, 0, kv, kv, T, n_rows=none())
    svg.kv_commit(cache, none(T), none())
    svg.kv_fork(cache, none(), cache.other_tables())
    svg.kv_reserve(cache, none(), none(), svg.kv_workspace(cache))
    torch.cuda.synchronize()
    assert not C.host(cache.refs).any()


# ------------------------------------------------------------------- the build
def test_the_digest_covers_the_flags_of_each_source(monkeypatch):
    from speculative_verify_gemm_amd import build as B
    less = B.LESS_FLAGS["tree_attention.hip"]
    assert all(f not in B.flags_of("tree_attention.hip") for f in less[1:]) and all(f in B.flags_of("layout.hip") for f in less)
    now = B.source_digest()
    monkeypatch.setattr(B, "LESS_FLAGS", {})
    assert B.source_digest() != now
    monkeypatch.setattr(B, "LESS_FLAGS", {"tree_attention.hip": less, "layout.hip": less})
    assert B.source_digest() != now
    monkeypatch.setattr(B, "LESS_FLAGS", {"tree_attention.hip": less})
    assert B.source_digest() == now


@pytest.mark.gpu
def test_without_counts_no_page_is_passed_over(gpu):
    """refs NULL (the C calls): append, attention and commit go by the tables alone."""
    T = 8
    c, cache = refused_forks()
    cache._c.refs = None
    c["refs"][:] = 0
    k, v, kp, vp = rows(4, 3, T)
    n = [T, T, 0]                        # one of the two slots over the same page
    svg.kv_append(cache, 1, k, v, T, n_rows=A.i32(n))
    CO.append(c, 1, kp, vp, T, n)
    K.same(cache, c, ("k", "v"))
    q, qd = A.queries(np.random.default_rng(8), 3, T, 4, 64)
    ref, spread = AO.attention(c, A.wide("fp16"), 1, q, None, T, n, 64 ** -0.5)
    got = A.run(cache, qd, None, T, layer=1, n_nodes=n)
    assert np.isfinite(ref[:2]).all()
    A.close(got[:2], ref[:2], A.bound(c, "fp16", spread, 80)[:2])
    path = np.full((3, T), -1, np.int32)
    path[:, 0] = 4
    svg.kv_commit(cache, A.i32(path), A.i32([2, 2, 0]))
    c["len"] = CO.commit(c, path, [2, 2, 0])
    assert list(c["len"]) == [12, 42, 40]
    K.same(cache, c, ("k", "v", "len"))


@pytest.mark.gpu
@pytest.mark.parametrize("seed,kind,careful", [(1, "fp16", False), (2, "bf16", False), (3, "fp16", True), (4, "bf16", True)])
def test_serving_from_a_pool_that_is_too_small(gpu, seed, kind, careful):
    """Turns of fork, reserve, append, attention and commit with refusals in most of them; every call against the oracle.
    careful: refused slots are given no rows, nodes and tokens; otherwise the program goes on with them."""
    S, T, H, G, dim, page = 6, 12, 2, 2, 64, 32
    rng = np.random.default_rng(seed)
    c = K.make(seed, [int(x) for x in rng.integers(1, 70, S)], 0, H=H, dim=dim, page=page, spare=0, width=12)
    A.fill(c, rng, kind)
    cache = K.to_library(svg, c, kind)
    ws, kv_ws, status = svg.tree_attention_workspace(cache, H * G, T), svg.kv_workspace(cache), A.i32([0] * S)
    refused = nan_slots = 0
    for turn in range(14):
        src = np.where(rng.random(S) < 0.12, rng.integers(0 if turn % 5 else -1, S, S), np.arange(S))
        other = cache.other_tables()
        svg.kv_fork(cache, A.i32(src), other)
        c, cache = CO.fork(c, src), other
        K.same(cache, c)
        assert np.array_equal(CO.holders(c), c["refs"])
        n = rng.integers(0, T + 1, S)
        svg.kv_reserve(cache, A.i32(n), status, kv_ws)
        state = CO.reserve(c, n)
        assert np.array_equal(C.host(status), state)
        K.same(cache, c)
        refused += int((state != 0).sum())
        if careful:
            n = np.where(state == 0, n, 0)
        k, v, kp, vp = rows(100 * seed + turn, S, T, kind)
        svg.kv_append(cache, 0, k, v, T, n_rows=A.i32(n))
        CO.append(c, 0, kp, vp, T, n)
        K.same(cache, c)
        parent = A.trees(rng, S, T)
        q, qd = A.queries(rng, S, T, H * G, dim)
        covered = c["len"] + n <= c["pages"] * page
        ref, spread = AO.attention(c, A.wide(kind), 0, q, parent, T, np.where(covered, n, 0), dim ** -0.5)
        tol = A.bound(c, kind, spread, int(c["len"].max()) + T)
        got = A.run(cache, qd, parent, T, n_nodes=n, workspace=ws)
        for s in range(S):
            A.close(got[s, :n[s]], ref[s, :n[s]], tol[s, :n[s]])
            assert (got[s, n[s]:] == 7.0).all()
            nan_slots += bool(np.isnan(got[s, :n[s]]).any())
        count = np.minimum(rng.integers(1, T + 1, S), n)
        path = np.full((S, T), -1, np.int32)
        for s in range(S):
            if count[s] > 1:
                path[s, :count[s] - 1] = np.sort(rng.choice(np.arange(1, n[s]), size=count[s] - 1, replace=False))
        svg.kv_commit(cache, A.i32(path), A.i32(count))
        c["len"] = CO.commit(c, path, count)
        K.same(cache, c)
    assert refused > 3 and (nan_slots > 0) != careful
