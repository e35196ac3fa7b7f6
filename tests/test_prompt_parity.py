"""A prompt's pass on the device against the oracle (oracle/prompt_oracle.py).

Tolerances, from the number formats; u is half a step of the type that is written (fp16 2^-11, bf16 2^-8,
fp32 2^-24) and e = 2^-24.  fp16 numbers below 2^-14 lie 2^-24 apart: they are off by up to 2^-25, which is more than
u of themselves (half_step).
  rope       cosine and sine are within 2 units of fp32's last place (4 e of themselves), then a product and a
             fused product-sum: 6 e (|a c| + |b s|), and u of the value.
  linears    W8: the sum's conversion, the product of the scales and the last product: 3 e of the value.  W4: a conversion and a
             fused product-sum a group and the last product: (groups + 2) e of sum |s S| x_scale.  Then u of the value.
  attention  a score is a sum of dim products of 16-bit numbers in fp32: with B = scale * sum |q k| a probability is
             off by E = 2 (dim + 8) e B + 2^-20 (the exponential and its argument) relative, and by u for its rounding; numerator and
             denominator, which carry the same weights, are both off by that: 2 (E + u) (mean |v| + |o|) / 2; the sums over the tiles
             add (tiles + 64) e max |v|; a probability below fp16's smallest step is off by 2^-33 of the largest: L 2^-33 max |v|;
             and the output by u of itself."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache_oracle as CO
from oracle import norm_oracle as NO
from oracle import prompt_oracle as PO
from oracle import svg_oracle as O

U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
E = 2.0 ** -24
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}

pytestmark = pytest.mark.gpu


def half_step(kind, ref):
    return np.maximum(U[kind] * np.abs(ref), 2.0 ** -25 if kind == "fp16" else 0.0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    global C, K, svg
    import svg_cases as C  # noqa: F401
    import cache_cases as K  # noqa: F401
    import speculative_verify_gemm_amd as svg


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=C.DEV)


def wide(kind):
    return lambda a: torch.from_numpy(np.ascontiguousarray(a)).view(TYPES[kind]).double().numpy()


def fill(c, rng, kind):
    for name in ("k", "v"):
        c[name] = K.bits(torch.from_numpy(rng.standard_normal(c[name].shape).astype(np.float32)).to(TYPES[kind]))


def host64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ row map
def trees(rng, S, T):
    parent = np.full((S, T), -1, np.int32)
    for s in range(S):
        for i in range(1, T):
            parent[s, i] = i - 1 if s == 0 else rng.integers(0, i)
    return parent


def check_map(c, n_new, T, n_rows, parent=None, slot=True):
    cache = K.to_library(svg, c)
    rows = svg.RowMap.empty(cache, n_rows)
    for t in (rows.start, rows.count, rows.pos, rows.place, rows.slot):
        t.fill_(77)
    if not slot:
        rows = svg.RowMap(rows.start, rows.count, rows.pos, rows.place)
    svg.kv_row_map(cache, i32(n_new), rows, T=T, parent=None if parent is None else i32(parent))
    want = PO.row_map(c, n_new, T, n_rows, parent)
    for name, w in zip(("start", "count", "slot", "pos", "place"), want):
        t = getattr(rows, name)
        if t is not None:
            assert np.array_equal(C.host(t), w), name
    return cache, rows


@pytest.mark.parametrize("S,page,most,spare_rows", [(1, 32, 1, 0), (3, 32, 70, 5), (7, 64, 40, 0), (257, 128, 9, 300), (1024, 32, 3, 1)])
def test_packed_rows(S, page, most, spare_rows):
    C.say(f"kv_row_map packed S={S} page={page} most={most}")
    rng = np.random.default_rng(S)
    n = rng.integers(-1, most + 1, S)
    n[0] = most
    c = K.make(S, list(rng.integers(0, 100, S)), most, page=page, H=1, dim=64)
    # refused slots: pages missing, a page of two holders, a page number outside the cache, a length that is none
    c["pages"][S // 2] = max(0, c["pages"][S // 2] - 1)
    c["refs"][c["table"][S // 3, 0]] = 2
    c["table"][S - 1, 0] = (1 << 20) if S % 2 else -5
    c["len"][S // 5] = -3 if S > 5 else c["len"][S // 5]
    total = int(np.maximum(n, 0).sum())
    for rows in {total + spare_rows, total, max(total - 2, 0), 1}:
        check_map(c, n, 0, rows, slot=rows != total)


def test_packed_rows_of_huge_numbers():
    c = K.make(1, [5, 9, 0], 4, H=1, dim=64)
    for n in ([2 ** 31 - 1] * 3, [0, 2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, 3, 2 ** 31 - 1]):
        check_map(c, n, 0, 100)
    c["len"][:] = 2 ** 31 - 2
    check_map(c, [3, 3, 3], 0, 9)


def test_no_rows():
    c = K.make(1, [5, 9], 4, H=1, dim=64)
    check_map(c, [0, 0], 0, 0)
    check_map(c, [3, 4], 0, 0)
    check_map(c, [0, -1], 0, 7)


@pytest.mark.parametrize("S,T,page,tree", [(1, 1, 32, False), (3, 5, 32, False), (5, 300, 64, False), (1, 1, 32, True), (3, 32, 32, True),
                                           (9, 7, 64, True), (17, 17, 128, True), (40, 2, 32, True)])
def test_dense_rows(S, T, page, tree):
    C.say(f"kv_row_map dense S={S} T={T} page={page} tree={tree}")
    rng = np.random.default_rng(S + T)
    c = K.make(T, list(rng.integers(0, 90, S)), T, page=page, H=1, dim=64)
    parent = trees(rng, S, T) if tree else None
    check_map(c, [T] * S, T, S * T, parent)
    n = rng.integers(-1, T + 3, S)
    c["refs"][c["table"][S // 3, -3 % c["table"].shape[1]]] = 2
    if tree and T > 4:
        parent[S // 2, T // 2] = T // 2          # not before itself
        parent[-1, 0] = 0                        # a root with a parent
        parent[0, T - 1] = 2 ** 30
    check_map(c, n, T, S * T, parent)


# --------------------------------------------------------------------- rope
def rope_case(lens, n, H, G, dim, rot, page, x, q, kind, inter, seed, L=2, amplitude=1.25):
    rng = np.random.default_rng(seed)
    c = K.make(seed, lens, max(n) if n else 1, L=L, H=H, dim=dim, page=page)
    fill(c, rng, kind)
    cache = K.to_library(svg, c, kind)
    R, A = sum(n) + 3, H * G                         # three rows of no slot behind them
    rows = svg.RowMap.empty(cache, R)
    svg.kv_row_map(cache, i32(n), rows)
    mat = torch.from_numpy(rng.standard_normal((R, (A + 2 * H) * dim + 8)).astype(np.float32)).to(TYPES[x])
    d = mat.to(C.DEV)
    parts = lambda m: (m[:, :A * dim].unflatten(1, (A, dim)) if A else None, m[:, A * dim:(A + H) * dim],  # noqa: E731
                       m[:, (A + H) * dim:(A + 2 * H) * dim])
    freq = 500000.0 ** -(np.arange(0, rot, 2) / rot)
    rope = svg.Rope(C.to_dev(freq), interleaved=inter, amplitude=amplitude)
    out = torch.full((R, A, dim), 7.0, dtype=TYPES[q], device=C.DEV)
    return c, cache, rows, rope, freq, parts(d), parts(mat), out


def check_rope(c, cache, rows, rope, freq, host_parts, out, kind, layer, inter, amplitude=1.25):
    q, k, v = host_parts
    dim, H = c["dim"], c["k"].shape[2]
    pos, place = C.host(rows.pos), C.host(rows.place)
    if q is not None:
        ref, size = PO.rope(q.float().numpy(), pos, freq, inter, amplitude)
        got = host64(out)
        live = pos >= 0
        form = next(n for n, t in TYPES.items() if t == out.dtype)
        assert np.all(np.abs(got - ref)[live] <= (6 * E * size * (1 + U[form]) + half_step(form, ref))[live])
        assert np.all(got[~live] == 7.0)
    ref, size = PO.rope(k.float().numpy().reshape(len(pos), H, dim), pos, freq, inter, amplitude)
    u = U[kind]
    before = {n: c[n].copy() for n in ("k", "v")}
    PO.write(c, layer, place, np.zeros((len(pos), H, dim), np.int16), K.bits(v.to(TYPES[kind])).reshape(len(pos), H, dim))
    assert np.array_equal(K.bits(cache.v), c["v"])
    got = K.bits(cache.k)
    d = np.arange(dim)
    for r in np.flatnonzero(place >= 0):
        p, t = place[r] // c["page"], place[r] % c["page"]
        at = CO.key_at(t, d, dim)
        y = wide(kind)(got[layer, p][:, at])
        assert np.all(np.abs(y - ref[r]) <= 6 * E * size[r] * (1 + u) + half_step(kind, ref[r])), r
        got[layer, p][:, at] = before["k"][layer, p][:, at]
    assert np.array_equal(got, before["k"])          # and nothing else was written


ROPE = [  # lens, new rows, H, G, dim, rot, page, x, q, kind, interleaved
    ([0], [1], 1, 1, 64, 64, 32, "fp32", "fp32", "fp16", False), ([5, 0, 33], [3, 4, 1], 2, 4, 128, 128, 64, "fp32", "fp32", "fp16", False),
    ([30, 100], [70, 37], 2, 2, 64, 32, 32, "bf16", "bf16", "bf16", True), ([31], [130], 1, 7, 256, 64, 128, "fp16", "fp16", "fp16", False),
    ([2, 1, 3], [33, 0, 64], 3, 1, 128, 48, 32, "fp16", "fp32", "bf16", True), ([60000], [5], 8, 4, 128, 128, 64, "bf16", "bf16", "bf16", False),
    ([7] * 40, [1] * 40, 2, 0, 64, 16, 32, "fp32", "fp32", "fp16", False), ([17, 4], [200, 100], 32, 1, 64, 64, 64, "fp32", "fp16", "fp16", True),
]


@pytest.mark.parametrize("lens,n,H,G,dim,rot,page,x,q,kind,inter", ROPE)
def test_rope_append(lens, n, H, G, dim, rot, page, x, q, kind, inter):
    C.say(f"rope_append lens={lens[:4]} n={n[:4]} H={H} G={G} dim={dim} rot={rot} {x} {q} {kind} interleaved={inter}")
    c, cache, rows, rope, freq, dev, hostp, out = rope_case(lens, n, H, G, dim, rot, page, x, q, kind, inter, dim + rot)
    svg.rope_append(cache, 1, rows, rope, dev[0], dev[1], dev[2], out if G else None)
    check_rope(c, cache, rows, rope, freq, hostp, out, kind, 1, inter)


def test_rope_of_trees_and_rows_without_a_place():
    """Positions of a tree are depths; a refused slot's queries are turned and its rows passed over."""
    S, T, H, dim = 3, 9, 2, 64
    rng = np.random.default_rng(5)
    c = K.make(8, [40, 3, 60], T, L=1, H=H, dim=dim, page=32)
    c["refs"][c["table"][1, 0]] = 2
    fill(c, rng, "fp16")
    cache = K.to_library(svg, c)
    parent = trees(rng, S, T)
    parent[2, 4] = 4
    rows = svg.RowMap.empty(cache, S * T)
    svg.kv_row_map(cache, i32([T, T, T]), rows, T=T, parent=i32(parent))
    pos, place = C.host(rows.pos), C.host(rows.place)
    assert (pos[T:2 * T] >= 0).all() and (place[T:2 * T] < 0).all() and (pos[2 * T:] < 0).any()
    x = torch.from_numpy(rng.standard_normal((S * T, 4 * H * dim)).astype(np.float32))
    d = x.to(C.DEV)
    cut = lambda m: (m[:, :2 * H * dim].unflatten(1, (2 * H, dim)), m[:, 2 * H * dim:3 * H * dim], m[:, 3 * H * dim:])  # noqa: E731
    freq = 100.0 ** -(np.arange(0, dim, 2) / dim)
    out = torch.full((S * T, 2 * H, dim), 7.0, device=C.DEV)
    rope = svg.Rope(C.to_dev(freq))
    svg.rope_append(cache, 0, rows, rope, *cut(d), out)
    check_rope(c, cache, rows, rope, freq, cut(x), out, "fp16", 0, False, amplitude=1.0)


def test_rope_places_outside_the_cache_are_passed_over():
    c, cache, rows, rope, freq, dev, hostp, out = rope_case([3], [6], 1, 1, 64, 64, 32, "fp32", "fp32", "fp16", False, 3)
    last = cache.n_pages * 32
    bad = i32([last, 2 ** 31 - 1, last + 5, -1, -2 ** 31, last - 1, -1, -1, -1])
    rows.place.copy_(bad)
    svg.rope_append(cache, 0, rows, rope, *dev, out)
    rows.place.copy_(i32([-1, -1, -1, -1, -1, last - 1, -1, -1, -1]))
    check_rope(c, cache, rows, rope, freq, hostp, out, "fp16", 0, False)


def test_rope_at_far_positions():
    """Positions to 2^31 - 1: angles of 2e9 radians."""
    c, cache, rows, rope, freq, dev, hostp, out = rope_case([3], [6], 2, 2, 64, 64, 32, "fp32", "fp32", "fp16", True, 4)
    rows.pos.copy_(i32([2 ** 31 - 1, 2 ** 31 - 2, 10 ** 9 + 7, 2 ** 25, 123456789, 0, -1, -1, -1]))
    svg.rope_append(cache, 1, rows, rope, *dev, out)
    check_rope(c, cache, rows, rope, freq, hostp, out, "fp16", 1, True)


# ---------------------------------------------------------------- attention
def attention_bound(c, kind, ref, size, most):
    u, dim = U[kind], c["dim"]
    e = 2 * (dim + 8) * E * size[..., 0:1] + 2.0 ** -20
    a = np.abs(np.nan_to_num(ref))
    return ((e + u) * (size[..., 2:3] + a) + size[..., 1:2] * ((most / 32 + 64) * E + most * 2.0 ** -33)) * (1 + u) + half_step(kind, a)


def check_attention(c, kind, q, qd, start, count, scale=None, layer=0, cache=None, workspace=None, before=7.0):
    R, A, dim = qd.shape
    cache = cache or K.to_library(svg, c, kind)
    guard = 256
    buf = torch.full((R * A * dim + 2 * guard,), before, dtype=TYPES[kind], device=C.DEV)
    out = buf[guard:-guard].view(R, A, dim)
    rows = svg.RowMap(i32(start), i32(count), n_rows=R)
    ws = svg.prompt_attention_workspace(cache, A, R) if workspace is None else workspace
    ws.fill_(0xFF)
    svg.prompt_attention(cache, layer, rows, qd, out, ws, scale=scale)
    assert bool((buf[:guard] == before).all()) and bool((buf[-guard:] == before).all())
    got = host64(out)
    ref, mine, size = PO.attention(c, wide(kind), layer, host64(qd), start, count, dim ** -0.5 if scale is None else scale)
    assert np.all(got[~mine] == before)
    bad = np.isnan(ref)
    assert np.array_equal(np.isnan(got)[mine], bad[mine])
    most = int(max(c["len"])) + int(max(count))
    tol = attention_bound(c, kind, ref, size, most)
    err = np.where(bad, 0, np.abs(got - np.nan_to_num(ref)))
    assert np.all(err[mine] <= tol[mine]), float((err / np.maximum(tol, 1e-300))[mine].max())
    return got


def queries(rng, R, A, dim, kind, size=1.0):
    """Rows as slices of a wider matrix."""
    x = rng.standard_normal((R, (A + 1) * dim)).astype(np.float32) * np.float32(size)
    x[:, :A * dim] *= np.repeat(np.linspace(0.3, 3.0, A), dim).astype(np.float32)
    d = torch.from_numpy(x).to(TYPES[kind]).to(C.DEV)
    return x, d[:, :A * dim].unflatten(1, (A, dim))


def packed(n):
    return list(np.cumsum([0] + list(n[:-1]))), list(n)


ATT = [  # lens, new rows, H, G, dim, page, kind
    ([0], [1], 1, 1, 64, 32, "fp16"), ([0], [130], 2, 1, 64, 32, "bf16"), ([1], [33], 1, 3, 128, 64, "fp16"),
    ([31], [2], 2, 4, 128, 32, "bf16"), ([32], [65], 1, 7, 64, 64, "fp16"), ([500, 0, 3, 64], [40, 129, 0, 1], 2, 2, 64, 32, "bf16"),
    ([100, 33, 257], [5, 77, 20], 1, 8, 256, 32, "bf16"), ([0, 10], [70, 64], 2, 1, 256, 128, "fp16"),
    ([2000], [17], 2, 5, 128, 128, "bf16"), ([(37 * s) % 300 for s in range(50)], [1 + (s % 5 == 0) * 9 for s in range(50)], 2, 4, 64, 32, "fp16"),
    ([9] * 300, [1] * 300, 1, 1, 64, 32, "bf16"), ([700], [300], 1, 12, 64, 64, "fp16"), ([3000], [1], 1, 1, 128, 64, "fp16"),
    ([0], [600], 1, 2, 128, 32, "bf16"), ([1024, 2], [31, 260], 1, 16, 64, 32, "bf16"),
]


@pytest.mark.parametrize("lens,n,H,G,dim,page,kind", ATT)
def test_attention(lens, n, H, G, dim, page, kind):
    C.say(f"prompt_attention lens={lens[:4]} n={n[:4]} H={H} G={G} dim={dim} page={page} {kind}")
    rng = np.random.default_rng(dim + len(lens) + G)
    c = K.make(dim + H, lens, max(n), L=2, H=H, dim=dim, page=page)
    fill(c, rng, kind)
    q, qd = queries(rng, sum(n) + 2, H * G, dim, kind)
    start, count = packed(n)
    check_attention(c, kind, q[:, :H * G * dim].reshape(-1, H * G, dim), qd, start, count, layer=1)


def test_attention_of_many_short_items():
    """Shares of many items, which go over heads, slots and slots without rows."""
    rng = np.random.default_rng(17)
    lens, n = rng.integers(0, 120, 200).tolist(), rng.integers(0, 13, 200).tolist()
    n[3:9], n[-1] = [0] * 6, 0
    c = K.make(3, lens, max(n), H=8, dim=64, page=32)
    fill(c, rng, "fp16")
    q, qd = queries(rng, sum(n), 8, 64, "fp16")
    check_attention(c, "fp16", q[:, :8 * 64].reshape(-1, 8, 64), qd, *packed(n))


@pytest.mark.parametrize("lens,n,H,G,dim,page,kind", [([2100, 3300], [5000, 1200], 8, 4, 64, 32, "fp16"), ([4000], [2500], 8, 2, 128, 32, "bf16"),
                                                      ([2500, 0], [1500, 700], 8, 2, 256, 32, "bf16")])
def test_attention_of_long_items_of_one_slot(lens, n, H, G, dim, page, kind):
    """Shares that go on from item to item of a slot whose table row is longer than a wave looks up at once; the reference in
    64 bits on the device, with the oracle's formulas."""
    C.say(f"prompt_attention lens={lens} n={n} H={H} G={G} dim={dim} page={page} {kind}")
    rng = np.random.default_rng(dim)
    c = K.make(dim, lens, max(n), H=H, dim=dim, page=page)
    fill(c, rng, kind)
    R, A = sum(n), H * G
    qd = torch.from_numpy(rng.standard_normal((R, A, dim)).astype(np.float32)).to(C.DEV).to(TYPES[kind])
    start, count = packed(n)
    cache = K.to_library(svg, c, kind)
    out = torch.full_like(qd, 7.0)
    svg.prompt_attention(cache, 0, svg.RowMap(i32(start), i32(count), n_rows=R), qd, out, svg.prompt_attention_workspace(cache, A, R))
    f64 = lambda t: t.to(C.DEV, torch.float64)  # noqa: E731
    for s in range(len(n)):
        at = np.arange(lens[s] + n[s])
        pg = c["table"][s][at // page].astype(np.int64)
        t, d = (at % page)[:, None], np.arange(dim)[None, :]
        sees = torch.arange(len(at), device=C.DEV)[None, :] <= lens[s] + torch.arange(n[s], device=C.DEV)[:, None]
        for a in range(0, A, 3):
            h = a // G
            Kt, V = (f64(torch.from_numpy(wide(kind)(c[x][0, pg, h][np.arange(len(at))[:, None], f(t, d, dim)])))
                     for x, f in (("k", CO.key_at), ("v", CO.value_at)))
            x = f64(qd[start[s]:start[s] + n[s], a])
            w = Kt.T.contiguous()
            p = torch.softmax((dim ** -0.5 * (x @ w)).masked_fill(~sees, -np.inf), 1)
            ref = p @ V
            size = torch.stack(((dim ** -0.5 * (x.abs() @ w.abs())).masked_fill(~sees, 0).amax(1),
                                V.abs().amax(1).cummax(0).values[lens[s]:], (p @ V.abs()).amax(1)), 1)
            tol = attention_bound(c, kind, host64(ref), host64(size), len(at))
            assert np.all(np.abs(host64(out[start[s]:start[s] + n[s], a]) - host64(ref)) <= tol), (s, a)


def test_attention_of_rows_in_any_order():
    """Slots whose rows lie apart, in another order, dense with unused rows between, past the end."""
    rng = np.random.default_rng(4)
    c = K.make(5, [40, 0, 100, 7, 9], 40, H=2, dim=64, page=32)
    fill(c, rng, "fp16")
    q, qd = queries(rng, 60, 4, 64, "fp16")
    for start, count in (([30, 20, 0, 50, 45], [15, 9, 20, 10, 0]), ([-5, 70, 0, 58, 60], [3, 3, 4, 9, 1]), ([0, 12, 24, 36, 48], [12, 1, 0, 7, -4])):
        check_attention(c, "fp16", q[:, :256].reshape(-1, 4, 64), qd, start, count)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_tokens_that_no_row_sees_do_not_reach_it(kind):
    """NaN and infinities in everything behind each row: other slots' pages, the rest of the last page, later rows."""
    rng = np.random.default_rng(6)
    lens, n = [20, 64, 90], [50, 1, 37]
    c = K.make(9, lens, 64, H=1, dim=64, page=32)
    fill(c, rng, kind)
    clean = K.copy_of(c)
    bad = K.bits(torch.tensor([float("nan"), float("inf"), -float("inf")]).to(TYPES[kind]))
    own = np.zeros(len(c["refs"]) * 32, bool)
    for s in range(3):
        for t in range(lens[s] + n[s]):
            own[c["table"][s, t // 32] * 32 + t % 32] = True
    d = np.arange(64)
    for p in range(len(c["refs"])):
        for t in range(32):
            if not own[p * 32 + t]:
                c["k"][0, p][:, CO.key_at(t, d, 64)] = bad[(t + d) % 3]
                c["v"][0, p][:, CO.value_at(t, d, 64)] = bad[(t + d + 1) % 3]
    q, qd = queries(rng, sum(n), 2, 64, kind)
    start, count = packed(n)
    got = check_attention(c, kind, q, qd, start, count)
    assert np.array_equal(got, check_attention(clean, kind, q, qd, start, count))


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_numbers_that_are_not_finite_reach_the_rows_that_see_them(kind):
    rng = np.random.default_rng(7)
    base, n = 70, 60
    for what, pos in (("v", 100), ("v", 75), ("v", 3), ("k", 100), ("k", 3)):
        for value in (float("nan"), float("inf")):
            c = K.make(9, [base], n, H=1, dim=64, page=32)
            fill(c, rng, kind)
            clean = K.copy_of(c)
            d = 5
            at = (CO.value_at if what == "v" else CO.key_at)(pos % 32, d, 64)
            c[what][0, c["table"][0, pos // 32], 0, at] = K.bits(torch.tensor([value]).to(TYPES[kind]))[0]
            q, qd = queries(rng, n, 1, 64, kind)
            q64 = host64(qd)
            cache, rows = K.to_library(svg, c, kind), svg.RowMap(i32([0]), i32([n]), n_rows=n)
            out = torch.zeros((n, 1, 64), dtype=TYPES[kind], device=C.DEV)
            svg.prompt_attention(cache, 0, rows, qd, out, svg.prompt_attention_workspace(cache, 1, n))
            got = host64(out)
            ref, _, size = PO.attention(clean, wide(kind), 0, q64, [0], [n], 0.125)
            tol = attention_bound(clean, kind, ref, size, base + n)
            sees = np.arange(n) >= pos - base
            near = np.abs(got - ref) <= tol
            if what == "v":
                assert near[:, :, np.arange(64) != d].all() and near[~sees].all() and not np.isfinite(got[sees][:, :, d]).any()
            elif np.isnan(value):
                assert near[~sees].all() and np.isnan(got[sees]).all()
            else:                    # the score's sign is that of q's value: +infinity is NaN, -infinity leaves the token out
                up = q64[:, 0, d] > 0
                assert near[~sees].all() and np.isnan(got[sees & up]).all() and np.isfinite(got[sees & ~up]).all()


def test_pages_that_are_not_the_slots():
    rng = np.random.default_rng(8)
    lens, n = [40, 40, 40, 40, 33], [70, 70, 70, 10, 40]
    c = K.make(2, lens, 80, H=2, dim=64, page=32)
    fill(c, rng, "bf16")
    c["table"][0, 2] = 1 << 20           # positions 64 .. 95: rows from 24 on
    c["refs"][c["table"][1, 2]] = 2      # the same of the step's own
    c["table"][2, 0] = -1                # all rows
    c["pages"][3] = 1                    # not enough pages
    c["refs"][c["table"][4, 0]] = 2      # committed tokens in a page that others hold too are read
    q, qd = queries(rng, sum(n), 4, 64, "bf16")
    start, count = packed(n)
    got = check_attention(c, "bf16", q, qd, start, count)
    assert np.isfinite(got[:24]).all() and np.isnan(got[24:70]).all() and np.isfinite(got[220:]).all()


def test_scores_of_every_size():
    """Scales of zero and below, and scores far apart (the exponent's range, sums of one token)."""
    rng = np.random.default_rng(9)
    c = K.make(3, [300, 5], 40, H=1, dim=64, page=64)
    fill(c, rng, "fp16")
    q, qd = queries(rng, 45, 2, 64, "fp16")
    start, count = packed([40, 5])
    for scale in (0.0, -0.125, 1e-30, 3.0, 40.0):
        check_attention(c, "fp16", q, qd, start, count, scale=scale)


def test_equal_scores_over_many_tokens():
    """Flat rows over a long context: every probability counts the same."""
    rng = np.random.default_rng(10)
    for kind in ("fp16", "bf16"):
        c = K.make(3, [20000], 3, H=1, dim=64, page=128)
        fill(c, rng, kind)
        q, qd = queries(rng, 3, 2, 64, kind, size=1e-3)
        check_attention(c, kind, q, qd, [0], [3])


def test_workspaces_streams_and_graphs():
    """Two calls at once on streams of their own, and a captured one replayed over other lengths."""
    rng = np.random.default_rng(11)
    c = K.make(3, [900, 33], 50, H=2, dim=128, page=64)
    fill(c, rng, "bf16")
    cache = K.to_library(svg, c, "bf16")
    q, qd = queries(rng, 64, 8, 128, "bf16")
    rows = svg.RowMap(i32([0, 40]), i32([40, 24]), n_rows=64)
    outs = [torch.zeros((64, 8, 128), dtype=torch.bfloat16, device=C.DEV) for _ in range(3)]
    spaces = [svg.prompt_attention_workspace(cache, 8, 64) for _ in range(3)]
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for turn in range(10):
        for i in range(2):
            with torch.cuda.stream(side[i]):
                svg.prompt_attention(cache, 0, rows, qd, outs[i], spaces[i])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svg.prompt_attention(cache, 0, rows, qd, outs[2], spaces[2])
    for n in ([40, 24], [1, 0], [17, 20], [40, 24]):
        rows.count.copy_(i32(n))
        outs[2].fill_(7)
        g.replay()
        torch.cuda.synchronize()
        ref, mine, size = PO.attention(c, wide("bf16"), 0, host64(qd), [0, 40], n, 128 ** -0.5)
        got = host64(outs[2])
        assert np.all(got[~mine] == 7) and np.all((np.abs(got - ref) <= attention_bound(c, "bf16", ref, size, 950))[mine])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ------------------------------------------------------------------ linears
def codes(rng, M, Kd):
    q = np.clip(np.rint(rng.standard_normal((M, Kd)) * 35), -127, 127).astype(np.int8)
    q[0, ::7] = 127
    q[-1, ::3] = -127
    return q


def weights(rng, N, Kd, fmt, group):
    """Canonical arrays, the device storage, and fp64 (scales [N, groups], codes less zeros [N, K])."""
    if fmt == "w8":
        q = codes(rng, N, Kd)
        s = (rng.random(N) * 2e-3 + 1e-3).astype(np.float16)
        wq, ws, wz = svg.empty_weights(N, Kd, fmt, 0, C.DEV)
        svg.import_weights(C.to_dev(q), C.to_dev(s), None, fmt, 0, Kd, wq, ws)
        return wq, ws, wz, s.astype(np.float64)[:, None], q.astype(np.int64)
    ng = Kd // group
    q = rng.integers(0, 16, (N, Kd)).astype(np.uint8)
    z = rng.integers(0, 16, (N, ng)).astype(np.uint8)
    z[0], z[-1] = 0, 15
    s = (rng.random((N, ng)) * 2e-2 + 1e-2).astype(np.float16)
    packed_q = q[:, 0::2] | (q[:, 1::2] << 4)
    if fmt == "w4_z4":
        zp = np.zeros((N, (ng + 1) // 2), np.uint8)
        zp |= z[:, 0::2]
        zp[:, :ng // 2] |= z[:, 1::2] << 4
    else:
        zp = z.astype(np.float16)
    wq, ws, wz = svg.empty_weights(N, Kd, fmt, group, C.DEV)
    svg.import_weights(C.to_dev(packed_q), C.to_dev(s), C.to_dev(zp), fmt, group, Kd, wq, ws, wz)
    return wq, ws, wz, s.astype(np.float64), q.astype(np.int64) - np.repeat(z.astype(np.int64), group, 1)


def check_linear(M, N, Kd, fmt, group, y, seed=0):
    rng = np.random.default_rng(M * 7 + N + Kd + seed)
    wq, ws, wz, s, w = weights(rng, N, Kd, fmt, group)
    x = codes(rng, M, Kd)
    xs = (rng.random(M) * 1e-2 + 1e-4).astype(np.float32)
    xq = C.to_dev(NO.slab_codes(x).reshape(M, Kd))
    guard = 64
    buf = torch.full((M * N + 2 * guard,), 7.0, dtype=TYPES[y], device=C.DEV)
    out = buf[guard:-guard].view(M, N)
    if fmt == "w8":
        svg.w8a8_prompt_linear(xq, C.to_dev(xs), wq, ws, N, out)
    else:
        svg.w4a8_prompt_linear(xq, C.to_dev(xs), wq, ws, wz, fmt, group, N, out)
    assert bool((buf[:guard] == 7).all()) and bool((buf[-guard:] == 7).all())
    ng = s.shape[1]
    ref, size = np.zeros((M, N)), np.zeros((M, N))
    for g in range(ng):
        k = slice(g * (Kd // ng), (g + 1) * (Kd // ng))
        part = (x[:, k].astype(np.float64) @ w[:, k].astype(np.float64).T) * s[:, g]       # whole numbers below 2^53: exact
        ref += part
        size += np.abs(part)
    ref, size = ref * xs.astype(np.float64)[:, None], size * xs.astype(np.float64)[:, None]
    tol = (3 * E * np.abs(ref) if fmt == "w8" else (ng + 2) * E * size) * (1 + U[y]) + half_step(y, ref)
    got = host64(out)
    err = np.abs(got - ref)
    assert np.all(err <= tol * (1 + 1e-6)), float((err / np.maximum(tol, 1e-300)).max())
    return got


SIZES = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (16, 48, 128), (31, 100, 160), (32, 64, 512), (33, 130, 1024), (40, 300, 224), (64, 256, 2048),
         (65, 129, 96), (100, 40, 4096), (127, 513, 256), (128, 128, 128), (129, 257, 384), (256, 512, 640), (257, 33, 64), (300, 1000, 1056),
         (513, 260, 320), (1030, 70, 128)]


@pytest.mark.parametrize("M,N,Kd", SIZES)
def test_w8_linear(M, N, Kd):
    C.say(f"w8a8_prompt_linear M={M} N={N} K={Kd}")
    for y in ("fp32", "bf16", "fp16"):
        check_linear(M, N, Kd, "w8", 0, y)


@pytest.mark.parametrize("fmt", ["w4_z16", "w4_z4"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,Kd", SIZES)
def test_w4_linear(M, N, Kd, group, fmt):
    Kd = -(-Kd // group) * group
    C.say(f"w4a8_prompt_linear M={M} N={N} K={Kd} {fmt} g{group}")
    check_linear(M, N, Kd, fmt, group, ("fp32", "bf16", "fp16")[(M + N) % 3])


@pytest.mark.parametrize("M,N,Kd", [(300, 4100, 32), (300, 4101, 192), (449, 4099, 1056), (130, 12290, 96)])
def test_w8_linear_of_medium_sizes(M, N, Kd):
    for y in ("fp32", "bf16"):
        check_linear(M, N, Kd, "w8", 0, y)


@pytest.mark.parametrize("fmt", ["w4_z16", "w4_z4"])
@pytest.mark.parametrize("M,N,Kd,group", [(515, 4100, 32, 32), (260, 4099, 96, 32), (515, 4101, 64, 64), (321, 4112, 704, 64), (515, 4100, 128, 128),
                                          (400, 4097, 1152, 128), (200, 8211, 576, 64)])
def test_w4_linear_of_medium_sizes(M, N, Kd, group, fmt):
    for y in ("fp32", "fp16"):
        check_linear(M, N, Kd, fmt, group, y)


@pytest.mark.parametrize("M,N,Kd,fmt,group", [(1408, 12288, 1024, "w8", 0), (2561, 8200, 1056, "w8", 0), (1100, 8208, 1024, "w4_z16", 64),
                                              (1300, 4112, 4096, "w4_z4", 128)])
def test_linears_of_many_tiles(M, N, Kd, fmt, group):
    """More tiles than a round of workgroups has, rows past whole large tiles; the reference in 64 bits on the device."""
    C.say(f"prompt linear M={M} N={N} K={Kd} {fmt} group={group}")
    rng = np.random.default_rng(M)
    wq, ws, wz, s, w = weights(rng, N, Kd, fmt, group)
    x = codes(rng, M, Kd)
    xs = (rng.random(M) * 1e-2 + 1e-4).astype(np.float32)
    y = torch.full((M, N), 7.0, device=C.DEV)
    xq, xsd = C.to_dev(NO.slab_codes(x).reshape(M, Kd)), C.to_dev(xs)
    if fmt == "w8":
        svg.w8a8_prompt_linear(xq, xsd, wq, ws, N, y)
    else:
        svg.w4a8_prompt_linear(xq, xsd, wq, ws, wz, fmt, group, N, y)
    f64 = lambda t: torch.from_numpy(np.ascontiguousarray(t)).to(C.DEV).double()  # noqa: E731
    ng, ref, size = s.shape[1], 0, 0
    for g in range(ng):
        k = slice(g * (Kd // ng), (g + 1) * (Kd // ng))
        part = (f64(x[:, k]) @ f64(w[:, k].T)) * f64(s[:, g]) * f64(xs)[:, None]
        ref, size = ref + part, size + part.abs()
    tol = (3 if fmt == "w8" else ng + 2) * E * size * (1 + 1e-6)
    assert bool(((y.double() - ref).abs() <= tol).all())


def test_the_linears_of_both_kinds_agree():
    """The prompt linear on the rows of a verify batch: the verify linear's results."""
    rng = np.random.default_rng(3)
    for M, N, Kd in ((1, 64, 512), (16, 320, 1024), (32, 128, 2048)):
        x = C.to_dev(NO.slab_codes(codes(rng, M, Kd)).reshape(M, Kd))
        xs = C.to_dev((rng.random(M) * 1e-2).astype(np.float32))
        for fmt, group in (("w8", 0), ("w4_z16", 64), ("w4_z4", 128)):
            wq, ws, wz, _, _ = weights(rng, N, Kd, fmt, group)
            a, b = (torch.empty((M, N), device=C.DEV) for _ in range(2))
            if fmt == "w8":
                svg.w8a8_linear(x, xs, wq, ws, N, a)
                svg.w8a8_prompt_linear(x, xs, wq, ws, N, b)
            else:
                svg.w4a8_linear(x, xs, wq, ws, wz, fmt, group, N, a)
                svg.w4a8_prompt_linear(x, xs, wq, ws, wz, fmt, group, N, b)
            assert float((a - b).abs().max()) <= 1e-4 * float(a.abs().max())


def test_w8_rows_do_not_depend_on_the_number_of_rows():
    rng = np.random.default_rng(5)
    N, Kd, most = 272, 1088, 700
    wq, ws, wz, _, _ = weights(rng, N, Kd, "w8", 0)
    x, xs = codes(rng, most, Kd), (rng.random(most) * 1e-2).astype(np.float32)
    first = None
    for M in (most, 513, 300, 129, 128, 64, 33, 32, 5, 1):
        y = torch.empty((M, N), device=C.DEV)
        svg.w8a8_prompt_linear(C.to_dev(NO.slab_codes(x[:M]).reshape(M, Kd)), C.to_dev(xs[:M]), wq, ws, N, y)
        first = y if first is None else first
        assert torch.equal(y, first[:M]), M


def test_w8_rows_past_a_launch_of_few_columns():
    """2^23 and more rows of few columns: more tiles of rows than a launch has workgroups in its second dimension."""
    M, N, Kd = (1 << 23) + 131, 5, 32
    C.say(f"w8a8_prompt_linear M={M} N={N} K={Kd}")
    rng = np.random.default_rng(11)
    wq, ws, _, s, w = weights(rng, N, Kd, "w8", 0)
    g = torch.Generator(device=C.DEV).manual_seed(5)
    x = torch.randint(-127, 128, (M, Kd), dtype=torch.int8, device=C.DEV, generator=g)  # (with 32 codes a row, slabs are rows)
    xs = torch.rand(M, device=C.DEV, generator=g) * 1e-2 + 1e-4
    y = torch.full((M, N), 7.0, device=C.DEV)
    svg.w8a8_prompt_linear(x, xs, wq, ws, N, y)
    for at in range(0, M, 1 << 21):
        part = slice(at, min(at + (1 << 21), M))
        ref = (x[part].double() @ torch.from_numpy(w.T.copy()).to(C.DEV).double()) * torch.from_numpy(s[:, 0]).to(C.DEV) * xs[part, None].double()
        assert bool(((y[part].double() - ref).abs() <= 3 * E * ref.abs() * (1 + 1e-6)).all()), at



# --------------------------------------------------------------- gated rows
@pytest.mark.parametrize("M,Kd,block", [(1, 32, 32), (1, 4096, 64), (5, 96, 32), (31, 1024, 32), (33, 1088, 64), (64, 12288, 32), (70, 640, 64),
                                        (3, 32768, 64), (600, 2048, 32), (1030, 544, 32), (520, 5120, 32), (513, 12288, 64), (515, 9216, 32)])
@pytest.mark.parametrize("x_type", ["fp32", "fp16", "bf16"])
def test_gated_quant(M, Kd, block, x_type):
    C.say(f"gated_quant_i8 M={M} K={Kd} block={block} {x_type}")
    rng = np.random.default_rng(M + Kd)
    both = torch.from_numpy((rng.standard_normal((M, 2 * Kd)) * 2).astype(np.float32)).to(TYPES[x_type])
    both[:, Kd:][:, ::37] *= 30
    both[0, :min(Kd, 8)] = torch.tensor([0.0, -0.0, 100.0, -100.0, 3e4, -3e4, 1e-6, -20.0]).to(both.dtype)
    both[M // 2] = 0
    signs = np.where(rng.integers(0, 2, Kd) == 1, 1, -1).astype(np.int8)
    d, sd = both.to(C.DEV), C.to_dev(signs)
    for gate in (True, False):
        xq = torch.full((M, Kd), 99, dtype=torch.int8, device=C.DEV)
        xs = torch.full((M,), 7.0, device=C.DEV)
        svg.gated_quant_i8(d[:, Kd:], d[:, :Kd] if gate else None, sd, xq, xs, block=block)
        x = both.float().numpy()
        q, s = PO.gated_quant(x[:, Kd:], x[:, :Kd] if gate else None, signs, block)
        assert np.array_equal(C.host(xs), s)
        assert np.array_equal(C.host(xq).reshape(-1), NO.slab_codes(q))


def test_gated_rows_are_the_norms_rows():
    """Without a gate the codes are act_rht_quant_i8's."""
    x = torch.randn((17, 2048), device=C.DEV)
    signs = (torch.randint(0, 2, (2048,), device=C.DEV) * 2 - 1).to(torch.int8)
    a, b = (torch.empty((17, 2048), dtype=torch.int8, device=C.DEV) for _ in range(2))
    sa, sb = (torch.empty(17, device=C.DEV) for _ in range(2))
    svg.act_rht_quant_i8(x, signs, a, sa)
    svg.gated_quant_i8(x, None, signs, b, sb)
    assert torch.equal(a, b) and torch.equal(sa, sb)


# ------------------------------------------------------------------ refusals
def test_binding_refusals():
    c = K.make(1, [5, 9], 8, H=2, dim=64)
    cache = K.to_library(svg, c)
    rows = svg.RowMap.empty(cache, 10)
    f = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device=C.DEV)  # noqa: E731
    rope = svg.Rope.make(64, device=C.DEV)
    q, k, v, out = f(10, 4, 64), f(10, 128), f(10, 2, 64), f(10, 4, 64)
    svg.rope_append(cache, 0, rows, rope, q, k, v, out)
    n = i32([1, 2])
    h = torch.float16
    bad = [
        (ValueError, lambda: svg.kv_row_map(cache, n[:1], rows)), (TypeError, lambda: svg.kv_row_map(cache, n.long(), rows)),
        (ValueError, lambda: svg.kv_row_map(cache, n, rows, T=4, parent=i32(np.zeros((2, 3))))), (svg.SvgError, lambda: svg.kv_row_map(cache, n, rows, T=4)),
        (ValueError, lambda: svg.RowMap(n, n)), (ValueError, lambda: svg.RowMap(n, n, rows.pos)), (TypeError, lambda: svg.RowMap(n.float(), n, n_rows=1)),
        (ValueError, lambda: svg.RowMap(n, n, rows.pos, rows.place, n_rows=9)), (ValueError, lambda: svg.RowMap(n.cpu(), n.cpu(), n_rows=1)),
        (ValueError, lambda: svg.kv_row_map(cache, n, svg.RowMap(n, n, n_rows=3))), (TypeError, lambda: svg.Rope(f(32))),
        (ValueError, lambda: svg.rope_append(cache, 0, rows, rope, q[:9], k, v, out)), (ValueError, lambda: svg.rope_append(cache, 0, rows, rope, q, k[:9], v, out)),
        (TypeError, lambda: svg.rope_append(cache, 0, rows, rope, q.half(), k, v, out)), (TypeError, lambda: svg.rope_append(cache, 0, rows, rope, q, k, v.half(), out)),
        (TypeError, lambda: svg.rope_append(cache, 0, rows, rope, q, k, v, out.bfloat16())), (ValueError, lambda: svg.rope_append(cache, 0, rows, rope, q, k, v)),
        (ValueError, lambda: svg.rope_append(cache, 0, rows, rope, q, f(10, 256)[:, ::2], v, out)),
        (svg.SvgError, lambda: svg.rope_append(cache, 0, rows, svg.Rope.make(128, device=C.DEV), q, k, v, out)),
        (svg.SvgError, lambda: svg.rope_append(cache, 1, rows, rope, q, k, v, out)),
        (TypeError, lambda: svg.prompt_attention(cache, 0, rows, q, out, svg.prompt_attention_workspace(cache, 4, 10))),
        (ValueError, lambda: svg.prompt_attention(cache, 0, rows, f(10, 4, 64, t=h), f(10, 4, 64, t=h), f(16, t=torch.uint8))),
        (ValueError, lambda: svg.prompt_attention(cache, 0, rows, f(9, 4, 64, t=h), f(9, 4, 64, t=h), svg.prompt_attention_workspace(cache, 4, 10))),
        (svg.SvgError, lambda: svg.prompt_attention(cache, 0, rows, f(10, 3, 64, t=h), f(10, 3, 64, t=h), f(16, t=torch.uint8))),
        (svg.SvgError, lambda: svg.prompt_attention_workspace(cache, 3, 10)),
        (ValueError, lambda: svg.gated_quant_i8(f(4, 64), f(4, 32), f(64, t=torch.int8), f(4, 64, t=torch.int8), f(4))),
        (TypeError, lambda: svg.gated_quant_i8(f(4, 64), f(4, 64, t=h), f(64, t=torch.int8), f(4, 64, t=torch.int8), f(4))),
        (ValueError, lambda: svg.gated_quant_i8(f(4, 64), None, f(32, t=torch.int8), f(4, 64, t=torch.int8), f(4))),
        (svg.SvgError, lambda: svg.gated_quant_i8(f(4, 48), None, f(48, t=torch.int8), f(4, 48, t=torch.int8), f(4))),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()
    wq, ws, _ = svg.empty_weights(64, 128, "w8", 0, C.DEV)
    x, xs, y = f(40, 128, t=torch.int8), f(40), f(40, 64)
    for error, call in [(ValueError, lambda: svg.w8a8_prompt_linear(x, xs, wq[:100], ws, 64, y)), (ValueError, lambda: svg.w8a8_prompt_linear(x, xs, wq, ws, 65, y)),
                        (TypeError, lambda: svg.w8a8_prompt_linear(x, xs, wq, ws, 64, y.double())), (ValueError, lambda: svg.w8a8_prompt_linear(x, xs[:9], wq, ws, 64, y)),
                        (TypeError, lambda: svg.w8a8_prompt_linear(x.float(), xs, wq, ws, 64, y)), (ValueError, lambda: svg.w8a8_prompt_linear(x, xs, wq.cpu(), ws, 64, y))]:
        with pytest.raises(error):
            call()
    none = f(0, 128, t=torch.int8)
    svg.w8a8_prompt_linear(none, f(0), wq, ws, 64, f(0, 64))
    svg.gated_quant_i8(f(0, 64), None, f(64, t=torch.int8), f(0, 64, t=torch.int8), f(0))
