"""Edges of a prompt's operators: scores and values far from ordinary ones, buffers that are replaced, every kernel of the
linears, sizes at the limits.  Tolerances by the number formats as in tests/test_prompt_parity.py (u, e and half_step)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache_oracle as CO
from oracle import norm_oracle as NO
from oracle import prompt_oracle as PO

E = 2.0 ** -24


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    global C, K, P, svg
    import cache_cases as K  # noqa: F401
    import svg_cases as C  # noqa: F401
    import test_prompt_parity as P  # noqa: F401
    import speculative_verify_gemm_amd as svg
    P.svg, P.C, P.K = svg, C, K


# ---------------------------------------------------------------- attention
def attend(c, kind, q, start, count, scale):
    """(out fp64, the queries as the device has them)."""
    R, A, _ = q.shape
    qd = torch.from_numpy(q.astype(np.float32)).to(P.TYPES[kind]).to(C.DEV)
    cache, rows = K.to_library(svg, c, kind), svg.RowMap(P.i32(start), P.i32(count), n_rows=R)
    out = torch.full_like(qd, 7.0)
    svg.prompt_attention(cache, 0, rows, qd, out, svg.prompt_attention_workspace(cache, A, R), scale=scale)
    return P.host64(out), P.host64(qd)


def tokens(c, kind, s, n, head=0):
    """Keys and values of slot s's first n tokens, fp64."""
    at = np.arange(n)
    pg, t, d = c["table"][s][at // c["page"]].astype(np.int64), (at % c["page"])[:, None], np.arange(c["dim"])[None, :]
    return tuple(P.wide(kind)(c[x][0, pg, head][at[:, None], f(t, d, c["dim"])]) for x, f in (("k", CO.key_at), ("v", CO.value_at)))


def put(c, kind, name, s, values, head=0):
    """Values [n, dim] as slot s's first n keys ("k") or values ("v")."""
    w = K.bits(torch.from_numpy(np.asarray(values, np.float32)).to(P.TYPES[kind]))
    d = np.arange(c["dim"])
    for t in range(len(values)):
        page, i = c["table"][s, t // c["page"]], t % c["page"]
        c[name][0, page, head][(CO.key_at if name == "k" else CO.value_at)(i, d, c["dim"])] = w[t]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("power", [4, 10, 14, 17, 20, 22, 24, 26, 30])
def test_scores_far_apart(gpu, power, dim, kind):
    """Scales of 2^power and -2^power.  A score is off by (dim + 8) e B at most, B = |scale| sum |q k|: where the best token leads by
    twice that and 40 more, the others together weigh less than 2^-49 and the row is that token's value: p v / p, two roundings of
    fp32 and the output's.  Any other row lies between the smallest and the largest value."""
    C.say(f"prompt_attention scale=2^{power} dim={dim} {kind}")
    rng = np.random.default_rng(power)
    lens, n = [300, 5, 900], [40, 5, 3]
    c = K.make(3, lens, max(n), H=1, dim=dim, page=64)
    P.fill(c, rng, kind)
    start, count = P.packed(n)
    q = rng.standard_normal((sum(n), 2, dim))
    for scale in (2.0 ** power, -2.0 ** power):
        got, q64 = attend(c, kind, q, start, count, scale)
        assert np.isfinite(got).all()
        clear = 0
        for s in range(len(n)):
            keys, v = tokens(c, kind, s, lens[s] + n[s])
            for i in range(n[s]):
                L = lens[s] + i + 1
                for a in range(2):
                    x, y = q64[start[s] + i, a], got[start[s] + i, a]
                    sc = scale * (keys[:L] @ x)
                    lead = 2 * (dim + 8) * E * abs(scale) * (np.abs(keys[:L]) @ np.abs(x)).max() + 40
                    best = int(sc.argmax())
                    if L == 1 or sc[best] - np.delete(sc, best).max() > lead:
                        clear += 1
                        big = np.abs(v[:L]).max()
                        assert np.all(np.abs(y - v[best]) <= P.half_step(kind, v[best]) + 4 * E * np.abs(v[best]) + 2.0 ** -48 * big), (s, i, a)
                    else:
                        low, high = v[:L].min(0), v[:L].max(0)
                        room = (L + 8) * E * np.abs(v[:L]).max()
                        assert np.all(y >= low - room - P.half_step(kind, low)) and np.all(y <= high + room + P.half_step(kind, high)), (s, i, a)
        assert power < 10 or clear >= 0.4 * 2 * sum(n)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("power", [0, 12, 15, 18, 21, 24, 25, 26, 27, 30])
def test_equal_scores_of_any_size(gpu, power, kind):
    """Every key is the same: all probabilities are one number, and the row is the mean of its values.  L products and their sums in
    fp32 are off by L e of the sum of the sizes, numerator and denominator each."""
    rng = np.random.default_rng(power)
    lens, n = [1000, 7], [40, 6]
    c = K.make(3, lens, max(n), H=1, dim=64, page=32)
    P.fill(c, rng, kind)
    key = rng.standard_normal(64)
    for s in range(2):
        put(c, kind, "k", s, np.repeat(key[None], lens[s] + n[s], 0))
    start, count = P.packed(n)
    for sign in (1, -1):
        got, _ = attend(c, kind, np.repeat(sign * key[None, None], sum(n), 0), start, count, 2.0 ** power)
        for s in range(2):
            v = tokens(c, kind, s, lens[s] + n[s])[1]
            for i in range(n[s]):
                L = lens[s] + i + 1
                ref, size = v[:L].mean(0), np.abs(v[:L]).mean(0)
                assert np.all(np.abs(got[start[s] + i, 0] - ref) <= (2 * L + 8) * E * size * 1.01 + P.half_step(kind, ref)), (sign, s, i)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("first", [2.0 ** 23, 2.0 ** 24, 2.0 ** 25, -2.0 ** 24, -2.0 ** 25])
def test_scores_that_just_pass_the_largest_so_far(gpu, first, kind):
    """Scores of 2^24 and 8 powers of two more behind them, where the steps of fp32 are 2 (and 4): the products of a score with scale and
    log2(e) are off by 3 steps of half an ulp together, so that the ratio of two probabilities is 2^8 within 2^-6 and 2^6 at 2^24, within
    2^12 at 2^25.  Values 0 for the first and 1 for the others; 128 of the one, 192 and more of the others."""
    rng = np.random.default_rng(3)
    ctx, n = 320, 20
    c = K.make(3, [ctx], n, H=1, dim=64, page=32)
    P.fill(c, rng, kind)
    later = np.arange(ctx + n) >= 128
    keys, q = np.zeros((ctx + n, 64)), np.zeros((n, 1, 64))
    q[..., 0], q[..., 1] = np.sign(first) * 2.0 ** 12, 1
    keys[:, 0], keys[:, 1] = abs(first) / 2.0 ** 12, 8 * later
    put(c, kind, "k", 0, keys)
    put(c, kind, "v", 0, np.repeat(later[:, None] * 1.0, 64, 1))
    got, _ = attend(c, kind, q, [0], [n], float(np.log(2.0)))
    ulp = max(1.0, abs(first) * 2.0 ** -23)
    ratio = 2.0 ** (8 - 3 * ulp) * 193 / 128
    assert np.isfinite(got).all()
    assert np.all(got >= ratio / (1 + ratio) * (1 - 2 * P.U[kind])) and np.all(got <= 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("exponent", [127, 120, 113, 100, -60, -85, -100, -110, -126])
def test_values_of_any_size_in_a_bf16_cache(gpu, exponent, dim):
    """Values of up to 2^exponent (127: bf16's largest number): a row is a mean of values, so it is finite.  Accumulators end at 2^-149 and
    the probabilities at 2^-33 or more for the largest: a rounding there is off by 2^-149 / 2^-33, and there is one for each of up to
    L products and the joins."""
    rng = np.random.default_rng(exponent + 130)
    lens, n = [1500, 0, 70], [30, 40, 1]
    c = K.make(3, lens, max(n), H=1, dim=dim, page=64)
    P.fill(c, rng, "bf16")
    largest = float(torch.finfo(torch.bfloat16).max)
    for s in range(3):
        size = rng.random((lens[s] + n[s], dim)) * 0.5 + 0.5
        size[::7] = 1.0
        sign = np.where(rng.random(size.shape) < 0.9, 1.0, -1.0) if s else 1.0
        put(c, "bf16", "v", s, np.clip(np.ldexp(size, exponent + (exponent == 127)), 0, largest) * sign)
    start, count = P.packed(n)
    for spread in (1e-3, 1.0, 30.0):
        got, q64 = attend(c, "bf16", rng.standard_normal((sum(n), 2, dim)), start, count, spread / dim ** 0.5)
        assert np.isfinite(got).all()
        ref, _, size = PO.attention(c, P.wide("bf16"), 0, q64, start, count, spread / dim ** 0.5)
        tol = P.attention_bound(c, "bf16", ref, size, 1530) + 1600 * 2.0 ** (-149 + 33)
        assert np.all(np.abs(got - ref) <= tol), float((np.abs(got - ref) / tol).max())



@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_queries_that_are_not_finite(gpu, value, kind):
    """A row whose query is not finite is NaN; every other row is, bit for bit, what it is without that."""
    rng = np.random.default_rng(3)
    lens, n = [200, 7], [30, 20]
    c = K.make(3, lens, max(n), H=2, dim=64, page=32)
    P.fill(c, rng, kind)
    start, count = P.packed(n)
    q = rng.standard_normal((sum(n), 6, 64))
    clean, _ = attend(c, kind, q, start, count, 0.125)
    at = [(0, 0), (7, 3), (29, 5), (33, 1)]
    for r, a in at:
        q[r, a, 11] = value
    got, _ = attend(c, kind, q, start, count, 0.125)
    for r, a in at:
        assert np.isnan(got[r, a]).all() or np.isinf(value)      # (an infinite one may leave tokens out: their scores are -infinity)
        got[r, a] = clean[r, a]
    assert np.array_equal(got, clean)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_tokens_that_are_left_out(gpu, kind):
    """Keys that give scores of -infinity: the first 150 of 400 for every row, then all that some rows see (NaN)."""
    rng = np.random.default_rng(5)
    lens, n = [400, 0], [40, 37]
    c = K.make(3, lens, max(n), H=1, dim=64, page=32)
    P.fill(c, rng, kind)
    keys, _v = tokens(c, kind, 0, 440)
    keys[:150, 9] = -np.inf
    put(c, kind, "k", 0, keys)
    keys, _v = tokens(c, kind, 1, 37)
    keys[:20, 9] = -np.inf
    put(c, kind, "k", 1, keys)
    q = rng.standard_normal((77, 2, 64))
    q[..., 9] = 1.0
    start, count = P.packed(n)
    got, q64 = attend(c, kind, q, start, count, 0.125)
    for s, first in ((0, 150), (1, 20)):
        keys, v = tokens(c, kind, s, lens[s] + n[s])
        for i in range(n[s]):
            L = lens[s] + i + 1
            for a in range(2):
                y = got[start[s] + i, a]
                if L <= first:
                    assert np.isnan(y).all(), (s, i, a)
                    continue
                x = q64[start[s] + i, a]
                w = np.exp(0.125 * (keys[first:L] @ x))
                w /= w.sum()
                size = np.array([0.125 * (np.abs(keys[first:L]) @ np.abs(x)).max(), np.abs(v[:L]).max(), (w @ np.abs(v[first:L])).max()])
                ref = w @ v[first:L]
                assert np.all(np.abs(y - ref) <= P.attention_bound(c, kind, ref, size, L)), (s, i, a)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_pages_past_32_bits(gpu, kind):
    """A pool of 8 GiB of keys and as many of values: what its last pages give is what the same pages of a small pool give."""
    H, dim, page, ctx, n, many = 8, 128, 128, 500, 300, 2 ** 15 + 3
    C.say(f"rope_append, prompt_attention: {many} pages of {H * page * dim * 2} bytes {kind}")
    held = -(-(ctx + n) // page)
    rng = np.random.default_rng(3)
    ids = [many - 1, 5, 2 ** 14 + 1, many - 2, 2 ** 14, many - 9, 2 ** 13 + 1][:held]
    x = torch.from_numpy(rng.standard_normal((n, 3 * H, dim)).astype(np.float32)).to(P.TYPES[kind]).to(C.DEV)
    old = torch.from_numpy(rng.standard_normal((2, held, H, page * dim)).astype(np.float32)).to(P.TYPES[kind]).to(C.DEV)
    rope, got = svg.Rope.make(dim, device=C.DEV), []
    for pages, at in ((held, list(range(held))), (many, ids)):
        cache = svg.KVCache.empty(1, pages, H, dim, page, 1, held, dtype=P.TYPES[kind], device=C.DEV)
        where = torch.tensor(at, device=C.DEV)
        cache.k[0, where], cache.v[0, where] = old[0], old[1]
        cache.table.copy_(where[None]), cache.pages.fill_(held), cache.len.fill_(ctx)
        cache.refs[where] = 1
        rows = svg.RowMap.empty(cache, n)
        svg.kv_row_map(cache, P.i32([n]), rows)
        q, out = (torch.zeros((n, H, dim), dtype=P.TYPES[kind], device=C.DEV) for _ in range(2))
        svg.rope_append(cache, 0, rows, rope, x[:, :H], x[:, H:2 * H], x[:, 2 * H:], q)
        svg.prompt_attention(cache, 0, rows, q, out, svg.prompt_attention_workspace(cache, H, n))
        got.append((cache.k[0, where], cache.v[0, where], q, out))
        del cache
    torch.cuda.empty_cache()
    assert bool(torch.isfinite(got[0][3].float()).all())
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_rows_that_lie_gigabytes_apart(gpu):
    """Row strides of 2^30 bytes: a call's rows are those of a compact copy."""
    M, ld, H, dim = 5, 2 ** 29 + 64, 1, 64
    C.say(f"strides of {2 * ld} bytes")
    wide = torch.empty(M * ld, dtype=torch.float16, device=C.DEV).view(M, ld)
    part = wide[:, 8:8 + 6 * dim]
    part.copy_(torch.randn((M, 6 * dim), device=C.DEV))
    assert part.stride(0) == ld
    signs = (torch.randint(0, 2, (2 * dim,), device=C.DEV) * 2 - 1).to(torch.int8)
    c = K.make(3, [40], M, H=H, dim=dim, page=32)
    P.fill(c, np.random.default_rng(1), "fp16")
    rope, got = svg.Rope.make(dim, device=C.DEV), []
    for x in (part, part.contiguous()):
        cache = K.to_library(svg, c)
        rows = svg.RowMap.empty(cache, M)
        svg.kv_row_map(cache, P.i32([M]), rows)
        q, k, v = x[:, :4 * dim].unflatten(1, (4, dim)), x[:, 4 * dim:5 * dim], x[:, 5 * dim:]
        turned, out = (torch.zeros((M, 4, dim), dtype=torch.float16, device=C.DEV) for _ in range(2))
        svg.rope_append(cache, 0, rows, rope, q, k, v, turned)
        svg.prompt_attention(cache, 0, rows, q, out, svg.prompt_attention_workspace(cache, 4, M))
        codes, scale = torch.zeros((M, 2 * dim), dtype=torch.int8, device=C.DEV), torch.zeros(M, device=C.DEV)
        svg.gated_quant_i8(x[:, :2 * dim], x[:, 2 * dim:4 * dim], signs, codes, scale)
        got.append((turned, out, codes, scale, cache.k, cache.v))
    del wide, part
    torch.cuda.empty_cache()
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ linears
FEW, SMALL, MID, BIG = range(4)
ROWS, COLS = {FEW: 100, SMALL: 300, MID: 1001, BIG: 1150}, {FEW: 515, SMALL: 4091, MID: 4091, BIG: 8187}


def linear_cases():
    """(format, group, ways as svg_prompt_linear_choice has them, M, N, K, y): every kernel, of 1 to 3 steps of K, of one more than the
    ring has places, with a rest of K; odd numbers of columns, and whole tiles (stored four values at a time); more than one
    tile for a workgroup; every type of output."""
    cases = []
    types = ("fp32", "bf16", "fp16")

    def add(fmt, group, way, M, N, K, then=None):
        ways = (way, M if then is None else M & ~255, -1 if then is None else then)
        for y in (types if way == BIG or (K > 500 and way != FEW) else (types[len(cases) % 3],)):
            cases.append((fmt, group, ways, M, N, K, y))

    for way in (FEW, SMALL, MID, BIG):
        for K in (32, 64, 96, 192, 256, 320, 1056):
            add("w8", 0, way, ROWS[way], COLS[way], K)
    for way, M, N in ((SMALL, 320, 4096), (MID, 1024, 4096), (BIG, 1280, 12288)):
        for K in (32, 160, 640):
            add("w8", 0, way, M, N, K)
    add("w8", 0, MID, 2049, 3010, 96)
    add("w8", 0, BIG, 1283, 12277, 1056, FEW)
    add("w8", 0, BIG, 2304, 12288, 320)
    for fmt in ("w4_z16", "w4_z4"):
        for group in (32, 64, 128):
            for way in (FEW, SMALL, MID):
                for K in (group, 128 + group, 256 + group, 384, 1024 + group):
                    add(fmt, group, way, ROWS[way], COLS[way], K)
            add(fmt, group, SMALL, 320, 4096, 512)
            add(fmt, group, MID, 1024, 4096, 512 + group)
            add(fmt, group, MID, 1921, 4091 if group == 32 else 8187, 256 + group)
    return cases


def choice(lib, fmt, group, M, N, K, cus):
    import ctypes
    got = (ctypes.c_int32 * 3)()
    lib.svg_prompt_linear_choice({"w4_z4": 0, "w4_z16": 1, "w8": 2}[fmt], group, M, N, K, cus, got)
    return tuple(got)


def test_the_sizes_take_every_kernel_of_the_linears():
    """The rule on 256 compute units, on the host: each case takes the kernel that it names, and all kernels of all formats are taken."""
    import speculative_verify_gemm_amd as lib
    taken = set()
    for fmt, group, ways, M, N, K, y in linear_cases():
        assert choice(lib.lib, fmt, group, M, N, K, 256) == ways, (fmt, group, M, N, K)
        taken |= {(fmt, group, w, y) for w in ways[::2] if w >= 0}
    for fmt, group in [("w8", 0)] + [(f, g) for f in ("w4_z16", "w4_z4") for g in (32, 64, 128)]:
        for way in (FEW, SMALL, MID) + ((BIG,) if fmt == "w8" else ()):
            types = {t[3] for t in taken if t[:3] == (fmt, group, way)}
            assert types == {"fp32", "bf16", "fp16"} if way != FEW else types, (fmt, group, way, types)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,group,ways,M,N,K,y", linear_cases())
def test_every_kernel_of_the_linears(gpu, fmt, group, ways, M, N, K, y):
    """Against the formula in 64 bits on the device; bounds as in tests/test_prompt_parity.py."""
    C.say(f"prompt linear {fmt} group={group} ways={ways} M={M} N={N} K={K} {y}")
    cus = torch.cuda.get_device_properties(C.DEV).multi_processor_count
    assert choice(svg.lib, fmt, group, M, N, K, cus) == ways
    rng = np.random.default_rng(M * 7 + N + K)
    wq, ws, wz, s, w = P.weights(rng, N, K, fmt, group)
    x = P.codes(rng, M, K)
    xs = (rng.random(M) * 1e-2 + 1e-4).astype(np.float32)
    guard = 64
    buf = torch.full((M * N + 2 * guard,), 7.0, dtype=P.TYPES[y], device=C.DEV)
    out = buf[guard:-guard].view(M, N)
    xq, xsd = C.to_dev(NO.slab_codes(x).reshape(M, K)), C.to_dev(xs)
    if fmt == "w8":
        svg.w8a8_prompt_linear(xq, xsd, wq, ws, N, out)
    else:
        svg.w4a8_prompt_linear(xq, xsd, wq, ws, wz, fmt, group, N, out)
    f64 = lambda t: torch.from_numpy(np.ascontiguousarray(t)).to(C.DEV).double()  # noqa: E731
    xd, wd, sd, rows = f64(x), f64(w), f64(s), f64(xs)[:, None]
    ng, ref, size = s.shape[1], 0, 0
    for g in range(ng):
        k = slice(g * (K // ng), (g + 1) * (K // ng))
        part = (xd[:, k].contiguous() @ wd[:, k].T.contiguous()) * sd[:, g] * rows
        ref, size = ref + part, size + part.abs()
    half = (ref.abs() * P.U[y]).clamp(min=2.0 ** -25 if y == "fp16" else 0.0)
    tol = (3 if fmt == "w8" else ng + 2) * E * size * (1 + P.U[y]) + half
    assert bool(((out.double() - ref).abs() <= tol * (1 + 1e-6)).all()), float(((out.double() - ref).abs() / tol).max())
    assert bool((buf[:guard] == 7).all()) and bool((buf[-guard:] == 7).all())



@pytest.mark.gpu
@pytest.mark.parametrize("fmt,group,M,N,K", [("w8", 0, 100, 512, 96), ("w8", 0, 320, 4096, 320), ("w8", 0, 1024, 4096, 320), ("w8", 0, 1280, 12288, 96),
                                             ("w4_z16", 32, 100, 512, 160), ("w4_z16", 64, 320, 4096, 192), ("w4_z4", 64, 1024, 4096, 192),
                                             ("w4_z4", 128, 1024, 4096, 128), ("w4_z16", 32, 1024, 4096, 416), ("w4_z4", 32, 100, 512, 96)])
def test_the_least_alignment(gpu, fmt, group, M, N, K):
    """y, scales and zeros at 4 bytes, not 8 or 16: the results of aligned ones, bit for bit."""
    C.say(f"prompt linear {fmt} group={group} M={M} N={N} K={K}, 4-byte alignment")
    rng = np.random.default_rng(M + K)
    wq, ws, wz, _s, _w = P.weights(rng, N, K, fmt, group)
    xq = C.to_dev(NO.slab_codes(P.codes(rng, M, K)).reshape(M, K))
    xs = torch.rand(M, device=C.DEV) * 1e-2 + 1e-4

    def moved(t):
        if t is None:
            return None
        step = 4 // t.element_size()
        b = torch.zeros(t.numel() + 2 * step, dtype=t.dtype, device=C.DEV)[step:step + t.numel()].view(t.shape)
        b.copy_(t)
        assert b.data_ptr() % 8 == 4
        return b

    for y in ("fp32", "bf16"):
        got = []
        for at in (lambda t: t, moved):
            out = at(torch.full((M, N), 7.0, dtype=P.TYPES[y], device=C.DEV))
            if fmt == "w8":
                svg.w8a8_prompt_linear(xq, at(xs), wq, at(ws), N, out)
            else:
                svg.w4a8_prompt_linear(xq, at(xs), wq, at(ws), at(wz), fmt, group, N, out)
            got.append(out)
        assert torch.equal(*got) and not bool((got[0] == 7).all())


@pytest.mark.parametrize("N", [2 ** 30 + 1, 2 ** 31 - 16, 2 ** 31 - 1])
def test_more_columns_than_a_linear_takes(N):
    """Columns are counted in 32 bits, a tile past the last one included."""
    import speculative_verify_gemm_amd as lib
    A = 0x10000      # aligned, never dereferenced: the call is refused
    for M in (0, 1, 40):
        assert lib.lib.w8a8_prompt_linear(A, A, M, 32, A, A, N, A, 0, None) == 2 and "N > 2^30" in lib.last_error()
        assert lib.lib.w4a8_prompt_linear(A, A, M, 64, A, A, A, 1, 64, N, A, 0, None) == 2 and "N > 2^30" in lib.last_error()
    assert lib.lib.w8a8_prompt_linear(A, A, 0, 32, A, A, 2 ** 30, A, 0, None) == 0


def test_the_widest_products_are_not_for_the_kernel_of_few_rows():
    """It has 512 threads for 16 columns, and a launch fewer than 2^32 in a dimension; 65535 workgroups in the other."""
    import speculative_verify_gemm_amd as lib
    for fmt, group in [("w8", 0)] + [(f, g) for f in ("w4_z16", "w4_z4") for g in (32, 64, 128)]:
        for N in (2 ** 27 - 511, 2 ** 27, 2 ** 27 + 16, 2 ** 28 + 5, 2 ** 30):
            for M in (1, 16, 17, 33, 100, 128, 129, 257, 300):
                if (M + 15) // 16 * (N // 16) < 2 ** 31:
                    for cus in (8, 64, 256, 304):
                        assert FEW not in choice(lib.lib, fmt, group, M, N, 128, cus)[::2], (fmt, group, M, N, cus)
        for M in (65535 * 128 + 1, 2 ** 24):
            assert choice(lib.lib, fmt, group, M, 5, 128, 256)[0] != FEW


@pytest.mark.gpu
def test_weights_past_32_bits(gpu):
    """Codes of 2^33 bytes and more: offsets of a column's codes that 32 bits do not hold."""
    M, N, Kd = 3, 2 ** 27 + 21, 64
    C.say(f"w8a8_prompt_linear M={M} N={N} K={Kd}")
    Np = -(-N // 16) * 16
    g = torch.Generator(device=C.DEV).manual_seed(3)
    wq = torch.randint(-127, 128, (Np * Kd,), dtype=torch.int8, device=C.DEV, generator=g)
    ws = (torch.rand(N, device=C.DEV, generator=g) * 2e-3 + 1e-3).half()
    x = P.codes(np.random.default_rng(1), M, Kd)
    xs = torch.rand(M, device=C.DEV, generator=g) * 1e-2 + 1e-4
    y = torch.full((M, N), 7.0, device=C.DEV)
    svg.w8a8_prompt_linear(C.to_dev(NO.slab_codes(x).reshape(M, Kd)), xs, wq, ws, N, y)
    xd, tiles = C.to_dev(x).double(), wq.view(Np // 16, 4, 16, 16)       # [tile][16 values of K][row][value]
    for at in range(0, N, 1 << 22):
        n = min(N - at, 1 << 22)
        w = tiles[at // 16:(at + n + 15) // 16].permute(0, 2, 1, 3).reshape(-1, Kd)[:n].double()
        ref = (xd @ w.T.contiguous()) * ws[at:at + n].double() * xs.double()[:, None]
        assert bool(((y[:, at:at + n].double() - ref).abs() <= 3 * E * ref.abs() * (1 + 1e-6)).all()), at


# ------------------------------------------------------- tensors that are replaced
@pytest.mark.gpu
def test_a_row_maps_tensors_may_be_replaced(gpu):
    """A call uses the tensors that the object has at that time, and the object keeps those."""
    c = K.make(1, [5, 40], 40, H=1, dim=64, page=32)
    cache = K.to_library(svg, c)
    rows = svg.RowMap.empty(cache, 12)
    svg.kv_row_map(cache, P.i32([3, 2]), rows)
    first = {n: getattr(rows, n) for n in ("start", "count", "slot", "pos", "place")}
    kept = {n: t.clone() for n, t in first.items()}
    for n, t in first.items():
        setattr(rows, n, torch.full_like(t, 77))
        assert getattr(rows, n) is not t
    svg.kv_row_map(cache, P.i32([7, 4]), rows)
    for n, w in zip(("start", "count", "slot", "pos", "place"), PO.row_map(c, [7, 4], 0, 12)):
        assert np.array_equal(C.host(getattr(rows, n)), w) and torch.equal(first[n], kept[n]), n
    # what reads them: the rotation takes pos and place, the attention start and count
    x = torch.randn((12, 3, 64), device=C.DEV)
    rope, out = svg.Rope.make(64, device=C.DEV), torch.full((12, 1, 64), 7.0, device=C.DEV)
    rows.pos, rows.place = torch.full_like(rows.pos, -1), torch.full_like(rows.place, -1)
    svg.rope_append(cache, 0, rows, rope, x[:, :1], x[:, 1:2], x[:, 2:], out)
    assert bool((out == 7).all())
    rows.pos = torch.zeros_like(rows.pos)
    svg.rope_append(cache, 0, rows, rope, x[:, :1], x[:, 1:2], x[:, 2:], out)
    assert torch.equal(out, x[:, :1])
    rows.count = torch.zeros_like(rows.count)
    q = torch.ones((12, 1, 64), dtype=torch.float16, device=C.DEV)
    o = torch.full_like(q, 7.0)
    svg.prompt_attention(cache, 0, rows, q, o, svg.prompt_attention_workspace(cache, 1, 12))
    assert bool((o == 7).all())
    for name, bad, error in (("pos", rows.pos[:11], ValueError), ("pos", None, ValueError), ("start", rows.start.long(), TypeError),
                             ("count", rows.count.cpu(), ValueError), ("place", torch.zeros(24, dtype=torch.int32, device=C.DEV)[::2], ValueError)):
        now = getattr(rows, name)
        with pytest.raises(error):
            setattr(rows, name, bad)
        assert getattr(rows, name) is now
    with pytest.raises(ValueError):
        svg.RowMap(rows.start, rows.count, n_rows=3).pos = rows.pos


@pytest.mark.gpu
def test_a_rotations_frequencies_may_be_replaced(gpu):
    c = K.make(1, [5], 8, H=1, dim=64, page=32)
    cache = K.to_library(svg, c)
    rows = svg.RowMap.empty(cache, 6)
    svg.kv_row_map(cache, P.i32([6]), rows)
    rope = svg.Rope.make(32, device=C.DEV)
    x = torch.randn((6, 3, 64), device=C.DEV)

    def turned(r):
        out = torch.zeros((6, 1, 64), device=C.DEV)
        svg.rope_append(cache, 0, rows, r, x[:, :1], x[:, 1:2], x[:, 2:], out)
        return out

    before = turned(rope)
    rope.freq = svg.Rope.make(32, 500.0, device=C.DEV).freq
    rope.interleaved, rope.amplitude = True, 1.5
    assert rope.interleaved is True and rope.amplitude == 1.5
    fresh = svg.Rope(svg.Rope.make(32, 500.0, device=C.DEV).freq, interleaved=True, amplitude=1.5)
    after = turned(rope)
    assert torch.equal(after, turned(fresh)) and not torch.equal(after, before)
    for bad, error in ((rope.freq[:15], ValueError), (rope.freq.float(), TypeError), (rope.freq.cpu(), ValueError)):
        with pytest.raises(error):
            rope.freq = bad
    rope.amplitude = float("nan")
    with pytest.raises(svg.SvgError):
        turned(rope)



# ------------------------------------------------------- more rows than one turn of a launch
def long_table(pages, page, S, heads=1, dim=64):
    """A cache whose S slots have `pages` pages each, in an order of their own."""
    cache = svg.KVCache.empty(1, S * pages, heads, dim, page, S, pages, device=C.DEV)
    g = torch.Generator(device=C.DEV).manual_seed(7)
    cache.k.zero_(), cache.v.zero_()
    cache.table = torch.randperm(S * pages, device=C.DEV, generator=g).int().view(S, pages)
    cache.pages.fill_(pages), cache.refs.fill_(1)
    return cache


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0, 2 ** 19 + 3])
def test_a_row_map_of_more_rows_than_threads(gpu, T):
    """A launch has 2^20 threads at most: rows go on behind them."""
    S, page, n = 3, 128, [2 ** 19 + 1, 7, 2 ** 19 - 5]
    C.say(f"kv_row_map T={T} n={n}")
    cache = long_table(-(-(max(n) + 50) // page), page, S)
    cache.len.copy_(P.i32([0, 40, 9]))
    R = S * T if T else sum(n) + 300
    rows = svg.RowMap.empty(cache, R)
    svg.kv_row_map(cache, P.i32(n), rows, T=T)
    assert R > 2 ** 20
    first = [s * T for s in range(S)] if T else list(np.cumsum([0] + n[:-1]))
    table, lens = C.host(cache.table).astype(np.int64), C.host(cache.len)
    slot, pos, place = (np.full(R, -1, np.int64) for _ in range(3))
    for s in range(S):
        at = slice(first[s], first[s] + n[s])
        p = lens[s] + np.arange(n[s])
        slot[at], pos[at], place[at] = s, p, table[s, p // page] * page + p % page
    for name, want in (("start", first), ("count", n), ("slot", slot), ("pos", pos), ("place", place)):
        assert np.array_equal(C.host(getattr(rows, name)), want), name


@pytest.mark.gpu
def test_a_rotation_of_more_rows_than_one_turn(gpu):
    """Workgroups take 2^21 rows at a time: as many again, and the rest, are the same as in calls of their own."""
    R, half, page = 2 ** 21 + 40, 2 ** 20 + 32, 32
    C.say(f"rope_append n_rows={R}")
    cache, other = (long_table(-(-R // page), page, 1) for _ in range(2))
    g = torch.Generator(device=C.DEV).manual_seed(5)
    k, v = (torch.randn((R, 64), device=C.DEV, generator=g).half() for _ in range(2))
    rope = svg.Rope.make(64, device=C.DEV)
    rows = svg.RowMap.empty(cache, R)
    svg.kv_row_map(cache, P.i32([R]), rows)
    assert bool((rows.place >= 0).all())
    svg.rope_append(cache, 0, rows, rope, None, k, v)
    for at in (slice(0, half), slice(half, R)):
        part = svg.RowMap(rows.start, rows.count, rows.pos[at], rows.place[at])
        svg.rope_append(other, 0, part, rope, None, k[at], v[at])
    assert torch.equal(cache.k, other.k) and torch.equal(cache.v, other.v)
    last = int(rows.place[-1])
    d = torch.arange(64)
    assert torch.equal(cache.v[0, last // page, 0].cpu()[CO.value_at(last % page, d, 64)], v[-1].cpu())


@pytest.mark.gpu
def test_codes_of_more_rows_than_a_launch_has_in_x(gpu):
    """Rows go on in the second dimension behind 2^20; the rows of whole slabs are those of a call of their own."""
    M, Kd, half = 2 ** 20 + 37, 32, 2 ** 19
    C.say(f"gated_quant_i8 M={M} K={Kd}")
    g = torch.Generator(device=C.DEV).manual_seed(5)
    x, gate = (torch.randn((M, Kd), device=C.DEV, generator=g).bfloat16() for _ in range(2))
    signs = (torch.randint(0, 2, (Kd,), device=C.DEV, generator=g) * 2 - 1).to(torch.int8)

    def call(x, gate):
        q, s = torch.full(x.shape, 99, dtype=torch.int8, device=C.DEV), torch.full(x.shape[:1], 7.0, device=C.DEV)
        svg.gated_quant_i8(x, gate, signs, q, s)
        return q.view(-1), s

    q, s = call(x, gate)
    parts = [call(x[at], gate[at]) for at in (slice(0, half), slice(half, M))]
    assert torch.equal(q, torch.cat([p[0] for p in parts])) and torch.equal(s, torch.cat([p[1] for p in parts]))
    at = slice(2 ** 20 - 64, M)                      # from the last slabs of the first dimension on
    codes, scales = PO.gated_quant(x[at].float().cpu().numpy(), gate[at].float().cpu().numpy(), C.host(signs), 32)
    assert np.array_equal(C.host(s[at]), scales) and np.array_equal(C.host(q[(2 ** 20 - 64) * Kd:]), NO.slab_codes(codes))



# ------------------------------------------------------------------ frequencies
@pytest.mark.parametrize("rot,base,trained,bounds", [(64, 1e4, 4096, (32.0, 1.0)), (128, 5e5, 8192, (32.0, 1.0)), (128, 1e6, 32768, (8.0, 2.0)),
                                                     (64, 1e4, 4096, (2.001, 2.0)), (16, 1e4, 100, (32.0, 1.0)), (64, 100.0, 10 ** 9, (32.0, 1.0))])
def test_bands_of_frequencies(rot, base, trained, bounds):
    """Pair by pair: x turns trained base^(-2 x / rot) / (2 pi) times, so n turns are at x = rot ln(trained / (2 pi n)) / (2 ln base); the
    weight of the divided frequency goes from 0 to 1 between the whole numbers around the two; a step where they are one."""
    import math

    import speculative_verify_gemm_amd as lib

    class Host:
        def __init__(self, freq, interleaved=False, amplitude=1.0):
            self.freq = freq

    got = lib.Rope.make.__func__(Host, rot, base, scaling="bands", factor=4.0, trained=trained, bounds=bounds, device="cpu").freq
    low, high = (rot * math.log(trained / (2 * math.pi * n)) / (2 * math.log(base)) for n in bounds)
    low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
    for i in range(rot // 2):
        part = 0.0 if i <= low else 1.0 if i >= high else (i - low) / (high - low)
        plain = base ** (-2 * i / rot)
        want = plain * (1 - part) + plain / 4 * part
        assert math.isclose(got[i], want, rel_tol=1e-13), i


# ------------------------------------------------------------------ the sources
def test_assembly_declares_the_registers_that_it_writes():
    """m0 holds where loads into LDS go: what writes it has to name it, or the compiler may keep a value of its own there."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_verify_gemm_amd", "csrc")
    found = 0
    for name in sorted(os.listdir(csrc)):
        for block in re.findall(r"\basm\s+volatile\s*\((.*?)\);", open(os.path.join(csrc, name)).read(), re.S):
            code, operands = block.split(":", 1) if ":" in block else (block, "")
            if re.search(r"s_mov_b32 m0\b", code):
                found += 1
                assert '"m0"' in operands.split(":")[-1], (name, code)
    assert found >= 3
