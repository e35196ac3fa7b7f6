"""A prompt's pass through one decoder layer as a program makes it, over several steps of unequal chunks: norm and
quantization, the fused projection, room in the pages, the row map, rotation and append, attention, codes without a gate, the
output projection, norm again, gate and up, the gated codes, down -- with a fork in between, and a draft tree verified on
what the prompt left in the cache.

Every call's result is checked against the oracle on the inputs that the device had at that call, so that each bound is
that call's own (codes, tables and maps: equal; the others: the bounds of tests/test_prompt_parity.py and
tests/test_tree_attention_parity.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import attention_oracle as AO
from oracle import cache_oracle as CO
from oracle import norm_oracle as NO
from oracle import prompt_oracle as PO

pytestmark = pytest.mark.gpu

S, HQ, HKV, DIM, HID, MLP, PAGE, EPS, R = 3, 4, 2, 64, 256, 384, 32, 1e-5, 150
GROUP, ROT, BASE = 64, 32, 10000.0
WIDE = (HQ + 2 * HKV) * DIM


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    global A, C, K, P, svg
    import cache_cases as K  # noqa: F401
    import svg_cases as C  # noqa: F401
    import test_prompt_parity as P  # noqa: F401
    import test_tree_attention_parity as A  # noqa: F401
    import speculative_verify_gemm_amd as svg
    A.svg, A.C, A.K = svg, C, K
    P.svg, P.C, P.K = svg, C, K


class Layer:
    """Weights of one layer (device storage and fp64) and the buffers of a step."""

    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        dev = lambda a: C.to_dev(np.ascontiguousarray(a))  # noqa: E731
        shapes = {"qkv": (WIDE, HID, "w4_z16"), "o": (HID, HQ * DIM, "w8"), "up": (2 * MLP, HID, "w4_z4"), "down": (HID, MLP, "w4_z16")}
        self.w = {n: P.weights(rng, N, Kd, f, GROUP) + (N, f) for n, (N, Kd, f) in shapes.items()}
        self.signs = {n: np.where(rng.integers(0, 2, Kd) == 1, 1, -1).astype(np.int8) for n, (_, Kd, _f) in shapes.items()}
        self.norm = [(1 + 0.1 * rng.standard_normal(HID)).astype(np.float32) for _ in range(2)]
        self.rope = svg.Rope.make(ROT, BASE, device=C.DEV)
        self.freq = C.host(self.rope.freq)
        self.d = dict(norm=[dev(n) for n in self.norm], signs={n: dev(v) for n, v in self.signs.items()})
        f = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device=C.DEV)  # noqa: E731
        bf, i8 = torch.bfloat16, torch.int8
        self.b = dict(res=f(R, HID), xq=f(R, HID, t=i8), xs=f(R), qkv=f(R, WIDE, t=bf), q=f(R, HQ, DIM, t=bf), att=f(R, HQ, DIM, t=bf),
                      aq=f(R, HQ * DIM, t=i8), as_=f(R), o=f(R, HID), up=f(R, 2 * MLP, t=bf), mq=f(R, MLP, t=i8), ms=f(R), down=f(R, HID),
                      need=f(S, t=torch.int32), status=f(S, t=torch.int32))

    def linear(self, name, xq, xs, y):
        wq, ws, wz, _, _, N, fmt = self.w[name]
        if fmt == "w8":
            svg.w8a8_prompt_linear(xq, xs, wq, ws, N, y)
        else:
            svg.w4a8_prompt_linear(xq, xs, wq, ws, wz, fmt, GROUP, N, y)

    def linear_ok(self, name, codes, xs, y):
        _, _, _, s, w, _, fmt = self.w[name]
        Kd, ng = codes.shape[1], s.shape[1]
        ref, size = 0, 0
        for g in range(ng):
            k = slice(g * (Kd // ng), (g + 1) * (Kd // ng))
            part = (codes[:, k].astype(np.float64) @ w[:, k].astype(np.float64).T) * s[:, g] * xs.astype(np.float64)[:, None]
            ref, size = ref + part, size + np.abs(part)
        kind = next(n for n, t in P.TYPES.items() if t == y.dtype)
        tol = (3 * P.E * np.abs(ref) if fmt == "w8" else (ng + 2) * P.E * size) * (1 + P.U[kind]) + P.half_step(kind, ref)
        assert np.all(np.abs(P.host64(y) - ref) <= tol * (1 + 1e-6))


def step(L, cache, rows, ws, kv_ws):
    """The calls of one step on the residual rows; every buffer is the layer's own, so it can be captured."""
    b, d = L.b, L.d
    q, k, v = b["qkv"].split([HQ * DIM, HKV * DIM, HKV * DIM], 1)
    yield "norm0", lambda: svg.add_rmsnorm_quant_i8(b["res"], None, d["norm"][0], EPS, d["signs"]["qkv"], b["xq"], b["xs"])
    yield "qkv", lambda: L.linear("qkv", b["xq"], b["xs"], b["qkv"])
    yield "reserve", lambda: svg.kv_reserve(cache, b["need"], b["status"], kv_ws)
    yield "map", lambda: svg.kv_row_map(cache, b["need"], rows)
    yield "rope", lambda: svg.rope_append(cache, 0, rows, L.rope, q.unflatten(1, (HQ, DIM)), k, v, b["q"])
    yield "attention", lambda: svg.prompt_attention(cache, 0, rows, b["q"], b["att"], ws)
    yield "codes", lambda: svg.gated_quant_i8(b["att"].view(R, HQ * DIM), None, d["signs"]["o"], b["aq"], b["as_"])
    yield "o", lambda: L.linear("o", b["aq"], b["as_"], b["o"])
    yield "norm1", lambda: svg.add_rmsnorm_quant_i8(b["o"], b["res"], d["norm"][1], EPS, d["signs"]["up"], b["xq"], b["xs"])
    yield "up", lambda: L.linear("up", b["xq"], b["xs"], b["up"])
    yield "gate", lambda: svg.gated_quant_i8(b["up"][:, MLP:], b["up"][:, :MLP], d["signs"]["down"], b["mq"], b["ms"])
    yield "down", lambda: L.linear("down", b["mq"], b["ms"], b["down"])
    yield "len", lambda: cache.len.add_(rows.count)


def start(seed):
    L = Layer(seed)
    c = K.make(seed, [5, 0, 64], 0, H=HKV, dim=DIM, page=PAGE, spare=40, width=14)
    P.fill(c, np.random.default_rng(seed), "bf16")
    cache = K.to_library(svg, c, "bf16")
    return L, c, cache, svg.RowMap.empty(cache, R), svg.prompt_attention_workspace(cache, HQ, R), svg.kv_workspace(cache)


def embed(L, seed):
    x = np.random.default_rng(seed).standard_normal((R, HID)).astype(np.float32)
    L.b["res"].copy_(torch.from_numpy(x))


def test_every_call_of_a_step():
    L, c, cache, rows, ws, kv_ws = start(3)
    b = L.b
    host = lambda n: C.host(b[n])  # noqa: E731
    for turn, n in enumerate(([37, 0, 70], [20, 5, 1], [1, 100, 40], [60, 1, 1])):
        embed(L, turn)
        b["need"].copy_(torch.tensor(n))
        if turn == 2:                    # the second slot starts over from the third one's state
            other = cache.other_tables()
            svg.kv_fork(cache, P.i32([0, 2, 2]), other)
            c = CO.fork(c, [0, 2, 2])
            cache = other
        for name, call in step(L, cache, rows, ws, kv_ws):
            res0, o0 = host("res").copy(), host("o").copy()
            if name == "rope":
                b["q"].fill_(7)          # (what stays where there is no row)
            call()
            if name in ("norm0", "norm1"):
                i = int(name[-1])
                x, r = (res0, None) if i == 0 else (o0, res0)
                h, _u, codes, xs = NO.norm_quant(x, r, L.norm[i], EPS, L.signs["qkv" if i == 0 else "up"], 32)
                assert np.array_equal(host("xq").reshape(-1), NO.slab_codes(codes)) and np.array_equal(host("xs"), xs)
                if i:
                    assert np.array_equal(host("res"), h)
            elif name in ("qkv", "o", "up", "down"):
                L.linear_ok(name, codes, xs, b[name])
            elif name == "reserve":
                assert not host("status").any() and not CO.reserve(c, n).any()
                K.same(cache, c)
            elif name == "map":
                want = PO.row_map(c, n, 0, R)
                start_, count, _slot, pos, place = want
                for t, w in zip(("start", "count", "slot", "pos", "place"), want):
                    assert np.array_equal(C.host(getattr(rows, t)), w), t
            elif name == "rope":
                q, k, v = b["qkv"].cpu().split([HQ * DIM, HKV * DIM, HKV * DIM], 1)
                P.check_rope(c, cache, rows, L.rope, L.freq, (q.unflatten(1, (HQ, DIM)), k, v), b["q"], "bf16", 0, False, amplitude=1.0)
                c["k"], c["v"] = K.bits(cache.k), K.bits(cache.v)
            elif name == "attention":
                ref, mine, size = PO.attention(c, P.wide("bf16"), 0, P.host64(b["q"]), start_, count, DIM ** -0.5)
                assert np.array_equal(mine, pos >= 0) and not np.isnan(ref[mine]).any()
                tol = P.attention_bound(c, "bf16", ref, size, int(c["len"].max()) + max(n))
                assert np.all((np.abs(P.host64(b["att"]) - ref) <= tol)[mine])
            elif name in ("codes", "gate"):
                x, g = (b["att"].view(R, -1), None) if name == "codes" else (b["up"][:, MLP:], b["up"][:, :MLP])
                x, g = (None if t is None else t.float().cpu().numpy() for t in (x, g))
                codes, xs = PO.gated_quant(x, g, L.signs["o" if name == "codes" else "down"], 32)
                q, s = ("aq", "as_") if name == "codes" else ("mq", "ms")
                assert np.array_equal(host(q).reshape(-1), NO.slab_codes(codes)) and np.array_equal(host(s), xs)
            else:
                c["len"] = (c["len"] + count).astype(np.int32)
                assert np.array_equal(C.host(cache.len), c["len"])
        assert np.array_equal(CO.holders(c), c["refs"])
    # a draft tree on what the prompts left: rotated by depth, appended, attended to, committed
    T = 7
    rng = np.random.default_rng(9)
    parent = A.trees(rng, S, T)
    tree = svg.RowMap.empty(cache, S * T)
    b["need"].fill_(T)
    svg.kv_reserve(cache, b["need"], b["status"], kv_ws)
    assert not host("status").any() and not CO.reserve(c, [T] * S).any()
    svg.kv_row_map(cache, b["need"], tree, T=T, parent=P.i32(parent))
    assert np.array_equal(C.host(tree.pos), PO.row_map(c, [T] * S, T, S * T, parent)[3])
    x = torch.from_numpy(rng.standard_normal((S * T, WIDE)).astype(np.float32)).to(C.DEV)
    q, k, v = x.split([HQ * DIM, HKV * DIM, HKV * DIM], 1)
    qt, att = torch.zeros((S * T, HQ, DIM), device=C.DEV), torch.zeros((S * T, HQ, DIM), device=C.DEV)
    svg.rope_append(cache, 0, tree, L.rope, q.unflatten(1, (HQ, DIM)), k, v, qt)
    svg.tree_attention(cache, 0, qt, P.i32(parent), att, svg.tree_attention_workspace(cache, HQ, T))
    c["k"], c["v"] = K.bits(cache.k), K.bits(cache.v)
    ref, spread = AO.attention(c, P.wide("bf16"), 0, C.host(qt).reshape(S, T, HQ, DIM), parent, T, None, DIM ** -0.5)
    A.close(C.host(att).reshape(S, T, HQ, DIM), ref, A.bound(c, "bf16", spread, int(c["len"].max()) + T))


def test_a_prompt_in_one_piece_and_in_chunks():
    """The same rows as one prompt and in three chunks: the same pages, and outputs within both bounds."""
    rng = np.random.default_rng(5)
    n, parts = 90, [33, 1, 56]
    x = torch.from_numpy(rng.standard_normal((n, WIDE)).astype(np.float32)).to(C.DEV).bfloat16()
    rope = svg.Rope.make(ROT, BASE, interleaved=True, device=C.DEV)
    got = []
    for pieces in ([n], parts):
        cache = svg.KVCache.empty(1, 8, HKV, DIM, PAGE, 1, 6, dtype=torch.bfloat16, device=C.DEV)
        cache.k.zero_(), cache.v.zero_()
        kv_ws, status, out, at = svg.kv_workspace(cache), P.i32([7]), [], 0
        for m in pieces:
            svg.kv_reserve(cache, P.i32([m]), status, kv_ws)
            rows = svg.RowMap.empty(cache, m)
            svg.kv_row_map(cache, P.i32([m]), rows)
            q, k, v = x[at:at + m].split([HQ * DIM, HKV * DIM, HKV * DIM], 1)
            qo = torch.empty((m, HQ, DIM), dtype=torch.bfloat16, device=C.DEV)
            svg.rope_append(cache, 0, rows, rope, q.unflatten(1, (HQ, DIM)), k, v, qo)
            o = torch.empty_like(qo)
            svg.prompt_attention(cache, 0, rows, qo, o, svg.prompt_attention_workspace(cache, HQ, m))
            cache.len.add_(rows.count)
            out.append(torch.cat((qo, o), 1))
            at += m
        got.append((K.bits(cache.k), K.bits(cache.v), torch.cat(out), cache))
    (k1, v1, o1, cache), (k2, v2, o2, _) = got
    assert np.array_equal(k1, k2) and np.array_equal(v1, v2) and torch.equal(o1[:, :HQ], o2[:, :HQ])
    c = dict(k=k1, v=v1, table=C.host(cache.table), pages=C.host(cache.pages), len=np.zeros(1, np.int32), refs=C.host(cache.refs), dim=DIM, page=PAGE)
    ref, _, size = PO.attention(c, P.wide("bf16"), 0, P.host64(o1[:, :HQ]), [0], [n], DIM ** -0.5)
    for o in (o1, o2):
        assert np.all(np.abs(P.host64(o[:, HQ:]) - ref) <= P.attention_bound(c, "bf16", ref, size, n))


def test_the_step_captured_and_replayed():
    """The same step as one graph, replayed with other chunks, with the eager steps of an equal set of buffers in between."""
    (L, _c, cache, rows, ws, kv_ws), (L2, _c2, cache2, rows2, ws2, kv_ws2) = start(7), start(7)

    def run(*args):
        for _name, call in step(*args):
            call()

    def put(turn, n):
        for layer in (L, L2):
            embed(layer, turn)
            layer.b["need"].copy_(torch.tensor(n))

    put(0, [4, 30, 2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(L, cache, rows, ws, kv_ws)
    side.synchronize()
    run(L2, cache2, rows2, ws2, kv_ws2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(L, cache, rows, ws, kv_ws)
    for turn, n in enumerate(([10, 0, 90], [0, 0, 0], [33, 1, 1], [1, 1, 100])):
        put(turn + 1, n)
        g.replay()
        torch.cuda.synchronize()
        run(L2, cache2, rows2, ws2, kv_ws2)
        torch.cuda.synchronize()
        for name in ("start", "count", "slot", "pos", "place"):
            assert torch.equal(getattr(rows, name), getattr(rows2, name)), name
        for name in L.b:
            assert torch.equal(L.b[name], L2.b[name]), (turn, name)
        for name in ("table", "pages", "len", "refs"):
            assert torch.equal(getattr(cache, name), getattr(cache2, name)), (turn, name)
        assert np.array_equal(K.bits(cache.k), K.bits(cache2.k)) and np.array_equal(K.bits(cache.v), K.bits(cache2.v))
