"""One decoder layer's verify pass as a program makes it, over several passes: norm and quantization, the fused
projection, the rows into the cache, attention of the trees, the output projection, norm again, logits,
greedy acceptance, the commit, room for the next trees -- with a fork in between.

Every call's result is checked against the oracle on the inputs that the device had at that call, so that
each bound is that call's own (codes, tokens, tables and cache patterns: equal; the linears: 2e-3 as in
their own tests; attention: the bound of tests/test_tree_attention_parity.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import synth
from oracle import attention_oracle as AO
from oracle import cache_oracle as CO
from oracle import norm_oracle as N
from oracle import svg_oracle as O
from oracle import tree_oracle as TO

pytestmark = pytest.mark.gpu

S, T, HQ, HKV, DIM, HID, VOCAB, PAGE, EPS = 2, 8, 4, 2, 64, 256, 160, 32, 1e-5
GROUP = 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    global A, C, K, svg
    import cache_cases as K  # noqa: F401
    import svg_cases as C  # noqa: F401
    import test_tree_attention_parity as A  # noqa: F401
    import speculative_verify_gemm_amd as svg
    A.svg, A.C, A.K = svg, C, K


class Layer:
    """Weights of one layer (quantized on the device and by the oracle) and the buffers of a pass."""

    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        dev = lambda a: C.to_dev(np.ascontiguousarray(a))  # noqa: E731
        self.rng = rng
        self.signs = {n: np.where(rng.integers(0, 2, k) == 1, 1, -1).astype(np.int8) for n, k in (("in", HID), ("o", HQ * DIM), ("head", HID))}
        shapes = {"in": ((HQ + 2 * HKV) * DIM, HID), "o": (HID, HQ * DIM), "head": (VOCAB, HID)}
        W = {n: (rng.standard_normal(s) * (0.08 if n != "head" else 0.2)).astype(np.float32) for n, s in shapes.items()}
        self.dev = {n: C.gpu_prepare(W[n], self.signs[n], "w4_z16", GROUP) for n in W}
        self.ora = {n: O.prepare_w4(W[n], self.signs[n], GROUP) for n in W}
        self.norm = [(1 + 0.1 * rng.standard_normal(HID)).astype(np.float32) for _ in range(2)]
        self.embed = rng.standard_normal((VOCAB, HID)).astype(np.float32)
        self.d = dict(norm=[dev(n) for n in self.norm], embed=dev(self.embed), signs={n: dev(v) for n, v in self.signs.items()})
        f = lambda *s: torch.empty(s, dtype=torch.float32, device=C.DEV)  # noqa: E731
        i = lambda *s: torch.zeros(s, dtype=torch.int32, device=C.DEV)  # noqa: E731
        M = S * T
        self.b = dict(res=f(M, HID), xq=torch.empty((M, HID), dtype=torch.int8, device=C.DEV), xs=f(M), qkv=f(M, (HQ + 2 * HKV) * DIM),
                      att=f(M, HQ, DIM), aq=torch.empty((M, HQ * DIM), dtype=torch.int8, device=C.DEV), as_=f(M), o=f(M, HID),
                      logits=f(M, VOCAB), target=i(S, T), path=i(S, T), emit=i(S, T), n=i(S), parent=i(S, T), draft=i(S, T),
                      need=i(S), status=i(S))
        self.accept_ws = svg.tree_workspace()

    def linear(self, name, xq, xs, y):
        w = self.dev[name]
        svg.w4a8_linear(xq, xs, w["wq"], w["ws"], w["wz"], "w4_z16", GROUP, w["N"], y)


def verify_pass(L, cache, ws, kv_ws):
    """The calls of one pass; every buffer is the layer's own, so it can be captured."""
    b, d = L.b, L.d
    M = S * T
    b["res"].copy_(d["embed"][b["draft"].view(-1).long()])
    yield "norm0", lambda: svg.add_rmsnorm_quant_i8(b["res"], None, d["norm"][0], EPS, d["signs"]["in"], b["xq"], b["xs"])
    yield "qkv", lambda: L.linear("in", b["xq"], b["xs"], b["qkv"])
    q, k, v = b["qkv"].split([HQ * DIM, HKV * DIM, HKV * DIM], 1)
    yield "reserve", lambda: svg.kv_reserve(cache, b["need"], b["status"], kv_ws)
    yield "append", lambda: svg.kv_append(cache, 0, k, v, T)
    yield "attention", lambda: svg.tree_attention(cache, 0, q.unflatten(1, (HQ, DIM)), b["parent"], b["att"], ws)
    w = L.dev["o"]
    yield "o", lambda: svg.act_quant_w4a8_linear(b["att"].view(M, HQ * DIM), d["signs"]["o"], b["aq"], b["as_"], w["wq"], w["ws"], w["wz"],
                                                 "w4_z16", GROUP, HID, b["o"])
    yield "norm1", lambda: svg.add_rmsnorm_quant_i8(b["o"], b["res"], d["norm"][1], EPS, d["signs"]["head"], b["xq"], b["xs"])
    yield "head", lambda: L.linear("head", b["xq"], b["xs"], b["logits"])

    def accept():
        for s in range(S):
            svg.tree_accept_greedy(b["logits"][s * T:(s + 1) * T], b["parent"][s], b["draft"][s], b["target"][s], b["path"][s],
                                   b["emit"][s], b["n"][s:s + 1], L.accept_ws)
    yield "accept", accept
    yield "commit", lambda: svg.kv_commit(cache, b["path"], b["n"])


def start(seed):
    L = Layer(seed)
    c = K.make(seed, [37, 64], 0, H=HKV, dim=DIM, page=PAGE, spare=20, width=9)
    A.fill(c, np.random.default_rng(seed), "bf16")
    cache = K.to_library(svg, c, "bf16")
    L.b["need"].fill_(T)
    return L, c, cache, svg.tree_attention_workspace(cache, HQ, T), svg.kv_workspace(cache)


def trees(L, turn):
    """Trees whose drafted tokens are random, apart from the root: the last token emitted (a fixed one at first)."""
    parent = np.stack([synth.draft_tree(T, VOCAB, seed=turn * 5 + s, shape="bushy")[1] for s in range(S)]).astype(np.int32)
    draft = L.rng.integers(0, VOCAB, (S, T)).astype(np.int32)
    return parent, draft


def test_every_step_of_a_layer_over_several_passes():
    L, c, cache, ws, kv_ws = start(21)
    b = L.b
    grown = 0
    for turn in range(4):
        parent, draft = trees(L, turn)
        b["parent"].copy_(torch.from_numpy(parent))
        b["draft"].copy_(torch.from_numpy(draft))
        if turn == 2:                # the second slot starts over from the first one's state
            other = cache.other_tables()
            svg.kv_fork(cache, A.i32([0, 0]), other)
            c = CO.fork(c, [0, 0])
            cache = other
            K.same(cache, c, ("pages", "len", "refs"))
        host = lambda n: C.host(b[n])  # noqa: E731
        for name, call in verify_pass(L, cache, ws, kv_ws):
            res0 = host("res").copy()
            o0 = host("o").copy()
            call()
            if name in ("norm0", "norm1"):
                i = int(name[-1])
                x, r = (res0, None) if i == 0 else (o0, res0)
                h, _u, qx, sx = N.norm_quant(x, r, L.norm[i], EPS, L.signs["in" if i == 0 else "head"], 32)
                assert np.array_equal(host("xq").reshape(-1), N.slab_codes(qx)) and np.array_equal(host("xs"), sx)
                if i:
                    assert np.array_equal(host("res"), h)
            elif name in ("qkv", "head"):
                w = L.ora["in" if name == "qkv" else "head"]
                ref = O.w4a8_output(sx, O.w4_group_partials(qx, w["q"], w["z"], GROUP), w["s"])
                e, r, _ = O.output_error(host("qkv" if name == "qkv" else "logits"), ref)
                assert e <= 2e-3 and r <= 2e-3
            elif name == "reserve":
                assert not host("status").any() and not CO.reserve(c, [T] * S).any()
                K.same(cache, c, ("pages", "len", "refs", "k", "v"))
            elif name == "append":
                kv = torch.from_numpy(host("qkv")[:, HQ * DIM:]).to(torch.bfloat16)
                pat = K.bits(kv).reshape(S, T, 2, HKV, DIM)
                CO.append(c, 0, pat[:, :, 0], pat[:, :, 1], T)
                K.same(cache, c, ("k", "v"))
            elif name == "attention":
                q = host("qkv")[:, :HQ * DIM].reshape(S, T, HQ, DIM)
                ref, spread = AO.attention(c, A.wide("bf16"), 0, q, parent, T, None, DIM ** -0.5)
                A.close(host("att").reshape(S, T, HQ, DIM), ref, A.bound(c, "bf16", spread, int(c["len"].max()) + T))
            elif name == "o":
                ref = O.linear_w4(host("att").reshape(S * T, HQ * DIM), L.signs["o"], L.ora["o"])[0]
                e, r, _ = O.output_error(host("o"), ref)
                assert e <= 2e-3 and r <= 2e-3
            elif name == "accept":
                counts, paths = [], np.full((S, T), -1, np.int32)
                for s in range(S):
                    _t, p, em = TO.verify_tree(host("logits")[s * T:(s + 1) * T], parent[s], draft[s])
                    counts.append(len(em))
                    paths[s, :len(p)] = p
                assert np.array_equal(host("n"), counts) and np.array_equal(host("path"), paths)
                if turn % 2:         # random drafts are hardly ever right: every second pass a path of its own
                    for s in range(S):
                        p = TO.root_path(parent[s], T - 1 - s)[1:]
                        counts[s], paths[s] = len(p) + 1, -1
                        paths[s, :len(p)] = p
                    b["n"].copy_(torch.tensor(counts))
                    b["path"].copy_(torch.from_numpy(paths))
            else:
                c["len"] = CO.commit(c, paths, counts)
                K.same(cache, c, ("k", "v", "len"))
                grown += sum(counts)
        assert np.array_equal(CO.holders(c), c["refs"])
    assert grown > 4 * S             # more than the roots were committed


def test_the_pass_captured_and_replayed():
    """The same pass as one graph, replayed with the eager passes of a second, equal set of buffers in between: equal bits."""
    (L, _c, cache, ws, kv_ws), (L2, _c2, cache2, ws2, kv_ws2) = start(33), start(33)
    parent, draft = trees(L, 0)

    def put(b, draft):
        b["parent"].copy_(torch.from_numpy(parent))
        b["draft"].copy_(torch.from_numpy(draft))

    def run(*args):
        for _name, call in verify_pass(*args):
            call()

    put(L.b, draft)
    put(L2.b, draft)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(L, cache, ws, kv_ws)
    side.synchronize()
    run(L2, cache2, ws2, kv_ws2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(L, cache, ws, kv_ws)
    for turn in range(4):
        draft = L.rng.integers(0, VOCAB, (S, T)).astype(np.int32)
        put(L.b, draft)
        put(L2.b, draft)
        g.replay()
        torch.cuda.synchronize()
        run(L2, cache2, ws2, kv_ws2)
        torch.cuda.synchronize()
        for n in ("xq", "xs", "qkv", "att", "o", "res", "logits", "path", "emit", "n", "status"):
            assert torch.equal(L.b[n], L2.b[n]), (turn, n)
        for n in ("table", "pages", "len", "refs"):
            assert torch.equal(getattr(cache, n), getattr(cache2, n)), (turn, n)
        assert np.array_equal(K.bits(cache.k), K.bits(cache2.k)) and np.array_equal(K.bits(cache.v), K.bits(cache2.v))
