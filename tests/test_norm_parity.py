"""add_rmsnorm_quant_i8 against the oracle (oracle/norm_oracle.py): residual,
normalised rows, codes and scales bit for bit.

Why bit for bit: every step that reaches a code is one fp32 operation in both,
except r, whose 64-bit sum differs from the oracle's by its order only: at most
K 2^-53 relative, 2^-38 for K = 32768, so its rounding to fp32 is another one
for less than one row in 2^13 of such length (one in 2^16 at K = 4096); the
inputs here are fixed."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import norm_oracle as N

pytestmark = pytest.mark.gpu

EPS = 1e-6
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    global C, svg
    import svg_cases as C  # noqa: F401
    import speculative_verify_gemm_amd as svg


def rows(M, K, seed, xt="fp32", wt="fp32"):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((M, K), dtype=np.float32)).to(DT[xt])
    res = rng.standard_normal((M, K), dtype=np.float32) * 3
    res[:, rng.choice(K, size=min(4, K), replace=False)] *= 50
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(K)).astype(np.float32)).to(DT[wt])
    signs = np.where(rng.integers(0, 2, K) == 1, 1, -1).astype(np.int8)
    return x, res, w, signs


def run(x, res, w, signs, block=32, eps=EPS, want_y=True):
    """Outputs of one call, written into buffers with guard bands around them."""
    M, K = x.shape
    guard = 64
    xq = torch.full((M * K + 2 * guard,), 77, dtype=torch.int8, device=C.DEV)
    xs = torch.full((M + 2 * guard,), 7.0, device=C.DEV)
    y = torch.full((M * K + 2 * guard,), 7.0, device=C.DEV) if want_y else None
    r = torch.full((M * K + 2 * guard,), 7.0, device=C.DEV)
    inner = lambda t, n: t[guard:guard + n]  # noqa: E731
    rin = None
    if res is not None:
        inner(r, M * K).copy_(C.to_dev(res).view(-1))
        rin = inner(r, M * K).view(M, K)
    svg.add_rmsnorm_quant_i8(x.to(C.DEV), rin, w.to(C.DEV), eps, C.to_dev(signs), inner(xq, M * K),
                             inner(xs, M), y=None if y is None else inner(y, M * K).view(M, K), block=block)
    for t, v in ((xq, 77), (xs, 7.0), (r, 7.0)) + (((y, 7.0),) if want_y else ()):
        assert bool((t[:guard] == v).all()) and bool((t[-guard:] == v).all())
    return (C.host(inner(r, M * K)).reshape(M, K), None if y is None else C.host(inner(y, M * K)).reshape(M, K),
            C.host(inner(xq, M * K)), C.host(inner(xs, M)))


def check(x, res, w, signs, block=32, eps=EPS, want_y=True):
    h, u, q, s = N.norm_quant(x.float().numpy(), res, w.float().numpy(), eps, signs, block)
    gh, gy, gq, gs = run(x, res, w, signs, block, eps, want_y)
    if res is not None:
        assert np.array_equal(gh, h)
    if want_y:
        assert np.array_equal(gy, u)
    assert np.array_equal(gs, s)
    assert np.array_equal(gq, N.slab_codes(q))


@pytest.mark.parametrize("M,K,block,xt,wt", [
    (1, 32, 32, "fp32", "fp32"), (1, 64, 64, "fp16", "bf16"), (2, 96, 32, "bf16", "fp16"),
    (3, 992, 32, "fp32", "bf16"), (16, 4096, 64, "fp32", "bf16"), (31, 1024, 32, "fp16", "fp32"),
    (32, 4096, 32, "fp32", "fp32"), (33, 4128, 32, "bf16", "bf16"), (67, 1088, 64, "fp16", "fp16"),
    (5, 12288, 32, "fp32", "fp32"), (2, 16384, 64, "bf16", "fp32"), (3, 20000, 32, "fp32", "fp16"),
    (2, 32768, 32, "fp16", "fp32"),
    # enough rows for the narrow workgroups, at each number of chunks a thread
    (515, 640, 32, "fp32", "fp32"), (512, 1984, 64, "fp16", "bf16"), (513, 4096, 32, "bf16", "fp32"), (1025, 6016, 32, "fp32", "fp16"),
])
def test_matches_the_oracle(M, K, block, xt, wt):
    C.say(f"add_rmsnorm_quant_i8 M={M} K={K} block={block} {xt} {wt}")
    x, res, w, signs = rows(M, K, M * 7 + K, xt, wt)
    check(x, res, w, signs, block, want_y=M % 2 == 1)


def test_without_a_residual_and_empty():
    x, _res, w, signs = rows(9, 512, 3, "bf16", "fp32")
    check(x, None, w, signs, 32)
    check(x[:0], None, w, signs, 32)


def test_extreme_rows():
    """An all-zero row (scale 0, codes 0), a row of denormals, a row whose
    squares pass fp32's range, one outlier, and eps far above the mean square."""
    x, res, w, signs = rows(6, 256, 11)
    x[:] = 0
    res[0] = 0
    res[1] = np.float32(1e-41)
    res[2] *= np.float32(1e25)
    res[3] = 0
    res[3, 7] = -3.5e4
    check(x, res, w, signs)
    check(x, res, w, signs, eps=10.0)


def test_the_separate_steps_give_the_same_codes():
    """The normalised rows through act_rht_quant_i8: the same bytes."""
    x, res, w, signs = rows(20, 2048, 5)
    _h, y, q, s = run(x, res, w, signs)
    xq, xs = C.gpu_quant_acts(y, signs)
    assert np.array_equal(C.host(xq).reshape(-1), q) and np.array_equal(C.host(xs), s)


def test_a_prompt_block_feeds_the_linear():
    """Rows 32 .. 40 of a 41-row call, as they lie, into w4a8_linear: the same
    result as quantizing these nine rows by themselves."""
    K, Nrow = 512, 48
    x, res, w, signs = rows(41, K, 6)
    wt = C.gpu_prepare(np.random.default_rng(1).standard_normal((Nrow, K)).astype(np.float32), signs, "w4_z16", 64)
    xq = torch.empty(41 * K, dtype=torch.int8, device=C.DEV)
    xs = torch.empty(41, device=C.DEV)
    y = torch.empty((41, K), device=C.DEV)
    svg.add_rmsnorm_quant_i8(x.to(C.DEV), C.to_dev(res), w.to(C.DEV), EPS, C.to_dev(signs), xq, xs, y=y)
    got, _ = C.gpu_linear(xq[32 * K:].view(9, K), xs[32:], wt, debug=False)
    q2, s2 = C.gpu_quant_acts(C.host(y)[32:], signs)
    ref, _ = C.gpu_linear(q2, s2, wt, debug=False)
    assert np.array_equal(C.host(got), C.host(ref))


def test_in_a_captured_graph_and_on_another_stream():
    x, res, w, signs = rows(16, 4096, 8)
    xd, wd, sd = x.to(C.DEV), w.to(C.DEV), C.to_dev(signs)
    r0 = C.to_dev(res)
    r = r0.clone()
    xq = torch.empty((16, 4096), dtype=torch.int8, device=C.DEV)
    xs = torch.empty(16, device=C.DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        svg.add_rmsnorm_quant_i8(xd, r, wd, EPS, sd, xq, xs)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svg.add_rmsnorm_quant_i8(xd, r, wd, EPS, sd, xq, xs)
    for turn in range(3):
        xd.copy_(x.to(C.DEV) * (turn + 1))
        r.copy_(r0)
        xq.zero_()
        g.replay()
        torch.cuda.synchronize()
        _h, _u, q, s = N.norm_quant((x * (turn + 1)).numpy(), res, w.numpy(), EPS, signs, 32)
        assert np.array_equal(C.host(xs), s) and np.array_equal(C.host(xq).reshape(-1), N.slab_codes(q))
