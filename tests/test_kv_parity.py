"""The cache's pages on the device against the oracle (oracle/cache_oracle.py):
tables, counts and every 16-bit pattern of the pool, equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache_oracle as CO

pytestmark = pytest.mark.gpu


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


def new_rows(seed, S, T, H, dim, kind, extra=0):
    """fp32 rows as slices of a wider matrix, and their rounded patterns [S, T, H, dim]."""
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn((S * T, 2 * H * dim + extra), generator=g)
    k, v = wide[:, :H * dim], wide[:, H * dim:2 * H * dim]
    pat = lambda t: K.bits(t.contiguous().to(K.TYPES[kind])).reshape(S, T, H, dim)  # noqa: E731
    d = wide.to(C.DEV)
    return d[:, :H * dim], d[:, H * dim:2 * H * dim], pat(k), pat(v)


@pytest.mark.parametrize("lens,T,H,dim,page,kind", [
    ([0], 1, 1, 64, 32, "fp16"), ([5], 7, 2, 64, 32, "bf16"), ([31, 0, 64], 4, 3, 128, 32, "fp16"),
    ([30, 63, 127, 2], 32, 2, 256, 64, "bf16"), ([100], 300, 2, 128, 128, "fp16"), ([1, 2, 3, 4, 5], 3, 32, 64, 64, "bf16"),
])
def test_append(lens, T, H, dim, page, kind):
    C.say(f"kv_append lens={lens} T={T} H={H} dim={dim} page={page} {kind}")
    S = len(lens)
    c = K.make(T * 7 + dim, lens, T, L=2, H=H, dim=dim, page=page)
    cache = K.to_library(svg, c, kind)
    k, v, kp, vp = new_rows(T, S, T, H, dim, kind, extra=8)
    svg.kv_append(cache, 1, k, v, T)
    CO.append(c, 1, kp, vp, T)
    K.same(cache, c)
    # again with unequal numbers of rows, some slots idle, one number past T
    n = [(5 * s + 2) % (T + 2) - 1 for s in range(S)]
    n[-1] = T + 9
    k, v, kp, vp = new_rows(T + 1, S, T, H, dim, kind)
    svg.kv_append(cache, 0, k, v, T, n_rows=i32(n))
    CO.append(c, 0, kp, vp, T, n)
    K.same(cache, c)


def test_append_rounds_once_and_keeps_special_values():
    c = K.make(1, [3], 4, H=1, dim=64)
    for kind in ("fp16", "bf16"):
        cache = K.to_library(svg, c, kind)
        x = torch.randn((4, 64), generator=torch.Generator().manual_seed(2)) * 10 ** torch.linspace(-9, 9, 64)
        x[0, :6] = torch.tensor([float("inf"), -float("inf"), 65520.0, 1e-8, -0.0, 3.3895e38])
        svg.kv_append(cache, 0, x.to(C.DEV), (-x).to(C.DEV), 4)
        ref = K.copy_of(c)
        CO.append(ref, 0, K.bits(x.to(K.TYPES[kind])).reshape(1, 4, 1, 64), K.bits((-x).to(K.TYPES[kind])).reshape(1, 4, 1, 64), 4)
        K.same(cache, ref)


def test_append_outside_the_pages_writes_nothing_there():
    """No page for the position, a page number outside the pool, a row count
    outside the table, a negative length: those rows are passed over."""
    c = K.make(4, [20, 40, 10, 7, 9], 12, H=2, dim=64, page=32)
    c["pages"][0] = 0
    c["table"][1, 1] = 10 ** 6
    c["table"][2, 0] = -5
    c["pages"][3] = 99
    c["len"][4] = -3
    cache = K.to_library(svg, c)
    k, v, kp, vp = new_rows(9, 5, 30, 2, 64, "fp16")
    svg.kv_append(cache, 0, k, v, 30)
    CO.append(c, 0, kp, vp, 30)
    K.same(cache, c)


def paths(rng, S, T, counts):
    path = np.full((S, T), -1, np.int32)
    for s in range(S):
        path[s, :counts[s] - 1] = np.sort(rng.choice(np.arange(1, T), size=counts[s] - 1, replace=False))
    return path


@pytest.mark.parametrize("lens,T,L,H,dim,page,kind", [
    ([0], 1, 1, 1, 64, 32, "fp16"), ([7], 2, 2, 2, 64, 32, "bf16"), ([31, 32, 1, 50], 16, 3, 2, 128, 32, "fp16"),
    ([120, 1, 63], 32, 2, 3, 256, 64, "bf16"), ([127], 32, 1, 8, 128, 128, "fp16"),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit(lens, T, L, H, dim, page, kind, in_place):
    C.say(f"kv_commit lens={lens} T={T} L={L} H={H} dim={dim} page={page} {kind} in_place={in_place}")
    S = len(lens)
    rng = np.random.default_rng(T + dim)
    c = K.make(T + dim, lens, T, L=L, H=H, dim=dim, page=page)
    cache = K.to_library(svg, c, kind)
    counts = [int(rng.integers(1, T + 1)) for _ in lens]
    counts[0] = T
    path = paths(rng, S, T, counts)
    out = torch.full((S,), -9, dtype=torch.int32, device=C.DEV)
    svg.kv_commit(cache, i32(path), i32(counts), None if in_place else out)
    new = CO.commit(c, path, counts)
    if in_place:
        c["len"] = new
    else:
        assert np.array_equal(C.host(out), new)
    K.same(cache, c)


def test_commit_refuses_bad_paths():
    T, lens = 6, [10, 11, 12, 13, 14, 15, 16, 17]
    c = K.make(3, lens, T, L=2)
    path = np.tile(np.array([1, 3, 5, -1, -1, -1], np.int32), (8, 1))
    n = np.full(8, 4)
    n[0], n[1] = 0, T + 1
    path[2, 1] = 1                   # not rising
    path[3, 2] = T                   # outside the tree
    path[4, 0] = 0                   # the root again
    c["pages"][5] = 0                # no pages
    c["table"][6, 0] = -1            # not a page
    cache = K.to_library(svg, c)
    out = torch.zeros(8, dtype=torch.int32, device=C.DEV)
    svg.kv_commit(cache, i32(path), i32(n), out)
    new = CO.commit(c, path, n)
    assert list(new[:7]) == lens[:7] and new[7] == 21
    assert np.array_equal(C.host(out), new)
    K.same(cache, c)


def check_state(cache, c, status=None, ref=None):
    K.same(cache, c)
    assert np.array_equal(CO.holders(c), c["refs"])
    if status is not None:
        assert np.array_equal(C.host(status), ref)


def test_fork_keep_free_and_reserve():
    """Branching as a search does it, several turns: forks of one slot, kept slots, freed ones, a
    number outside the slots, then room for new tokens; the tables after each."""
    rng = np.random.default_rng(5)
    lens = [40, 64, 5, 0, 33, 96]
    c = K.make(6, lens, 0, L=2, H=1, dim=64, spare=14)
    a = K.to_library(svg, c)
    b = a.other_tables()
    ws, status = svg.kv_workspace(a), torch.zeros(6, dtype=torch.int32, device=C.DEV)
    b.table.fill_(-1)
    turns = [[0, 0, 0, 3, 4, 0], [1, 0, -1, 2, 99, 4], [0, 1, 2, 3, 4, 5], [5, 5, 5, 5, 5, 5], [-1, 0, -7, 0, -1, 0], [3, 3, 3, 3, 3, 3]]
    for t, src in enumerate(turns):
        b.table.fill_(-1)
        svg.kv_fork(a, i32(src), b)
        c = CO.fork(c, src)
        check_state(b, c)
        need = rng.integers(-1, 45, 6)
        svg.kv_reserve(b, i32(need), status, ws)
        ref = CO.reserve(c, need)
        check_state(b, c, status, ref)
        grown = np.where((ref == 0) & (need > 0), need, 0)
        c["len"] += grown.astype(np.int32)
        b.len += i32(grown)
        a, b = b, a


@pytest.mark.parametrize("spare", [0, 1, 2, 3, 5, 9])
def test_reserve_with_too_few_pages(spare):
    """A shortage: slots are served in order, all or nothing; a slot that got
    nothing does not change what the ones behind it see."""
    lens = [33, 1, 40, 64, 0, 20, 70]
    c = K.make(7, lens, 0, L=1, H=2, dim=64, spare=spare)
    a = K.to_library(svg, c)
    b = a.other_tables()
    src = [0, 0, 0, 3, 4, 0, 6]
    svg.kv_fork(a, i32(src), b)
    c = CO.fork(c, src)
    need = [40, 1, 1, 90, 2, 33, 0]
    status = torch.zeros(7, dtype=torch.int32, device=C.DEV)
    svg.kv_reserve(b, i32(need), status, svg.kv_workspace(b))
    ref = CO.reserve(c, need)
    c2 = dict(c)
    tab = b.table.cpu().numpy()
    for s in range(7):  # entries behind a row's pages are not part of the state
        tab[s, c["pages"][s]:] = c["table"][s, c["pages"][s]:]
    c2["table"] = tab
    K.same(b, c2)
    assert np.array_equal(tab, c["table"])
    assert np.array_equal(C.host(status), ref)
    assert np.array_equal(CO.holders(c), c["refs"])


def test_reserve_refuses_slots_that_do_not_fit():
    c = K.make(8, [10, 20, 30, 40, 50], 0, spare=40, width=4)
    c["len"][0] = -1
    c["len"][1] = 10 ** 6
    c["table"][2, 0] = 77777
    c["pages"][4] = 9
    cache = K.to_library(svg, c)
    need = [5, 5, 5, 4 * 32 - 40 + 1, 5]
    status = torch.zeros(5, dtype=torch.int32, device=C.DEV)
    svg.kv_reserve(cache, i32(need), status, svg.kv_workspace(cache))
    assert list(C.host(status)) == [2, 2, 2, 2, 2]
    K.same(cache, c)
    need[3] -= 1                      # exactly the row's width
    c["len"][0], c["len"][1], c["table"][2, 0], c["pages"][4] = 10, 20, int(np.flatnonzero(c["refs"] == 1)[0]), 2
    cache = K.to_library(svg, c)
    svg.kv_reserve(cache, i32([2 ** 31 - 1, 2 ** 31 - 1, 0, need[3], -2 ** 31]), status, svg.kv_workspace(cache))
    ref = CO.reserve(c, [2 ** 31 - 1, 2 ** 31 - 1, 0, need[3], -2 ** 31])
    assert list(C.host(status)) == list(ref) == [2, 2, 0, 0, 0]
    K.same(cache, c)


def test_reserve_many_slots_and_a_large_pool():
    """1024 slots, a pool of pages that is searched in many turns."""
    rng = np.random.default_rng(9)
    lens = rng.integers(0, 130, 1024)
    c = K.make(10, [int(n) for n in lens], 0, L=1, H=1, dim=64, page=64, spare=3000)
    a = K.to_library(svg, c)
    b = a.other_tables()
    src = np.where(rng.random(1024) < 0.5, np.arange(1024), rng.integers(0, 40, 1024))
    svg.kv_fork(a, i32(src), b)
    c = CO.fork(c, src)
    need = rng.integers(0, 200, 1024)
    status = torch.zeros(1024, dtype=torch.int32, device=C.DEV)
    svg.kv_reserve(b, i32(need), status, svg.kv_workspace(b))
    ref = CO.reserve(c, need)
    check_state(b, c, status, ref)


@pytest.mark.parametrize("n,L,H,dim,page,kind", [(1, 1, 1, 64, 32, "fp16"), (7, 3, 2, 128, 64, "bf16"), (40, 2, 5, 256, 128, "fp16")])
def test_copy_pages(n, L, H, dim, page, kind):
    c = K.make(n, [1], 0, L=L, H=H, dim=dim, page=page, spare=2 * n + 5)
    cache = K.to_library(svg, c, kind)
    ids = np.random.default_rng(n).permutation(2 * n + 5)
    src, dst = ids[:n].copy(), ids[n:2 * n].copy()
    if n > 3:
        src[1], dst[2] = -1, 10 ** 7      # passed over
    svg.kv_copy_pages(cache, i32(src), i32(dst))
    CO.copy_pages(c, src, dst)
    K.same(cache, c)


def test_in_a_captured_graph():
    """append, commit in place, fork and reserve captured once and replayed, each replay against the oracle."""
    lens, T = [30, 45, 7], 8
    c = K.make(12, lens, 3 * T + 40, L=2, spare=20)
    a = K.to_library(svg, c)
    b = a.other_tables()
    k, v, kp, vp = new_rows(3, 3, T, 2, 64, "fp16")
    path, n = paths(np.random.default_rng(1), 3, T, [4, 1, 8]), [4, 1, 8]
    pd, nd, sd = i32(path), i32(n), i32([0, 0, 2])
    need, status, ws = i32([9, 9, 9]), i32([0, 0, 0]), svg.kv_workspace(a)

    def step():
        for layer in range(2):
            svg.kv_append(a, layer, k, v, T)
        svg.kv_commit(a, pd, nd)
        svg.kv_fork(a, sd, b)
        svg.kv_reserve(b, need, status, ws)
        for x, y in ((a.table, b.table), (a.pages, b.pages), (a.len, b.len)):
            x.copy_(y)

    def ref(c):
        for layer in range(2):
            CO.append(c, layer, kp, vp, T)
        c["len"] = CO.commit(c, path, n)
        c = CO.fork(c, [0, 0, 2])
        assert not CO.reserve(c, [9, 9, 9]).any()
        return c

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.table.fill_(-1)
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    c = ref(c)
    live = lambda t, n: [list(map(int, r[:m])) for r, m in zip(t, n)]  # noqa: E731
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _turn in range(2):
        g.replay()
        torch.cuda.synchronize()
        c = ref(c)
        K.same(a, c, ("k", "v", "pages", "len", "refs"))
        assert live(C.host(a.table), c["pages"]) == live(c["table"], c["pages"])
