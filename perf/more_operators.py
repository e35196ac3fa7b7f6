"""What is timed of a prompt's pass through a decoder layer: the map from packed rows to their slots, positions and
places in the paged cache; rotary positions with the rows' keys and values written into the pages; causal attention of
the rows over the cache; the integer products of many rows; the gated activation with rotation and int8 codes.

``own`` False computes each step in its plain form (torch, 32 bits, 64 where a rounding decides a code and for angles);
True makes the library's calls.  Page layout (one layer, one page, one head, PS tokens of D values, 16-bit):
  K  [PS/16][D/32][4][16][8]:  token 16 a + c, value 32 b + 8 g + e  at [a][b][g][c][e]
  V  [PS/32][D/16][4][16][2][4]:  token 32 a + 16 h + 4 g + j, value 16 b + c  at [a][b][g][c][h][j]
Codes of activations: 32 rows at a time, [K/32][rows][32].  Weights: 16-row tiles, W8 [N/16][K/64][4][16][16], W4 (two
codes a byte) [N/16][K/128][4][16][2 halves][2 words][4 bytes], parameters [N/16][K/512][16][512/group].
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the rows of a verify pass: 8 slots of 16 nodes, trees of unequal size
        dict(name="rows_verify", op="rows", S=8, T=16, new=16, ctx=3000, page=64, spare=7),
        # the packed prompts of a full batch, of every length from none on; some slots have no pages left, or shared ones
        dict(name="rows_prompts", op="rows", S=512, T=0, new=900, ctx=2000, page=32, spare=100),
        # a verify pass's rotation and append: heads of the 32-layer stack shared by four, fp32 rows of the projection
        dict(name="rope_verify", op="rope", S=4, T=8, new=8, ctx=5000, Hkv=8, G=4, D=128, rot=128, pair="half", page=64,
             x="fp32", q="fp32", type="fp16"),
        # a prompt's: 16-bit rows, half of each head rotated, interleaved pairs, far positions
        dict(name="rope_prompt", op="rope", S=3, T=0, new=2000, ctx=100000, Hkv=8, G=4, D=128, rot=64, pair="interleaved",
             page=64, x="bf16", q="bf16", type="bf16"),
        # one step of a serving batch: a few prompts' chunks among single tokens, wide heads
        dict(name="attn_step", op="attn", S=24, mix=True, new=300, ctx=4000, Hkv=2, G=8, D=256, page=32, type="bf16"),
        # a whole prompt over the stack's own heads (32 of 128, no sharing)
        dict(name="attn_prompt", op="attn", S=1, mix=False, new=4099, ctx=0, Hkv=32, G=1, D=128, page=64, type="fp16"),
        # a chunk of a long prompt behind what is cached of it, heads shared by four
        dict(name="attn_chunk", op="attn", S=1, mix=False, new=1000, ctx=30001, Hkv=8, G=4, D=128, page=128, type="bf16"),
        # the o projection of a short prompt
        dict(name="linear_short", op="linear", fmt="w8", group=0, M=40, N=4096, K=4096, y="fp32"),
        # gate and up of a long prompt
        dict(name="linear_w8", op="linear", fmt="w8", group=0, M=4099, N=24576, K=4096, y="bf16"),
        # down of an ordinary one, 4-bit weights
        dict(name="linear_w4", op="linear", fmt="w4_z16", group=64, M=1001, N=4096, K=12288, y="fp32"),
        # the input of a short prompt's o projection: attention's rows, no gate
        dict(name="quant_short", op="quant", M=40, K=4096, block=32, x="fp16", gate=False),
        # the input of a long prompt's down projection: gate and up side by side in the rows of one product
        dict(name="quant_gate", op="quant", M=4099, K=12288, block=32, x="bf16", gate=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rows", "rope", "attn", "attn", "attn", "linear", "linear", "linear", "quant"])
    kind = rng.choice(["fp16", "bf16"])
    page = rng.choice([32, 64, 128])
    if op == "rows":
        T = rng.choice([0, 0, 1, log(2, 32)])
        S = log(1, 512)
        return dict(op="rows", S=S, T=T, new=log(1, T) if T else log(1, 65536 // S), ctx=log(1, 3000), page=page,
                    spare=rng.choice([0, log(1, 200)]))
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 32])
    G = rng.choice([1, 2, 3, 4, 7, 8])
    if op == "rope":
        S = log(1, 32)
        T = rng.choice([0, 0, 1, log(2, 32)])
        most = max(1, (1 << 24) // (S * Hkv * (G + 2) * D))
        new = log(1, min(T, most)) if T else log(1, max(1, min(4099 // S, most)))
        return dict(op="rope", S=S, T=T, new=new, ctx=log(1, min(200000, (1 << 28) // (Hkv * D)) // S), Hkv=Hkv, G=G, D=D,
                    rot=rng.choice([D, D, D // 2, D // 4]), pair=rng.choice(["half", "interleaved"]), page=page,
                    x=rng.choice(["fp32", kind]), q=rng.choice(["fp32", kind]), type=kind)
    if op == "attn":
        S = rng.choice([1, 1, log(2, 32)])
        new, ctx = log(1, 4099), rng.choice([0, log(1, 30001)])
        # no more products than the largest listed case has, and scores that fit the plain form
        A = Hkv * G
        new = max(1, min(new, int(math.sqrt(1e9 / (S * A)))))
        ctx = int(max(0, min(ctx, 9e8 / (S * new * A) - new, 1.2e11 / (S * new * A * D) - new, 2.5e8 / (S * Hkv * D))))
        return dict(op="attn", S=S, mix=S > 2 and rng.random() < 0.5, new=new, ctx=ctx, Hkv=Hkv, G=G, D=D, page=page, type=kind)
    if op == "linear":
        fmt = rng.choice(["w8", "w4_z16", "w4_z4"])
        step = 32 if fmt == "w8" else 128
        K = step * log(max(1, 256 // step), 12288 // step)
        N = log(16, 24576)
        return dict(op="linear", fmt=fmt, group=0 if fmt == "w8" else rng.choice([32, 64, 64, 128]), M=log(1, 4099), N=N,
                    K=min(K, step * max(1, int(1e8 / N) // step)), y=rng.choice(["fp32", "fp16", "bf16"]))
    block = rng.choice([32, 64])
    return dict(op="quant", M=log(1, 4099), K=block * log(512 // block, 12288 // block), block=block,
                x=rng.choice(["fp32", "fp16", "bf16"]), gate=rng.random() < 0.6)


def counts_of(case):
    """New rows of each slot."""
    S, new, s = case["S"], case["new"], np.arange(case["S"], dtype=np.int64)
    if case["op"] == "attn" and case["mix"]:
        return np.where(s % 4 == 0, np.maximum(1, new - (3 * s % S) * new // S), 1)
    n = new - (5 * s % S) * new // S
    if case["op"] != "attn" and S > 2:
        n[S // 2] = 0  # a slot that takes no part
    return n


def lens_of(case):
    """Committed tokens of each slot (all of ctx for slot 0)."""
    s = np.arange(case["S"], dtype=np.int64)
    return case["ctx"] - (3 * s % case["S"]) * case["ctx"] // case["S"]


def row_space(case):
    """Rows of a step's buffers: T a slot, or the packed ones."""
    T = case.get("T", 0)
    return case["S"] * T if T else int(counts_of(case).sum())


# ------------------------------------------------------------ inputs, per case
def generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def i32(v):
    return torch.as_tensor(np.ascontiguousarray(v), dtype=torch.int32, device=DEV)


def tree_parents(g, S, T):
    """Random draft trees: parent[0] = -1, parent[i] < i, mostly the node before."""
    i = torch.arange(T, device=DEV)
    other = (torch.rand((S, T), device=DEV, generator=g) * i).long().clamp(max=(i - 1).clamp(min=0))
    parent = torch.where(torch.rand((S, T), device=DEV, generator=g) < 0.6, i - 1, other)
    parent[:, 0] = -1
    return parent.int()


def slot_tables(g, case, spare=4):
    """Pages for each slot's committed and new tokens, in shuffled order over the pool."""
    S, PS = case["S"], case["page"]
    lens = lens_of(case)
    held = -(-(lens + np.maximum(counts_of(case), case.get("T", 0))) // PS)
    n_pages = int(held.sum()) + spare + 1
    width = int(held.max()) + 2
    ids = torch.randperm(n_pages, device=DEV, generator=g)
    col = torch.arange(width, device=DEV)[None, :]
    has = i32(held).long()[:, None]
    first = has.cumsum(0) - has
    table = torch.where(col < has, ids[(first + col).clamp(max=n_pages - 1)], -1).int()
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    refs[ids[:int(held.sum())]] = 1
    return dict(table=table, pages=i32(held), len=i32(lens), refs=refs), n_pages


def pools(g, case, n_pages):
    shape = (1, n_pages, case["Hkv"], case["page"] * case["D"])
    t = TYPES[case["type"]]
    return (torch.randn(shape, device=DEV, generator=g, dtype=t), torch.randn(shape, device=DEV, generator=g, dtype=t))


def row_map(case, s):
    """Start and count of each slot, position and place of each row, as a step keeps them."""
    n, start, slot, i = rows_of(case["T"], row_space(case), s["n_new"])
    live = slot >= 0
    at = slot.clamp(min=0)
    where = s["len"].long()[at] + i
    page = torch.gather(s["table"][at].long(), 1, (where // case["page"])[:, None])[:, 0]
    place = torch.where(live, page * case["page"] + where % case["page"], -1)
    pos = torch.where(live, s["len"].long()[at] + depth_of(s, at, i), -1)
    return dict(start=start.int(), count=n.int(), pos=pos.int(), place=place.int())


def prepare(case, seed):
    g = generator(seed)
    op = case["op"]
    s = {"case": dict(case), "op": op}
    if op == "linear":
        return prepare_linear(g, case, s)
    if op == "quant":
        M, K = case["M"], case["K"]
        t = TYPES[case["x"]]
        if case["gate"]:
            rows = (2 * torch.randn((M, 2 * K), device=DEV, generator=g)).to(t)  # gate and up of one product
            s["gate"], s["x"] = rows[:, :K], rows[:, K:]
        else:
            s["gate"], s["x"] = None, torch.randn((M, K), device=DEV, generator=g).to(t)
        s["x"][:, torch.randperm(K, device=DEV, generator=g)[:4]] *= 20  # channels far above the rest
        s["signs"] = (torch.randint(0, 2, (K,), device=DEV, generator=g) * 2 - 1).to(torch.int8)
        s["xq"] = torch.zeros((M, K), dtype=torch.int8, device=DEV)
        s["x_scale"] = torch.zeros(M, device=DEV)
        return s
    state, n_pages = slot_tables(g, case, case.get("spare", 4))
    s.update(state)
    S, R = case["S"], row_space(case)
    s["n_new"] = i32(counts_of(case))
    T = case.get("T", 0)
    s["parent"] = tree_parents(g, S, T) if T else None
    if op == "rows":
        if case["spare"]:
            # slots that were refused: a page too few, or a page that another slot holds too
            s["pages"][S // 3] = (s["pages"][S // 3] - 1).clamp(min=0)
            s["refs"][s["table"][S // 4, (s["len"][S // 4] // case["page"]).long()].long()] = 2
        R += 0 if T else case["spare"]  # packed buffers longer than the rows
        s.update(start=torch.zeros(S, dtype=torch.int32, device=DEV), count=torch.zeros(S, dtype=torch.int32, device=DEV),
                 slot=torch.zeros(R, dtype=torch.int32, device=DEV), pos=torch.zeros(R, dtype=torch.int32, device=DEV),
                 place=torch.zeros(R, dtype=torch.int32, device=DEV))
        s["k"], s["v"] = (torch.zeros((1, n_pages, 1, case["page"] * 64), dtype=torch.float16, device=DEV) for _ in range(2))
        return s
    Hkv, G, D = case["Hkv"], case["G"], case["D"]
    A = Hkv * G
    s["k"], s["v"] = pools(g, case, n_pages)
    if op == "rope":
        s["map"] = row_map(case, s)
        rows = torch.randn((R, (A + 2 * Hkv) * D), device=DEV, generator=g).to(TYPES[case["x"]])  # a fused projection's output
        s["q"], s["k_new"], s["v_new"] = (t.unflatten(1, (-1, D)) for t in rows.split([A * D, Hkv * D, Hkv * D], 1))
        s["q_out"] = torch.zeros((R, A, D), dtype=TYPES[case["q"]], device=DEV)
        # base 500000, positions stretched by 4
        e = torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEV) / case["rot"]
        s["freq"] = 500000.0 ** -e / 4
        s["amplitude"] = 1.0 + 0.1 * math.log(4.0)
        return s
    n, start, slot, i = rows_of(0, R, s["n_new"])
    s.update(start=start.int(), count=n.int(), slot=slot, index=i)
    s["q"] = torch.randn((R, A, D), device=DEV, generator=g)
    s["q"] *= torch.linspace(0.5, 3.0, A, device=DEV)[None, :, None]  # flat heads and peaked ones
    s["q"] = s["q"].to(TYPES[case["type"]])
    s["out"] = torch.zeros_like(s["q"])
    s["scale"] = 1.0 / math.sqrt(D)
    return s


def prepare_linear(g, case, s):
    M, N, K, fmt = (case[k] for k in ("M", "N", "K", "fmt"))
    x = (torch.randn((M, K), device=DEV, generator=g) * 35).round().clamp(-127, 127).to(torch.int8)
    s["xq"] = to_slabs(x, M, K).view(M, K)
    s["x_scale"] = torch.rand(M, device=DEV, generator=g) * 1e-3 + 1e-4
    s["y"] = torch.zeros((M, N), dtype=TYPES[case["y"]], device=DEV)
    Np = ceil_div(N, 16) * 16
    if fmt == "w8":
        Kp = ceil_div(K, 64) * 64
        w = torch.zeros((Np, Kp), dtype=torch.int8, device=DEV)
        w[:N, :K] = (torch.randn((N, K), device=DEV, generator=g) * 30).round().clamp(-127, 127).to(torch.int8)
        s["wq"] = w.view(Np // 16, 16, Kp // 64, 4, 16).permute(0, 2, 3, 1, 4).reshape(-1)
        s["w_scale"] = (torch.rand(N, device=DEV, generator=g) * 2e-3 + 1e-3).half()
        s["w_zero"] = None
        return s
    group, Kp = case["group"], ceil_div(K, 128) * 128
    w = torch.zeros((Np, Kp), dtype=torch.uint8, device=DEV)
    w[:N, :K] = (torch.randn((N, K), device=DEV, generator=g) * 2.7 + 7.5).round().clamp(0, 15).to(torch.uint8)
    w = w.view(Np // 16, 16, Kp // 128, 2, 4, 2, 2, 4).permute(0, 2, 4, 1, 3, 5, 6, 7)  # [i][j][b][r][half][word][nibble][byte]
    s["wq"] = (w[..., 0, :] | (w[..., 1, :] << 4)).reshape(-1)
    KB, per = ceil_div(K, 512), 512 // group
    scale = torch.zeros((Np, KB * per), device=DEV)
    zero = torch.zeros((Np, KB * per), dtype=torch.uint8, device=DEV)
    scale[:N, :K // group] = torch.rand((N, K // group), device=DEV, generator=g) * 2e-2 + 1e-2
    zero[:N, :K // group] = torch.randint(5, 11, (N, K // group), device=DEV, generator=g).to(torch.uint8)
    scale, zero = (t.view(Np // 16, 16, KB, per).permute(0, 2, 1, 3).reshape(-1) for t in (scale, zero))
    s["w_scale"] = scale.half()
    s["w_zero"] = zero.half() if fmt == "w4_z16" else zero[0::2] | (zero[1::2] << 4)
    return s


def ceil_div(a, b):
    return -(-a // b)


def to_slabs(code, M, K):
    full = M // 32 * 32
    a = code[:full].view(full // 32, 32, K // 32, 32).permute(0, 2, 1, 3).reshape(-1)
    b = code[full:].view(M - full, K // 32, 32).permute(1, 0, 2).reshape(-1)
    return torch.cat((a, b))


def from_slabs(xq, M, K):
    full = M // 32 * 32
    flat = xq.view(-1)
    a = flat[:full * K].view(full // 32, K // 32, 32, 32).permute(0, 2, 1, 3).reshape(full, K)
    b = flat[full * K:].view(K // 32, M - full, 32).permute(1, 0, 2).reshape(M - full, K)
    return torch.cat((a, b))


# ------------------------------------------------------------------ one pass
def run(state):
    return PASSES[state["op"]](state)


def library():
    import speculative_verify_gemm_amd as svg
    return svg


def cache_of(s):
    """The library's handle of the state's cache, made once as a program keeps it."""
    if "cache" not in s:
        D = s["case"].get("D", 64)
        s["cache"] = library().KVCache(s["k"], s["v"], s["table"], s["pages"], s["len"], s["refs"], dim=D, page=s["case"]["page"])
    return s["cache"]


def rows_of(T, R, n_new):
    """(count, start) of each slot and (slot, index in it) of each row (-1 and 0 where there is none)."""
    S = n_new.shape[0]
    r = torch.arange(R, device=DEV)
    if T:
        n = n_new.long().clamp(0, T)
        slot, i = r // T, r % T
        live = i < n[slot]
        return n, torch.arange(S, device=DEV) * T, torch.where(live, slot, -1), torch.where(live, i, 0)
    n = n_new.long().clamp(min=0)
    end = n.cumsum(0)
    start = (end - n).clamp(max=R)
    slot = torch.searchsorted(end, r, right=True)
    live = slot < S
    i = r - start[slot.clamp(max=S - 1)]
    return torch.minimum(n, R - start), start, torch.where(live, slot, -1), torch.where(live, i, 0)


def depth_of(s, slot, i):
    """Steps of each row behind its slot's committed tokens: its node's depth in the tree, its index in a chain."""
    if s["parent"] is None:
        return i
    S, T = s["parent"].shape
    link = torch.zeros((S, T, T + 1), device=DEV).scatter_(2, (s["parent"].long() % (T + 1))[..., None], 1.0)[..., :T]
    above = (torch.matrix_power(torch.eye(T, device=DEV) + link, T) > 0).sum(2) - 1  # [S, T] nodes above each
    return above[slot, i]


def run_rows(s):
    c = s["case"]
    if own:
        if "rows" not in s:
            s["rows"] = library().RowMap(s["start"], s["count"], s["pos"], s["place"], s["slot"])
        library().kv_row_map(cache_of(s), s["n_new"], s["rows"], T=c["T"], parent=s["parent"])
    else:
        PS = c["page"]
        n, start, slot, i = rows_of(c["T"], s["slot"].shape[0], s["n_new"])
        live = slot >= 0
        at = slot.clamp(min=0)
        where = s["len"].long()[at] + i
        entry = where // PS
        page = torch.gather(s["table"][at], 1, entry.clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()
        fine = live & (entry < s["pages"][at]) & (page >= 0) & (page < s["refs"].shape[0])
        fine &= s["refs"][page.clamp(0, s["refs"].shape[0] - 1)] <= 1
        s["start"].copy_(start)
        s["count"].copy_(n)
        s["slot"].copy_(slot)
        s["pos"].copy_(torch.where(live, s["len"].long()[at] + depth_of(s, at, i), -1))
        s["place"].copy_(torch.where(fine, page * PS + where % PS, -1))
    return {k: s[k] for k in ("start", "count", "slot", "pos", "place")}


def rotated(x, c, s, pair, rot):
    """x [R, heads, D] fp32 by the angles' cos and sin [R, 1, rot / 2]."""
    turn, rest = x[..., :rot], x[..., rot:]
    if pair == "half":
        a, b = turn[..., :rot // 2], turn[..., rot // 2:]
        turn = torch.cat((a * c - b * s, b * c + a * s), -1)
    else:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    return torch.cat((turn, rest), -1)


def run_rope(s):
    c = s["case"]
    m = s["map"]
    if own:
        svg = library()
        if "rows" not in s:
            s["rows"] = svg.RowMap(m["start"], m["count"], m["pos"], m["place"])
            s["rope"] = svg.Rope(s["freq"], interleaved=c["pair"] == "interleaved", amplitude=s["amplitude"])
        svg.rope_append(cache_of(s), 0, s["rows"], s["rope"], s["q"], s["k_new"], s["v_new"], s["q_out"])
    else:
        angle = m["pos"].double()[:, None] * s["freq"][None, :]
        cs, sn = ((f(angle) * s["amplitude"]).float()[:, None, :] for f in (torch.cos, torch.sin))
        q = rotated(s["q"].float(), cs, sn, c["pair"], c["rot"])
        k = rotated(s["k_new"].float(), cs, sn, c["pair"], c["rot"])
        live = m["place"] >= 0
        s["q_out"].copy_(torch.where((m["pos"] >= 0)[:, None, None], q, s["q_out"].float()))
        # the rows that have a place, written to it
        ty, H, D, PS = TYPES[c["type"]], c["Hkv"], c["D"], c["page"]
        at = m["place"][live].long()
        page, t = at // PS, at % PS
        P = s["k"].shape[1]
        kv = s["k"].view(P, H, PS // 16, D // 32, 4, 16, 8)
        vv = s["v"].view(P, H, PS // 32, D // 16, 4, 16, 2, 4)
        kv[page, :, t // 16, :, :, t % 16, :] = k[live].to(ty).view(-1, H, D // 32, 4, 8)
        a = t % 32
        vv[page, :, t // 32, :, (a % 16) // 4, :, a // 16, a % 4] = s["v_new"][live].to(ty).reshape(-1, H, D // 16, 16)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def run_attn(s):
    c = s["case"]
    S, Hkv, G, D, PS = (c[k] for k in ("S", "Hkv", "G", "D", "page"))
    if own:
        svg = library()
        if "rows" not in s:
            R = s["q"].shape[0]
            s["rows"] = svg.RowMap(s["start"], s["count"], n_rows=R)
            s["workspace"] = svg.prompt_attention_workspace(cache_of(s), Hkv * G, R)
        svg.prompt_attention(cache_of(s), 0, s["rows"], s["q"], s["out"], s["workspace"], scale=s["scale"])
        return s["out"]
    most, longest = int(counts_of(c).max()), int((lens_of(c) + counts_of(c)).max())
    i = torch.arange(most, device=DEV)[None, :]
    row = (s["start"].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)                    # [S, most]
    q = s["q"].float()[row].view(S, most, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, most * G, D) * s["scale"]
    ids = s["table"][:, :ceil_div(longest, PS)].clamp(min=0).long()
    P = s["k"].shape[1]
    k = s["k"].view(P, Hkv, PS // 16, D // 32, 4, 16, 8)[ids].float()                         # [S, n, H, PS/16, D/32, 4, 16, 8]
    k = k.permute(0, 2, 1, 3, 6, 4, 5, 7).reshape(S, Hkv, -1, D)
    v = s["v"].view(P, Hkv, PS // 32, D // 16, 4, 16, 2, 4)[ids].float()                      # [S, n, H, PS/32, D/16, 4, 16, 2, 4]
    v = v.permute(0, 2, 1, 3, 7, 5, 8, 4, 6).reshape(S, Hkv, -1, D)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()).view(S, Hkv, most, G, -1)
    t = torch.arange(score.shape[-1], device=DEV)
    hidden = t[None, None, :] > (s["len"][:, None] + i)[..., None]                             # [S, most, L]
    score.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    p = torch.exp(score.sub_(score.amax(-1, keepdim=True)))
    o = torch.matmul(p.view(S, Hkv, most * G, -1), v) / p.sum(-1).view(S, Hkv, most * G, 1)
    o = o.view(S, Hkv, most, G, D).permute(0, 2, 1, 3, 4).reshape(S, most, Hkv * G, D)
    s["out"].copy_(o[s["slot"], s["index"]])
    return s["out"]


def run_linear(s):
    c = s["case"]
    M, N, K, fmt, group = (c[k] for k in ("M", "N", "K", "fmt", "group"))
    if own:
        if fmt == "w8":
            library().w8a8_prompt_linear(s["xq"], s["x_scale"], s["wq"], s["w_scale"], N, s["y"])
        else:
            library().w4a8_prompt_linear(s["xq"], s["x_scale"], s["wq"], s["w_scale"], s["w_zero"], fmt, group, N, s["y"])
        return s["y"]
    Np = ceil_div(N, 16) * 16
    x = from_slabs(s["xq"], M, K).float() * s["x_scale"][:, None]
    if fmt == "w8":
        w = s["wq"].view(Np // 16, -1, 4, 16, 16).permute(0, 3, 1, 2, 4).reshape(Np, -1)[:N, :K].float()
        w = w * s["w_scale"].float()[:, None]
    else:
        b = s["wq"].view(Np // 16, -1, 4, 16, 2, 2, 4)                       # [i][j][b][r][half][word][byte]
        code = torch.stack((b & 15, b >> 4), 6)                              # .. [word][nibble][byte]
        code = code.permute(0, 3, 1, 4, 2, 5, 6, 7).reshape(Np, -1)[:N, :K].float()
        z = s["w_zero"]
        if fmt == "w4_z4":
            z = torch.stack((z & 15, z >> 4), 1).view(-1)
        scale, zero = (t.view(Np // 16, -1, 16, 512 // group).permute(0, 2, 1, 3).reshape(Np, -1)[:N, :K // group].float()
                       for t in (s["w_scale"], z))
        w = ((code.view(N, K // group, group) - zero[..., None]) * scale[..., None]).view(N, K)
    s["y"].copy_(torch.matmul(x, w.t()))
    return s["y"]


def hadamard(u, B):
    """Sylvester's +/-1 transform of each run of B values, stage by stage (h = 1, 2, 4, ...)."""
    M, K = u.shape
    h = 1
    while h < B:
        v = u.view(M, K // (2 * h), 2, h)
        u = torch.stack((v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]), 2).view(M, K)
        h *= 2
    return u


def run_quant(s):
    c = s["case"]
    M, K, B = c["M"], c["K"], c["block"]
    if own:
        library().gated_quant_i8(s["x"], s["gate"], s["signs"], s["xq"], s["x_scale"], block=B)
        xq, scale = s["xq"], s["x_scale"]
    else:
        # the codes are defined by fp32 values, each rounded once from 64 bits, and fp32 steps after that
        u = s["x"].float()
        if s["gate"] is not None:
            a = s["gate"].double()
            u = (a / (1.0 + torch.exp(-a)) * s["x"].double()).float()
        u = hadamard(u * s["signs"].float(), B)
        amax = u.abs().amax(1, keepdim=True)
        sigma = (amax.double() / 127).float()
        code = torch.where(amax > 0, torch.round((u.double() / sigma.double()).float()).clamp(-127, 127), 0.0)
        scale = (sigma * (1.0 / B)).view(M)
        xq = to_slabs(code.to(torch.int8), M, K)
    return {"values": slabs(xq, scale, M, K), "scale": scale}


def slabs(xq, scale, M, K):
    """The values that codes in 32-row slab buffers stand for: the whole buffers, and the rest."""
    full, flat = M // 32 * 32, xq.view(-1)
    return [flat[:full * K].view(full // 32, K // 32, 32, 32) * scale[:full].view(full // 32, 1, 32, 1),
            flat[full * K:].view(K // 32, M - full, 32) * scale[full:].view(1, M - full, 1)]


PASSES = {"rows": run_rows, "rope": run_rope, "attn": run_attn, "linear": run_linear, "quant": run_quant}


# ------------------------------------------------------------------ the floor
def work(case):
    """Bytes and operations that a pass cannot do without."""
    op = case["op"]
    if op == "linear":
        M, N, K, g = (case[k] for k in ("M", "N", "K", "group"))
        w = N * K + 2 * N if case["fmt"] == "w8" else N * K // 2 + N * K // g * (4 if case["fmt"] == "w4_z16" else 2.5)
        return {"bytes": w + M * K + 4 * M + M * N * SIZE[case["y"]], "flops": 2.0 * M * N * K}
    if op == "quant":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (SIZE[case["x"]] * (2 if case["gate"] else 1) + 1) + K + 4 * M, "flops": 20.0 * M * K}
    n, lens, R = counts_of(case), lens_of(case), row_space(case)
    if op == "rows":
        met = int((n + case["page"] - 1).sum() // case["page"])
        return {"bytes": 12 * (R + case["spare"]) + 24 * case["S"] + 8 * met + (4 * R if case["T"] else 0), "flops": 0}
    H, G, D = case["Hkv"], case["G"], case["D"]
    if op == "rope":
        rows = int(n.sum())
        return {"bytes": rows * H * D * ((G + 2) * SIZE[case["x"]] + G * SIZE[case["q"]] + 4) + 8 * R + 4 * case["rot"],
                "flops": 3.0 * rows * H * (G + 1) * case["rot"]}
    pairs = int((n * lens + n * (n + 1) // 2).sum())
    return {"bytes": int((lens + n).sum()) * 4 * H * D + int(n.sum()) * 4 * H * G * D, "flops": 4.0 * D * H * G * pairs}


# ------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    if case["op"] == "rows":
        return None  # whole numbers
    s = prepare(case, seed)
    return {"rope": exact_rope, "attn": exact_attn, "linear": exact_linear, "quant": exact_quant}[case["op"]](case, s)


def exact_rope(c, s):
    rot, D, H, PS = c["rot"], c["D"], c["Hkv"], c["page"]
    m = {k: v.cpu().numpy() for k, v in s["map"].items()}
    ang = np.outer(m["pos"].astype(np.float64), s["freq"].cpu().numpy())
    turn = (np.cos(ang) + 1j * np.sin(ang)) * s["amplitude"]
    half = c["pair"] == "half"
    first = np.arange(rot // 2) if half else 2 * np.arange(rot // 2)
    second = first + (rot // 2 if half else 1)

    def turned(x):
        x = x.double().cpu().numpy()
        z = (x[..., first] + 1j * x[..., second]) * turn[:, None, :]
        y = x.copy()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q = np.where((m["pos"] >= 0)[:, None, None], turned(s["q"]), s["q_out"].double().cpu().numpy())
    new = {"k": turned(s["k_new"]), "v": s["v_new"].double().cpu().numpy()}
    t, d = np.meshgrid(np.arange(PS), np.arange(D), indexing="ij")
    index = {"k": ((t // 16) * (D // 32) + d // 32) * 512 + (16 * ((d % 32) // 8) + t % 16) * 8 + d % 8,
             "v": ((t // 32) * (D // 16) + d // 16) * 512 + (16 * ((t % 16) // 4) + d % 16) * 8 + 4 * ((t % 32) // 16) + t % 4}
    got = {"q": q}
    live = np.flatnonzero(m["place"] >= 0)
    page, tok = m["place"][live] // PS, m["place"][live] % PS
    for name in ("k", "v"):
        pool = s[name].double().cpu().numpy()
        for h in range(H):
            pool[0, page[:, None], h, index[name][tok]] = new[name][live, h]
        got[name] = pool
    return got


def exact_attn(c, s):
    S, Hkv, G, D, PS = (c[k] for k in ("S", "Hkv", "G", "D", "page"))
    n, lens, table = counts_of(c), lens_of(c), s["table"].cpu().numpy()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    tok, val = np.meshgrid(np.arange(PS), np.arange(D), indexing="ij")
    ki = torch.from_numpy(((tok // 16) * (D // 32) + val // 32) * 512 + (16 * ((val % 32) // 8) + tok % 16) * 8 + val % 8).to(DEV)
    vi = torch.from_numpy(((tok // 32) * (D // 16) + val // 16) * 512 + (16 * ((tok % 16) // 4) + val % 16) * 8
                          + 4 * ((tok % 32) // 16) + tok % 4).to(DEV)
    at = 0
    for b in range(S):
        m, L = int(n[b]), int(lens[b] + n[b])
        ids = torch.from_numpy(table[b, :ceil_div(L, PS)].astype(np.int64)).to(DEV)
        allow = torch.ones((m, L), dtype=torch.bool, device=DEV).tril(int(lens[b]))
        for h in range(Hkv):
            kk = s["k"][0, ids, h][:, ki].double().view(-1, D)[:L]
            vv = s["v"][0, ids, h][:, vi].double().view(-1, D)[:L]
            for a in range(h * G, h * G + G):
                sc = (s["q"][at:at + m, a].double() * s["scale"]) @ kk.t().contiguous()
                out[at:at + m, a] = torch.softmax(sc.masked_fill_(~allow, -math.inf), -1) @ vv
        at += m
    return out


def exact_linear(c, s):
    M, N, K, group = (c[k] for k in ("M", "N", "K", "group"))
    m, k = torch.arange(M, device=DEV)[:, None], torch.arange(K, device=DEV)[None, :]
    buf = torch.where(m < M // 32 * 32, 32, M % 32)
    x = s["xq"].view(-1)[m // 32 * 32 * K + (k // 32 * buf + m % 32) * 32 + k % 32].double() * s["x_scale"].double()[:, None]
    n = torch.arange(N, device=DEV)[:, None]
    if c["fmt"] == "w8":
        at = (n // 16 * ceil_div(K, 64) + k // 64) * 1024 + (16 * (k % 64 // 16) + n % 16) * 16 + k % 16
        w = s["wq"][at].double() * s["w_scale"].double()[:, None]
    else:
        b = k % 64  # the 16 k of a piece's half: words of 8 k, low nibbles the first four
        at = (n // 16 * ceil_div(K, 128) + k // 128) * 1024 + (16 * (b // 16) + n % 16) * 16 + k % 128 // 64 * 8 + b % 16 // 8 * 4 + k % 4
        code = (s["wq"][at] >> (k % 8 // 4 * 4).to(torch.uint8)) & 15
        g = k // group
        at = (n // 16 * ceil_div(K, 512) + k // 512) * (8192 // group) + n % 16 * (512 // group) + g % (512 // group)
        z = s["w_zero"][at] if c["fmt"] == "w4_z16" else (s["w_zero"][at // 2] >> (at % 2 * 4).to(torch.uint8)) & 15
        w = (code.double() - z.double()) * s["w_scale"][at].double()
    return x @ w.t().contiguous()


def exact_quant(c, s):
    M, K, B = c["M"], c["K"], c["block"]
    f = np.float32
    x = s["x"].double().cpu().numpy()
    if s["gate"] is not None:
        a = s["gate"].double().cpu().numpy()
        x = x * a / (1 + np.exp(-a))
    u = x.astype(f) * s["signs"].cpu().numpy().astype(f)
    step = 1
    while step < B:
        u = u.reshape(M, -1, 2, step)
        u = np.concatenate([u[:, :, :1] + u[:, :, 1:], u[:, :, :1] - u[:, :, 1:]], 2)
        step *= 2
    u = u.reshape(M, K)
    amax = np.abs(u).max(1)
    sigma = amax / f(127)
    with np.errstate(invalid="ignore", divide="ignore"):
        code = np.where(amax[:, None] > 0, np.clip(np.rint(u / sigma[:, None]), -127, 127), 0)
    scale = sigma.astype(np.float64) / B
    values = code * scale[:, None]
    full = M // 32 * 32
    return {"values": [np.ascontiguousarray(values[:full].reshape(full // 32, 32, K // 32, 32).transpose(0, 2, 1, 3)),
                       np.ascontiguousarray(values[full:].reshape(M - full, K // 32, 32).transpose(1, 0, 2))], "scale": scale}
