"""What is timed of the steps around a verify pass's linears: the norm in front of every quantization, attention of a
draft tree over a paged cache, and the calls that keep the cache's pages.

``own`` False computes each step in its plain form (torch, 32 bits, 64 where a rounding decides a code); True makes the
library's calls.  Page layout (one layer, one page, one head, PS tokens of D values, 16-bit):
  K  [PS/16][D/32][4][16][8]:  token 16 a + c, value 32 b + 8 g + e  at [a][b][g][c][e]
  V  [PS/32][D/16][4][16][2][4]:  token 32 a + 16 h + 4 g + j, value 16 b + c  at [a][b][g][c][h][j]
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoded token: the norm in front of a projection of the 32-layer stack (hidden size 4096)
        dict(name="norm_decode", op="norm", M=1, K=4096, block=32, x="fp32", w="fp32", y=False),
        # a 16-row verify batch, the wave-wide transform block, the normalised rows kept for a second reader
        dict(name="norm_verify", op="norm", M=16, K=4096, block=64, x="fp32", w="bf16", y=True),
        # a prompt: 16-bit embedding rows, a last slab of 3 rows
        dict(name="norm_prompt", op="norm", M=4099, K=4096, block=32, x="fp16", w="bf16", y=False),
        # plain decoding of one sequence, a short context
        dict(name="attn_decode", op="attn", S=1, T=1, Hkv=8, G=4, D=128, page=64, prefix=0, ctx=1000, type="fp16",
             ragged=False),
        # the 16-node verify pass of the stack's own heads (32 of 128, no sharing between heads)
        dict(name="attn_verify", op="attn", S=1, T=16, Hkv=32, G=1, D=128, page=64, prefix=0, ctx=8190, type="fp16",
             ragged=False),
        # the largest tree over a long context, heads shared by four
        dict(name="attn_long", op="attn", S=1, T=32, Hkv=8, G=4, D=128, page=128, prefix=0, ctx=131001, type="bf16",
             ragged=False),
        # 32 branches of one long prompt, a token each
        dict(name="attn_branches", op="attn", S=32, T=1, Hkv=8, G=4, D=128, page=64, prefix=32768, ctx=2000, type="fp16",
             ragged=False),
        # a few trees on one prompt, wide heads, trees of unequal size (one slot of them idle)
        dict(name="attn_trees", op="attn", S=6, T=7, Hkv=2, G=8, D=256, page=32, prefix=4992, ctx=301, type="bf16",
             ragged=True),
        # one layer's rows of a verify batch written into the pages
        dict(name="append_verify", op="append", S=4, T=8, Hkv=32, D=128, page=64, ctx=700, type="fp16"),
        # the accepted path of a tree in every layer of the stack
        dict(name="commit_stack", op="commit", S=8, T=16, L=32, Hkv=8, D=128, page=32, ctx=200, type="bf16"),
        # 16 branches start over from four of them: shared pages, then a private last page each, in every layer
        dict(name="branch_stack", op="branch", S=16, L=32, Hkv=8, D=128, page=64, ctx=450, need=16, parents=4, type="fp16"),
        # a block of pages moved in every layer
        dict(name="copy_pages", op="copy", n=97, L=32, Hkv=8, D=128, page=32, type="fp16"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm", "attn", "attn", "attn", "append", "commit", "branch", "copy"])
    kind = rng.choice(["fp16", "bf16"])
    if op == "norm":
        block = rng.choice([32, 64])
        return dict(op="norm", M=log(1, 4099), K=block * log(512 // block, 4096 // block), block=block,
                    x=rng.choice(["fp32", "fp16", "bf16"]), w=rng.choice(["fp32", "fp16", "bf16"]), y=rng.random() < 0.3)
    D = rng.choice([64, 128, 256])
    page = rng.choice([32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 32])
    if op == "attn":
        S = rng.choice([1, 1, log(2, 32)])
        T = rng.choice([1, log(2, 32)])
        G = rng.choice([1, 2, 4, 8])
        prefix = page * log(1, 32768 // page) if S > 1 else 0
        ctx = log(1, 131001 if S == 1 else 2000)
        # no more values read, and no more products, than the largest listed case has
        tokens = (1 << 27) // (Hkv * D)
        pairs = 4096 * 131001 // (S * T * Hkv * G * D // 32)
        prefix = min(prefix, min(tokens // 2, pairs // 2) // page * page)
        ctx = max(1, min(ctx, tokens // (2 * S), pairs // 2))
        return dict(op="attn", S=S, T=T, Hkv=Hkv, G=G, D=D, page=page, prefix=prefix, ctx=ctx, type=kind,
                    ragged=T > 1 and S > 1 and rng.random() < 0.5)
    if op == "append":
        S = log(1, 16)
        return dict(op="append", S=S, T=log(1, 64 // S), Hkv=Hkv, D=D, page=page, ctx=log(1, 3000), type=kind)
    Hkv, L = min(Hkv, 8), log(1, 32)
    if op == "commit":
        return dict(op="commit", S=log(1, 8), T=log(2, 32), L=L, Hkv=Hkv, D=D, page=page, ctx=log(1, 300), type=kind)
    if op == "branch":
        S = log(2, 16)
        return dict(op="branch", S=S, L=L, Hkv=Hkv, D=D, page=page, ctx=log(page, 450), need=log(1, 64),
                    parents=rng.randint(1, S - 1), type=kind)
    return dict(op="copy", n=log(1, 97), L=L, Hkv=Hkv, D=D, page=page, type=kind)


def own_lens(case):
    """Committed tokens of each slot: the shared prefix and some of its own (all of ctx for slot 0)."""
    S, ctx = case["S"], case["ctx"]
    return [case.get("prefix", 0) + max(1, ctx - (5 * s % S) * ctx // S) for s in range(S)]


def nodes_of(case):
    """Nodes of each slot's tree: unequal ones, and idle slots, where the case is ragged."""
    S, T = case["S"], case["T"]
    return [T - (3 * s) % (T + 1) if case["ragged"] else T for s in range(S)]


def ceil_div(a, b):
    return -(-a // b)


# ------------------------------------------------------------ inputs, per case
def generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def tree_parents(g, S, T):
    """Random draft trees: parent[0] = -1, parent[i] < i, mostly the node before."""
    i = torch.arange(T, device=DEV)
    other = (torch.rand((S, T), device=DEV, generator=g) * i).long().clamp(max=(i - 1).clamp(min=0))
    chain = torch.rand((S, T), device=DEV, generator=g) < 0.6
    parent = torch.where(chain, i - 1, other)
    parent[:, 0] = -1
    return parent.int()


def pools(g, case, n_pages, L):
    shape = (L, n_pages, case["Hkv"], case["page"] * case["D"])
    t = TYPES[case["type"]]
    return (torch.randn(shape, device=DEV, dtype=t, generator=g), torch.randn(shape, device=DEV, dtype=t, generator=g))


def slot_tables(g, case, room, spare, shared=0):
    """Pages of each slot (the shared ones first, the same in all), in shuffled order over the pool."""
    S, PS = case["S"], case["page"]
    lens = own_lens(case)
    held = [ceil_div(n + room, PS) for n in lens]
    common = shared // PS
    n_pages = common + sum(h - common for h in held) + spare
    ids = torch.randperm(n_pages, device=DEV, generator=g)
    width = max(held) + 2
    table = torch.full((S, width), -1, dtype=torch.int64, device=DEV)
    at = common
    for s, h in enumerate(held):
        table[s, :common] = ids[:common]
        table[s, common:h] = ids[at:at + h - common]
        at += h - common
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    refs[ids[:at]] = 1
    refs[ids[:common]] = S
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(table=table.int(), pages=i32(held), len=i32(lens), refs=refs), n_pages


def prepare(case, seed):
    g = generator(seed)
    op = case["op"]
    s = {"case": dict(case), "op": op}
    if op == "norm":
        M, K = case["M"], case["K"]
        # residual stream rows: a few channels far above the rest, as in the stack's activations
        x = torch.randn((M, K), device=DEV, generator=g)
        res = torch.randn((M, K), device=DEV, generator=g) * 3
        big = torch.randperm(K, device=DEV, generator=g)[:4]
        res[:, big] *= 50
        s["x"] = x.to(TYPES[case["x"]])
        s["residual"] = res
        s["weight"] = (1 + 0.2 * torch.randn(K, device=DEV, generator=g)).to(TYPES[case["w"]])
        s["signs"] = (torch.randint(0, 2, (K,), device=DEV, generator=g) * 2 - 1).to(torch.int8)
        s["xq"] = torch.zeros((M, K), dtype=torch.int8, device=DEV)
        s["x_scale"] = torch.zeros(M, device=DEV)
        s["y"] = torch.zeros((M, K), device=DEV) if case["y"] else None
        return s
    if op == "attn":
        S, T, Hkv, G, D = (case[k] for k in ("S", "T", "Hkv", "G", "D"))
        state, n_pages = slot_tables(g, case, T, 5, case["prefix"])
        s.update(state)
        s["k"], s["v"] = pools(g, case, n_pages, 1)
        rows = torch.randn((S * T, (Hkv * G + 2 * Hkv) * D), device=DEV, generator=g)  # a fused q, k, v projection's output
        s["q"] = rows[:, :Hkv * G * D].view(S * T, Hkv * G, D)
        s["q"] *= torch.linspace(0.5, 3.0, Hkv * G, device=DEV)[None, :, None]  # flat heads and peaked ones
        s["parent"] = tree_parents(g, S, T)
        s["n_nodes"] = torch.tensor(nodes_of(case), dtype=torch.int32, device=DEV) if case["ragged"] else None
        s["shared"] = torch.tensor([case["prefix"]], dtype=torch.int32, device=DEV) if case["prefix"] else None
        s["scale"] = 1.0 / math.sqrt(D)
        s["out"] = torch.zeros((S * T, Hkv * G, D), device=DEV)
        return s
    if op == "append":
        S, T, Hkv, D = (case[k] for k in ("S", "T", "Hkv", "D"))
        state, n_pages = slot_tables(g, case, T, 3)
        s.update(state)
        s["k"], s["v"] = pools(g, case, n_pages, 1)
        rows = torch.randn((S * T, 3 * Hkv * D), device=DEV, generator=g)
        s["k_rows"] = rows[:, Hkv * D:2 * Hkv * D].view(S * T, Hkv, D)
        s["v_rows"] = rows[:, 2 * Hkv * D:].view(S * T, Hkv, D)
        return s
    if op == "commit":
        S, T = case["S"], case["T"]
        state, n_pages = slot_tables(g, case, T, 3)
        s.update(state)
        s["k"], s["v"] = pools(g, case, n_pages, case["L"])
        n = commit_counts(case)
        # accepted nodes: rising node numbers, then -1
        order = torch.rand((S, T - 1), device=DEV, generator=g).argsort(1)
        count = torch.tensor(n, device=DEV)[:, None] - 1
        j = torch.arange(T - 1, device=DEV)[None, :]
        kept = torch.where(order < count, j + 1, T + 1).sort(1).values
        path = torch.full((S, T), -1, dtype=torch.int64, device=DEV)
        path[:, :T - 1] = torch.where(j < count, kept, -1)
        s["path"] = path.int()
        s["n_emit"] = torch.tensor(n, dtype=torch.int32, device=DEV)
        s["len_out"] = torch.zeros(S, dtype=torch.int32, device=DEV)
        return s
    if op == "branch":
        S = case["S"]
        state, n_pages = slot_tables(g, case, 0, S * (ceil_div(case["need"], case["page"]) + 2))
        s.update(state)
        s["k"], s["v"] = pools(g, case, n_pages, case["L"])
        src = torch.arange(S, device=DEV)
        src[case["parents"]:] = (torch.rand(S - case["parents"], device=DEV, generator=g) * case["parents"]).long()
        s["src"] = src.int()
        s["need"] = torch.full((S,), case["need"], dtype=torch.int32, device=DEV)
        s["status"] = torch.zeros(S, dtype=torch.int32, device=DEV)
        s["other"] = dict(table=torch.full_like(s["table"], -1), pages=torch.zeros_like(s["pages"]),
                          len=torch.zeros_like(s["len"]))
        return s
    n = case["n"]
    n_pages = 2 * n + 3
    s["k"], s["v"] = pools(g, case, n_pages, case["L"])
    ids = torch.randperm(n_pages, device=DEV, generator=g).int()
    s["src"], s["dst"] = ids[:n].contiguous(), ids[n:2 * n].contiguous()
    return s


def commit_counts(case):
    """Emitted tokens of each slot: from one (nothing drafted was right) to all of its tree."""
    S, T = case["S"], case["T"]
    return [1 + ((s + 1) * (T - 1) // S) for s in range(S)]


# ------------------------------------------------------------------ one pass
def run(state):
    return PASSES[state["op"]](state)


def library():
    import speculative_verify_gemm_amd as svg
    return svg


def cache_of(s):
    """The library's handle of the state's cache, made once as a program keeps it."""
    if "cache" not in s:
        s["cache"] = library().KVCache(s["k"], s["v"], s.get("table"), s.get("pages"), s.get("len"), s.get("refs"),
                                       dim=s["case"]["D"], page=s["case"]["page"])
    return s["cache"]


def slabs(xq, scale, M, K):
    """The values that codes in 32-row slab buffers stand for (scale: the row scales): the whole buffers, and the rest."""
    full = M // 32 * 32
    got = []
    if full:
        got.append(xq.view(-1)[:full * K].view(full // 32, K // 32, 32, 32) * scale[:full].view(full // 32, 1, 32, 1))
    if M > full:
        got.append(xq.view(-1)[full * K:].view(K // 32, M - full, 32) * scale[full:].view(1, M - full, 1))
    return got


def run_norm(s):
    c = s["case"]
    M, K, B = c["M"], c["K"], c["block"]
    if own:
        library().add_rmsnorm_quant_i8(s["x"], s["residual"], s["weight"], EPS, s["signs"], s["xq"], s["x_scale"], y=s["y"],
                                       block=B)
        xq, scale, y, h = s["xq"], s["x_scale"], s["y"], s["residual"]
    else:
        # the codes are defined by these fp32 steps, rounded one by one; sums and quotients that decide them in 64 bits
        h = s["x"].float() + s["residual"]
        s["residual"].copy_(h)
        r = (1.0 / torch.sqrt(h.double().square().mean(1, keepdim=True) + EPS)).float()
        y = (h * r) * s["weight"].float()
        u = hadamard(y * s["signs"].float(), B)
        amax = u.abs().amax(1, keepdim=True)
        sigma = (amax.double() / 127).float()
        code = torch.where(amax > 0, torch.round((u.double() / sigma.double()).float()).clamp(-127, 127), 0.0)
        scale = (sigma * (1.0 / B)).view(M)
        xq = to_slabs(code.to(torch.int8), M, K)
    return {"values": slabs(xq, scale, M, K), "scale": scale, "residual": h, "y": y if c["y"] else None}


def hadamard(u, B):
    """Sylvester's +/-1 transform of each run of B values, stage by stage (h = 1, 2, 4, ...)."""
    M, K = u.shape
    h = 1
    while h < B:
        v = u.view(M, K // (2 * h), 2, h)
        u = torch.stack((v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]), 2).view(M, K)
        h *= 2
    return u


def to_slabs(code, M, K):
    full = M // 32 * 32
    a = code[:full].view(full // 32, 32, K // 32, 32).permute(0, 2, 1, 3).reshape(-1)
    b = code[full:].view(M - full, K // 32, 32).permute(1, 0, 2).reshape(-1)
    return torch.cat((a, b))


def k_view(k, c):
    L, P, H, _ = k.shape
    return k.view(L, P, H, c["page"] // 16, c["D"] // 32, 4, 16, 8)


def v_view(v, c):
    L, P, H, _ = v.shape
    return v.view(L, P, H, c["page"] // 32, c["D"] // 16, 4, 16, 2, 4)


def k_rows(k, pages, c):
    """fp32 rows [..., tokens, H, D] of the pages [..., n] of layer 0."""
    t = k_view(k, c)[0][pages].float()                       # [..., n, H, PS/16, D/32, 4, 16, 8]
    lead = t.dim() - 7
    t = t.permute(*range(lead), *(lead + i for i in (0, 2, 5, 1, 3, 4, 6)))
    return t.reshape(*pages.shape[:-1], pages.shape[-1] * c["page"], k.shape[2], c["D"])


def v_rows(v, pages, c):
    t = v_view(v, c)[0][pages].float()                       # [..., n, H, PS/32, D/16, 4, 16, 2, 4]
    lead = t.dim() - 8
    t = t.permute(*range(lead), *(lead + i for i in (0, 2, 6, 4, 7, 1, 3, 5)))
    return t.reshape(*pages.shape[:-1], pages.shape[-1] * c["page"], v.shape[2], c["D"])


def run_attn(s):
    c = s["case"]
    if own:
        cache = cache_of(s)
        if "workspace" not in s:
            s["workspace"] = library().tree_attention_workspace(cache, c["Hkv"] * c["G"], c["T"])
        library().tree_attention(cache, 0, s["q"], s["parent"], s["out"], s["workspace"], scale=s["scale"],
                                 n_nodes=s["n_nodes"], shared=s["shared"])
        return s["out"]
    S, T, Hkv, G, D, PS, P0 = (c[k] for k in ("S", "T", "Hkv", "G", "D", "page", "prefix"))
    q = s["q"].view(S, T, Hkv, G, D).permute(0, 2, 1, 3, 4) * s["scale"]          # [S, Hkv, T, G, D]
    # the prefix once, for the rows of all slots
    pre = s["table"][0, :P0 // PS].long()
    kp, vp = k_rows(s["k"], pre, c), v_rows(s["v"], pre, c)                         # [P0, Hkv, D]
    qp = q.permute(1, 0, 2, 3, 4).reshape(Hkv, S * T * G, D)
    sp = torch.matmul(qp, kp.permute(1, 2, 0).contiguous())                         # [Hkv, S*T*G, P0]
    # each slot's own tokens and its tree
    most = max(own_lens(c)) - P0 + T
    rest = s["table"][:, P0 // PS:P0 // PS + ceil_div(most, PS)].clamp(min=0).long()
    ks, vs = k_rows(s["k"], rest, c), v_rows(s["v"], rest, c)                       # [S, Ls, Hkv, D]
    Ls = ks.shape[1]
    ss = torch.matmul(q.reshape(S, Hkv, T * G, D), ks.permute(0, 2, 3, 1).contiguous()).view(S, Hkv, T, G, Ls)
    eye = torch.eye(T, device=DEV)
    link = torch.zeros((S, T, T + 1), device=DEV).scatter_(2, (s["parent"].long() % (T + 1))[..., None], 1.0)[..., :T]
    seen = torch.matrix_power(eye + link, T) > 0                                    # [S, T, T]: node j on i's root path
    node = torch.arange(Ls, device=DEV)[None, :] - (s["len"] - P0)[:, None]        # node at each token, [S, Ls]
    inside = (node >= 0) & (node < T)
    on_path = torch.gather(seen, 2, node.clamp(0, T - 1)[:, None, :].expand(S, T, Ls))
    mask = (node < 0)[:, None, :] | (inside[:, None, :] & on_path)                  # [S, T, Ls]
    ss = torch.where(mask[:, None, :, None, :], ss, -math.inf)
    sp = sp.view(Hkv, S, T, G, P0).permute(1, 0, 2, 3, 4)
    score = torch.cat((sp, ss), -1)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    total = p.sum(-1, keepdim=True)
    pp = p[..., :P0].permute(1, 0, 2, 3, 4).reshape(Hkv, S * T * G, P0)
    o = torch.matmul(pp, vp.permute(1, 0, 2).contiguous()).view(Hkv, S, T, G, D).permute(1, 0, 2, 3, 4)
    ps = p[..., P0:].reshape(S, Hkv, T * G, Ls)
    o = o + torch.matmul(ps, vs.permute(0, 2, 1, 3).contiguous()).view(S, Hkv, T, G, D)
    o = (o / total).permute(0, 2, 1, 3, 4).reshape(S, T, Hkv * G, D)
    if s["n_nodes"] is not None:
        live = torch.arange(T, device=DEV)[None, :] < s["n_nodes"][:, None]
        o = torch.where(live[..., None, None], o, s["out"].view_as(o))
    s["out"].copy_(o.view_as(s["out"]))
    return s["out"]


def places(table, pos, PS):
    """(page, token in the page) of positions pos [S, n]."""
    return torch.gather(table, 1, (pos // PS)).long(), pos % PS


def write_rows(s, c, layers, page, t, k_new, v_new):
    """Rows [S, n, L, Hkv, D] to the places (page, t)."""
    S, n = page.shape
    L, H, D = k_new.shape[2:]
    kv, vv = k_view(s["k"], c)[layers], v_view(s["v"], c)[layers]
    kv[:, page, :, t // 16, :, :, t % 16, :] = k_new.view(S, n, L, H, D // 32, 4, 8)
    a = t % 32
    vv[:, page, :, t // 32, :, (a % 16) // 4, :, a // 16, a % 4] = v_new.view(S, n, L, H, D // 16, 16)


def read_rows(s, c, page, t):
    S, n = page.shape
    kv, vv = k_view(s["k"], c), v_view(s["v"], c)
    a = t % 32
    k = kv[:, page, :, t // 16, :, :, t % 16, :]
    v = vv[:, page, :, t // 32, :, (a % 16) // 4, :, a // 16, a % 4]
    return k.reshape(S, n, kv.shape[0], kv.shape[2], c["D"]), v.reshape(S, n, kv.shape[0], kv.shape[2], c["D"])


def run_append(s):
    c = s["case"]
    if own:
        library().kv_append(cache_of(s), 0, s["k_rows"], s["v_rows"], c["T"])
    else:
        S, T, H, D = (c[k] for k in ("S", "T", "Hkv", "D"))
        pos = s["len"].long()[:, None] + torch.arange(T, device=DEV)[None, :]
        page, t = places(s["table"], pos, c["page"])
        ty = TYPES[c["type"]]
        write_rows(s, c, slice(0, 1), page, t, s["k_rows"].reshape(S, T, 1, H, D).to(ty), s["v_rows"].reshape(S, T, 1, H, D).to(ty))
    return {"k": s["k"], "v": s["v"]}


def run_commit(s):
    c = s["case"]
    if own:
        library().kv_commit(cache_of(s), s["path"], s["n_emit"], s["len_out"])
    else:
        T = c["T"]
        j = torch.arange(1, T, device=DEV)[None, :]
        moved = j < s["n_emit"][:, None]
        base = s["len"].long()[:, None]
        src = base + torch.where(moved, s["path"][:, :T - 1].long(), 0)
        dst = base + torch.where(moved, j, 0)
        k, v = read_rows(s, c, *places(s["table"], src, c["page"]))
        write_rows(s, c, slice(None), *places(s["table"], dst, c["page"]), k, v)
        s["len_out"].copy_(s["len"] + s["n_emit"])
    return {"k": s["k"], "v": s["v"], "len": s["len_out"]}


def run_branch(s):
    """All slots start over from the sources' state, and get room for `need` more tokens of their own."""
    c = s["case"]
    now = {k: s[k] for k in ("table", "pages", "len")}
    new = s["other"]
    if own:
        svg = library()
        if "caches" not in s:
            s["caches"] = [svg.KVCache(s["k"], s["v"], t["table"], t["pages"], t["len"], s["refs"], dim=c["D"], page=c["page"])
                           for t in (now, new)]
            s["kv_workspace"] = svg.kv_workspace(s["caches"][0])
        a, b = s["caches"]
        svg.kv_fork(a, s["src"], b)
        svg.kv_reserve(b, s["need"], s["status"], s["kv_workspace"])
        s["caches"] = [b, a]
    else:
        plain_fork(s, c, now, new)
        plain_reserve(s, c, new)
    s["other"] = now
    s.update(new)
    return {"k": s["k"], "v": s["v"], "table": s["table"], "pages": s["pages"], "len": s["len"], "refs": s["refs"],
            "status": s["status"]}


def plain_fork(s, c, now, new):
    S, W = now["table"].shape
    src = s["src"].long()
    kept = src == torch.arange(S, device=DEV)
    col = torch.arange(W, device=DEV)[None, :]
    pages = torch.where(kept, now["pages"], (now["len"][src] + c["page"] - 1) // c["page"])
    old = (col < now["pages"][:, None]) & ~kept[:, None]
    add = (col < pages[:, None]) & ~kept[:, None]
    rows = now["table"][src]
    refs = s["refs"]
    refs.index_add_(0, now["table"].clamp(min=0).view(-1).long(), -old.view(-1).int())
    refs.index_add_(0, rows.clamp(min=0).view(-1).long(), add.view(-1).int())
    new["table"].copy_(torch.where(col < pages[:, None], rows, new["table"]))
    new["len"].copy_(now["len"][src])
    new["pages"].copy_(pages)


def plain_reserve(s, c, st):
    PS = c["page"]
    S, W = st["table"].shape
    table, pages, n, need, refs = st["table"], st["pages"], st["len"], s["need"], s["refs"]
    more = ((n + need + PS - 1) // PS - pages).clamp(min=0)
    at = (n // PS).long()
    part = torch.gather(table, 1, at[:, None])[:, 0].clamp(min=0).long()            # the page that holds token n - 1, if partly full
    partly = (n % PS != 0) & (need > 0)
    s_ = torch.arange(S, device=DEV)
    before = ((part[:, None] == part[None, :]) & partly[None, :] & (s_[None, :] < s_[:, None])).sum(1)
    copy = partly & (refs[part] - before > 1)
    want = more + copy
    first = want.cumsum(0) - want
    free = torch.argsort((refs != 0).int(), stable=True)                             # free pages, lowest first
    fresh = free[first.clamp(max=free.numel() - 1)]
    col = torch.arange(W, device=DEV)[None, :]
    i = col - pages[:, None]
    added = (i >= 0) & (i < more[:, None])
    new = free[(first[:, None] + copy[:, None].long() + i).clamp(0, free.numel() - 1)]
    table.copy_(torch.where(added, new.int(), table))
    taken = torch.arange(free.numel(), device=DEV) < want.sum()
    refs.index_add_(0, part, -copy.int())
    refs.index_add_(0, free, taken.int())
    table.copy_(torch.where(copy[:, None] & (col == at[:, None]), fresh[:, None].int(), table))
    a = torch.where(copy, part, table[:, 0].long())                                  # no copy: a page onto itself
    b = torch.where(copy, fresh, table[:, 0].long())
    s["k"][:, b] = s["k"][:, a]
    s["v"][:, b] = s["v"][:, a]
    pages += more
    s["status"].zero_()


def run_copy(s):
    if own:
        library().kv_copy_pages(cache_of(s), s["src"], s["dst"])
    else:
        s["k"][:, s["dst"].long()] = s["k"][:, s["src"].long()]
        s["v"][:, s["dst"].long()] = s["v"][:, s["src"].long()]
    return {"k": s["k"], "v": s["v"]}


PASSES = {"norm": run_norm, "attn": run_attn, "append": run_append, "commit": run_commit, "branch": run_branch,
          "copy": run_copy}


# ------------------------------------------------------------------ the floor
def work(case):
    """Bytes and operations that a pass cannot do without."""
    op = case["op"]
    if op == "norm":
        M, K = case["M"], case["K"]
        x, w = (4 if case[k] == "fp32" else 2 for k in ("x", "w"))
        return {"bytes": M * K * (x + 8 + 1 + (4 if case["y"] else 0)) + K * (w + 1) + 4 * M, "flops": 12.0 * M * K}
    H, D = case["Hkv"], case["D"]
    row = 4 * H * D  # K and V of one token of one layer
    if op == "attn":
        lens, nodes = own_lens(case), nodes_of(case)
        P0, G = case["prefix"], case["G"]
        tokens = P0 + sum(n - P0 + t for n, t in zip(lens, nodes) if t)
        pairs = sum(t * (n + (t + 1) / 2) for n, t in zip(lens, nodes))
        return {"bytes": tokens * row + sum(nodes) * 8 * H * G * D, "flops": 4.0 * D * H * G * pairs}
    if op == "append":
        return {"bytes": case["S"] * case["T"] * 3 * row, "flops": 0}
    if op == "commit":
        return {"bytes": sum(n - 1 for n in commit_counts(case)) * 2 * row * case["L"], "flops": 0}
    if op == "branch":
        S, PS = case["S"], case["page"]
        lens = own_lens(case)[:case["parents"]]
        # the last page of each child and of its source, all but one of them copied; tables and counts are small beside it
        copies = sum(1 for n in lens if n % PS) * (S - case["parents"]) / case["parents"]
        held = sum(ceil_div(n, PS) for n in own_lens(case))
        return {"bytes": copies * 2 * PS * row * case["L"] + 16 * held, "flops": 0}
    return {"bytes": case["n"] * 2 * case["page"] * row * case["L"], "flops": 0}


# ------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return exact_norm(case, s)
    if case["op"] == "attn":
        return exact_attn(case, s)
    return None  # values are moved or rounded once: equal to the plain form's, bit for bit


def exact_norm(case, s):
    M, K, B = case["M"], case["K"], case["block"]
    x = s["x"].float().cpu().numpy()
    res, w = s["residual"].cpu().numpy(), s["weight"].float().cpu().numpy()
    f = np.float32
    # the codes and scales are defined through fp32 values, each step rounded once
    h32 = x + res
    r64 = 1.0 / np.sqrt((h32.astype(np.float64) ** 2).sum(1) / K + EPS)
    u = (h32 * r64.astype(f)[:, None]) * w * s["signs"].cpu().numpy().astype(f)
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
    parts = []
    if full:
        parts.append(values[:full].reshape(full // 32, 32, K // 32, 32).transpose(0, 2, 1, 3))
    if M > full:
        parts.append(values[full:].reshape(M - full, K // 32, 32).transpose(1, 0, 2))
    h = x.astype(np.float64) + res.astype(np.float64)
    y = h / np.sqrt((h ** 2).mean(1, keepdims=True) + EPS) * w.astype(np.float64)
    return {"values": [np.ascontiguousarray(p) for p in parts], "scale": scale, "residual": h, "y": y if case["y"] else None}


def exact_attn(case, s):
    S, T, Hkv, G, D, PS = (case[k] for k in ("S", "T", "Hkv", "G", "D", "page"))
    table, lens = s["table"].cpu().numpy(), s["len"].cpu().numpy()
    parent, nodes = s["parent"].cpu().numpy(), nodes_of(case)
    q = s["q"].view(S, T, Hkv, G, D)
    out = torch.zeros((S, T, Hkv, G, D), dtype=torch.float64, device=DEV)
    a = np.arange(PS)
    for b in range(S):
        n, t = int(lens[b]), nodes[b]
        if t == 0:
            continue
        ids = torch.from_numpy(table[b, :ceil_div(n + t, PS)].astype(np.int64)).to(DEV)
        allow = torch.ones((t, n + t), dtype=torch.bool, device=DEV)
        tree = np.zeros((t, t), dtype=bool)
        for i in range(t):
            j = i
            while j >= 0:
                tree[i, j] = True
                j = int(parent[b, j])
        allow[:, n:] = torch.from_numpy(tree).to(DEV)
        for hd in range(Hkv):
            # element (token, value) of a page, from the layout's formula
            tok, val = np.meshgrid(a, np.arange(D), indexing="ij")
            ki = ((tok // 16) * (D // 32) + val // 32) * 512 + (16 * ((val % 32) // 8) + tok % 16) * 8 + val % 8
            vi = (((tok // 32) * (D // 16) + val // 16) * 512 + (16 * ((tok % 16) // 4) + val % 16) * 8
                  + 4 * ((tok % 32) // 16) + tok % 4)
            kk = s["k"][0, ids, hd][:, torch.from_numpy(ki).to(DEV)].double().view(-1, D)[:n + t]
            vv = s["v"][0, ids, hd][:, torch.from_numpy(vi).to(DEV)].double().view(-1, D)[:n + t]
            sc = (q[b, :t, hd].double().reshape(t * G, D) * s["scale"]) @ kk.t().contiguous()
            sc = sc.view(t, G, n + t).masked_fill(~allow[:, None, :], -math.inf)
            p = torch.softmax(sc, -1)
            out[b, :t, hd] = (p.view(t * G, n + t) @ vv).view(t, G, D)
    return out.view(S * T, Hkv * G, D)
