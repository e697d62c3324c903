"""The 8-bit KV cache's operators and the rotated append: cases, plain forms and exact values.

Four operators, one case dict each ("op"):
  append    rotate the new rows' q and k, write k and v to the paged bf16 cache
  append8   the same into the e4m3 cache with one power-of-two scale per (page, KV head, K or V)
  attend8   verify attention over the e4m3 cache
  commit8   keep the accepted nodes of a draft tree, compacted, in every layer of the e4m3 cache

Pages hold 16 tokens: pools [num_blocks][Hkv][16][D], scales fp32 [num_blocks][Hkv][2] (K, V).
"""
import math

import torch

own = False

PAGE = 16
TREE = [-1, 0, 0, 0, 1, 1, 2, 4, 4, 7, 5]   # the tree-verify workload's draft tree


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one rollout left of a batch, four drafts: latency of one layer's attention
        dict(name="attend8_b1", op="attend8", B=1, N=5, Hq=40, Hkv=8, D=128, lo=6151, hi=6151, tree=False),
        # the long tail: eight rollouts of 4k to 16k tokens
        dict(name="attend8_b8_tail", op="attend8", B=8, N=5, Hq=28, Hkv=4, D=128, lo=4096, hi=16384, tree=False),
        # a batch in full flight with eight drafts, contexts spread over two orders of magnitude
        dict(name="attend8_b64_g8", op="attend8", B=64, N=9, Hq=40, Hkv=8, D=128, lo=512, hi=32768, tree=False),
        # draft trees of ten nodes over 24k tokens
        dict(name="attend8_b16_tree", op="attend8", B=16, N=11, Hq=32, Hkv=4, D=128, lo=24576, hi=24576, tree=True),
        # plain decode steps (one row per sequence) with 64-wide heads
        dict(name="attend8_b32_d64", op="attend8", B=32, N=1, Hq=32, Hkv=8, D=64, lo=1000, hi=8200, tree=False),
        # the step's new rows of one rollout: latency
        dict(name="append_b1", op="append", B=1, N=5, Hq=28, Hkv=4, D=128, rotary=128, half=True, lo=6151, hi=6151,
             fused=False, ragged=False, tree=False),
        # a full batch's new rows, cut out of a fused projection's output
        dict(name="append_b256_g8", op="append", B=256, N=9, Hq=40, Hkv=8, D=128, rotary=128, half=True, lo=512,
             hi=32768, fused=True, ragged=False, tree=False),
        # the same calls into the 8-bit cache
        dict(name="append8_b1", op="append8", B=1, N=5, Hq=28, Hkv=4, D=128, rotary=128, half=True, lo=6151, hi=6151,
             fused=False, ragged=False, tree=False),
        dict(name="append8_b64_tree", op="append8", B=64, N=11, Hq=32, Hkv=4, D=128, rotary=128, half=True, lo=512,
             hi=24576, fused=True, ragged=False, tree=True),
        # prompts of a rollout batch, ragged, rotation of half the head in the interleaved layout
        dict(name="append8_prompts", op="append8", B=16, N=1500, Hq=32, Hkv=8, D=128, rotary=64, half=False, lo=1500,
             hi=1500, fused=True, ragged=True, tree=False),
        # accepted paths of draft trees, all layers in one call
        dict(name="commit8_b1_l28", op="commit8", B=1, N=11, Hkv=4, D=128, L=28, lo=6151, hi=6151),
        dict(name="commit8_b64_l48", op="commit8", B=64, N=11, Hkv=4, D=128, L=48, lo=512, hi=24576),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend8", "attend8", "append", "append8", "commit8"])
    Hq, Hkv, D = rng.choice([(40, 8, 128), (28, 4, 128), (32, 4, 128), (32, 8, 128), (4, 1, 64), (32, 8, 64),
                             (8, 8, 128), (16, 1, 128)])
    B = _log(rng, 1, 64)
    if op == "attend8":
        tree = rng.random() < 0.25
        N = len(TREE) if tree else _log(rng, 1, 16)
        # no more keys than the largest listed case reads
        most = min(32768, (64 * 7700 * 8 * 128) // (B * Hkv * D))
        hi = _log(rng, N, max(N, most))
        lo = _log(rng, N, hi)
        return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, lo=lo, hi=hi, tree=tree)
    if op == "commit8":
        hi = _log(rng, len(TREE), 32768)
        return dict(op=op, B=B, N=len(TREE), Hkv=Hkv, D=D, L=_log(rng, 1, 48), lo=_log(rng, len(TREE), hi), hi=hi)
    ragged = rng.random() < 0.4
    tree = not ragged and rng.random() < 0.3
    N = len(TREE) if tree else (_log(rng, 1, max(1, 24000 // B)) if ragged else _log(rng, 1, 64))
    hi = max(N, _log(rng, 1, 32768))
    return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, rotary=rng.choice([D, D, D // 2, D // 4]),
                half=rng.random() < 0.6, lo=max(N, _log(rng, 1, hi)), hi=hi, fused=rng.random() < 0.5, ragged=ragged,
                tree=tree)


def _lens(case):
    """Context lengths of the case, new rows included: spread from lo to hi over their logarithm."""
    lo, hi = case["lo"], case["hi"]
    return [max(case["N"], int(lo * (hi / lo) ** ((0.618034 * (b + 1)) % 1.0))) for b in range(case["B"])]


def _new_lens(case):
    """Rows each sequence appends: all N, or (ragged) from none to N."""
    N, B = case["N"], case["B"]
    if not case.get("ragged"):
        return [N] * B
    return [N if b == 0 else int(round(N * ((0.754878 * b) % 1.0))) for b in range(B)]


def work(case):
    op, B, N, Hkv, D = case["op"], case["B"], case["N"], case["Hkv"], case["D"]
    lens = _lens(case)
    pages = sum(-(-c // PAGE) for c in lens)
    if op == "attend8":
        Hq = case["Hq"]
        return {"bytes": sum(lens) * 2 * Hkv * D + 8 * Hkv * pages + 4 * pages + 4 * B * N * Hq * D + 4 * B
                + (8 * B * N if case["tree"] else 0),
                "flops": 4.0 * N * Hq * D * sum(lens)}
    if op == "commit8":
        alen, path = _paths(case)
        moved = sum(sum(1 for k in range(a) if p[k] != k + 1) for a, p in zip(alen, path))
        return {"bytes": moved * 2 * 2 * Hkv * D * case["L"] + B * (4 * (N - 1) + 16), "flops": 0}
    Hq = case["Hq"]
    nl = _new_lens(case)
    rows, kept, touched = sum(nl), 0, 0
    for c, n in zip(lens, nl):
        if n:
            kept += (c - n) % PAGE
            touched += (c - 1) // PAGE - (c - n) // PAGE + 1
    got = rows * (4 * Hq * D + 4 * Hkv * D + 4 * case["rotary"]) + 4 * touched + 4 * B
    if op == "append":
        got += rows * 4 * Hkv * D
    else:  # 8-bit rows out, the rows already in a partly filled page read, both scales of a page written
        got += rows * 2 * Hkv * D + kept * 2 * Hkv * D + 8 * Hkv * touched
    return {"bytes": got, "flops": rows * 3.0 * case["rotary"] * (Hq + Hkv)}


def _paths(case):
    """Accepted paths down the tree, of every depth, most of them off the first branch."""
    kids = [[c for c in range(1, len(TREE)) if TREE[c] == v] for v in range(len(TREE))]
    alen, path = [], []
    for b in range(case["B"]):
        v, p = 0, []
        while kids[v] and len(p) < 1 + (b + 2) % 4:
            v = kids[v][(b + len(p)) % len(kids[v])]
            p.append(v)
        alen.append(len(p))
        path.append(p + [-1] * (case["N"] - 1 - len(p)))
    return alen, path


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pools8(shape, g):
    """An e4m3 pool as appended rows leave it: pages whose largest entries come near the format's end, under
    power-of-two scales that differ from page to page."""
    pool = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(64).clamp_(-448, 448)
    return pool.to(torch.float8_e4m3fn)


def _scales8(shape, g):
    return torch.exp2(torch.randint(-7, -4, shape, generator=g, device="cuda").float())


def _tail_table(case, lens, nl, g):
    """A block table whose pages that hold new rows (or are kept beside them) are each sequence's own."""
    T = (case["N"] + PAGE - 1) // PAGE + 1
    nb = case["B"] * T + 3
    perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((case["B"], max(-(-c // PAGE) for c in lens)), dtype=torch.int32, device="cuda")
    for b, (c, n) in enumerate(zip(lens, nl)):
        first, last = (c - n) // PAGE, -(-c // PAGE)
        table[b, first:last] = perm[b * T:b * T + last - first]
    return table, nb


def prepare(case, seed):
    g = _gen(seed)
    op, B, N, Hkv, D = case["op"], case["B"], case["N"], case["Hkv"], case["D"]
    lens = _lens(case)
    s = {"case": case, "ctx": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if op == "attend8":
        counts = [-(-c // PAGE) for c in lens]
        nb = sum(counts) + 1
        perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, max(counts)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(counts):
            table[b, :n] = perm[at:at + n]
            at += n
        s["table"] = table.clamp_(min=0)
        s["k"], s["v"] = _pools8((nb, Hkv, PAGE, D), g), _pools8((nb, Hkv, PAGE, D), g)
        s["scales"] = _scales8((nb, Hkv, 2), g)
        s["q"] = torch.randn((B, N, case["Hq"], D), generator=g, device="cuda").to(torch.bfloat16)
        s["mask"] = None
        if case["tree"]:
            bits = []
            for i in range(N):
                m, j = 0, i
                while j >= 0:
                    m |= 1 << j
                    j = TREE[j]
                bits.append(m)
            s["mask"] = torch.tensor([bits] * B, dtype=torch.int64, device="cuda")
        if own:
            import speculative_decoding_rl_b200 as sv
            from speculative_decoding_rl_b200.session import AttentionQ8Call
            desc = sv.SvAttnDesc(B, N, case["Hq"], Hkv, D, PAGE, s["table"].shape[1], nb)
            s["call"] = AttentionQ8Call(desc, (s["k"], s["v"], s["scales"]), s["table"], s["ctx"], s["q"], s["mask"])
        return s
    if op == "commit8":
        L = case["L"]
        s["table"], nb = _tail_table(case, lens, [N] * B, g)
        s["k"], s["v"] = _pools8((L, nb, Hkv, PAGE, D), g), _pools8((L, nb, Hkv, PAGE, D), g)
        s["scales"] = _scales8((L, nb, Hkv, 2), g)
        alen, path = _paths(case)
        s["alen"], s["path"] = i32(alen), i32(path)
        if own:
            import speculative_decoding_rl_b200 as sv
            from speculative_decoding_rl_b200.session import CommitQ8Call
            desc = sv.SvAttnDesc(B, N, Hkv, Hkv, D, PAGE, s["table"].shape[1], nb)
            layers = [(s["k"][i], s["v"][i], s["scales"][i]) for i in range(L)]
            s["call"] = CommitQ8Call(desc, layers, s["table"], s["ctx"], s["alen"], s["path"])
        return s
    Hq, R = case["Hq"], case["rotary"]
    nl = _new_lens(case)
    s["table"], nb = _tail_table(case, lens, nl, g)
    if case["fused"]:
        qkv = torch.randn((B, N, Hq + 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        s["q"], s["kn"], s["vn"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    else:
        new = lambda h: torch.randn((B, N, h, D), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        s["q"], s["kn"], s["vn"] = new(Hq), new(Hkv), new(Hkv)
    s["new_lens"] = i32(nl) if case["ragged"] else None
    s["positions"] = None
    if case["tree"]:  # a node's position is its depth below the root's
        depth = [0] * N
        for c in range(1, N):
            depth[c] = depth[TREE[c]] + 1
        s["positions"] = s["ctx"][:, None] - N + i32(depth)[None]
    freq = 1e6 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
    angle = torch.arange(max(lens), device="cuda", dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    if op == "append":
        s["k"] = torch.randn((nb, Hkv, PAGE, D), generator=g, device="cuda").to(torch.bfloat16)
        s["v"] = torch.randn((nb, Hkv, PAGE, D), generator=g, device="cuda").to(torch.bfloat16)
    else:
        s["k"], s["v"] = _pools8((nb, Hkv, PAGE, D), g), _pools8((nb, Hkv, PAGE, D), g)
        s["scales"] = _scales8((nb, Hkv, 2), g)
    s["q_out"] = torch.zeros((B, N, Hq, D), dtype=torch.bfloat16, device="cuda")
    if own:
        import speculative_decoding_rl_b200 as sv
        from speculative_decoding_rl_b200.session import AppendCall, AppendQ8Call
        desc = sv.SvAttnDesc(B, N, Hq, Hkv, D, PAGE, s["table"].shape[1], nb)
        rope = sv.make_rope_desc(s["cos_sin"], interleaved=not case["half"])
        kv = (s["k"], s["v"]) if op == "append" else (s["k"], s["v"], s["scales"])
        s["call"] = (AppendCall if op == "append" else AppendQ8Call)(
            desc, rope, kv, s["table"], s["ctx"], s["q"], s["kn"], s["vn"], positions=s["positions"],
            new_lens=s["new_lens"], q_out=s["q_out"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if op == "attend8":
        return s["call"].run() if own else _attend8(s)
    if op == "commit8":
        ctx = s["call"].run() if own else _commit8(s)
        return {"ctx": ctx, "k": s["k"], "v": s["v"], "scales": s["scales"]}
    if own:
        s["call"].run()
    else:
        _append(s)
    out = {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if op == "append8":
        out["scales"] = s["scales"]
    return out


# ------------------------------------------------------------------ plain forms
def _attend8(s):
    case, q, table, ctx = s["case"], s["q"], s["table"].long(), s["ctx"].long()
    B, N, Hq, Hkv, D = case["B"], case["N"], case["Hq"], case["Hkv"], case["D"]
    T = table.shape[1] * PAGE

    def whole(pool, which):  # [B][Hkv][T][D] in 32 bits
        x = pool[table].float() * s["scales"][table][..., which, None, None]
        return x.transpose(1, 2).reshape(B, Hkv, T, D)

    t = torch.arange(T, device=q.device)
    new = t[None] - (ctx[:, None] - N)                       # index among the new keys, [B][T]
    row = torch.arange(N, device=q.device)
    if s["mask"] is None:
        sees = new[:, None, :] <= row[None, :, None]
    else:
        sees = (new[:, None, :] < 0) | ((s["mask"][:, :, None] >> new[:, None, :].clamp(0, 63)) & 1).bool()
    sees &= (t[None] < ctx[:, None])[:, None]                # [B][N][T]
    qh = q.float().view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    w = qh @ whole(s["k"], 0).transpose(2, 3) * D ** -0.5    # [B][Hkv][N*G][T]
    w = w.view(B, Hkv, N, -1, T).masked_fill_(~sees[:, None, :, None], -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True).clamp_(min=-3e38))
    total = w.sum(-1, keepdim=True)
    out = w.view(B, Hkv, -1, T) @ whole(s["v"], 1)
    out = out.view(B, Hkv, N, -1, D) / total.clamp_(min=1e-38)
    return out.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(torch.bfloat16)


def _rotate(x, cs, half):
    """x [B][N][H][D] in 32 bits, cs [B][N][R]: pairs of the first R entries turned by their position's angles."""
    R = cs.shape[-1]
    c, sn = cs[..., None, :R // 2], cs[..., None, R // 2:]
    y = x.clone()
    if half:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2] = a * c - b * sn
        y[..., R // 2:R] = b * c + a * sn
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2] = a * c - b * sn
        y[..., 1:R:2] = b * c + a * sn
    return y


def _append(s):
    case, ctx = s["case"], s["ctx"].long()
    N = case["N"]
    n = ctx * 0 + N if s["new_lens"] is None else s["new_lens"].long()
    i = torch.arange(N, device=ctx.device)[None]
    at = (ctx - n)[:, None] + i                              # cache position of each new row
    real = i < n[:, None]
    pos = at if s["positions"] is None else s["positions"].long()
    cs = s["cos_sin"][pos.clamp(0, s["cos_sin"].shape[0] - 1)]
    q = _rotate(s["q"].float(), cs, case["half"]).to(torch.bfloat16)
    s["q_out"].copy_(torch.where(real[..., None, None], q, s["q_out"]))
    k, v = _rotate(s["kn"].float(), cs, case["half"]), s["vn"].float()
    if case["op"] == "append":
        blk = s["table"].long().gather(1, (at // PAGE).clamp(0, s["table"].shape[1] - 1))[real]
        s["k"][blk, :, (at % PAGE)[real]] = k[real].to(torch.bfloat16)
        s["v"][blk, :, (at % PAGE)[real]] = v[real].to(torch.bfloat16)
        return
    # the pages from the first new row's on, [B][T]
    T = (N + PAGE - 1) // PAGE + 1
    page = (ctx - n)[:, None] // PAGE + torch.arange(T, device=ctx.device)[None]
    t = page[..., None] * PAGE + torch.arange(PAGE, device=ctx.device)   # [B][T][16]
    src = (t - (ctx - n)[:, None, None])
    new = (src >= 0) & (src < n[:, None, None])
    blk = s["table"].long().gather(1, page.clamp(0, s["table"].shape[1] - 1))
    some = new.any(-1)
    b = torch.arange(case["B"], device=ctx.device)[:, None, None]
    for pool, rows, which in ((s["k"], k, 0), (s["v"], v, 1)):
        old = pool[blk].float() * s["scales"][blk][..., which, None, None]     # [B][T][Hkv][16][D]
        val = torch.where(new[:, :, None, :, None], rows[b, src.clamp(0, N - 1)].transpose(2, 3), old)
        _store8(pool, s["scales"], which, blk, val, t < ctx[:, None, None], some)


def _store8(pool, scales, which, blk, val, keep, some):
    """Writes the kept rows of the pages `some` under the smallest power of two that holds them."""
    top = (val.abs() * keep[:, :, None, :, None]).amax((-1, -2))               # [B][T][Hkv]
    m, x = torch.frexp(top)
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp(-100, 119)                 # 448 = 0.875 * 2^9
    e = torch.where(top > 0, e, torch.full_like(e, -100)).float()
    new8 = (val * torch.exp2(-e)[..., None, None]).to(torch.float8_e4m3fn)
    at = (keep & some[..., None])[:, :, None, :, None]
    old8 = pool[blk]
    merged = torch.where(at, new8.view(torch.uint8), old8.view(torch.uint8))
    pool.view(torch.uint8)[blk[some]] = merged[some]
    scales[..., which][blk[some]] = torch.exp2(e)[some]


def _commit8(s):
    case, ctx, alen, path = s["case"], s["ctx"].long(), s["alen"].long(), s["path"].long()
    B, N, L = case["B"], case["N"], case["L"]
    nb = s["k"].shape[1]
    root = ctx - N
    T = (N + PAGE - 1) // PAGE + 1
    page = root[:, None] // PAGE + torch.arange(T, device=ctx.device)[None]
    t = page[..., None] * PAGE + torch.arange(PAGE, device=ctx.device)         # [B][T][16]
    j = t - root[:, None, None] - 1                                            # place on the path
    on = (j >= 0) & (j < alen[:, None, None])
    node = path.gather(1, j.clamp(0, N - 2).view(B, -1)).view_as(j)
    moved = on & (node != j + 1)
    src = torch.where(moved, root[:, None, None] + node, t) - page[:, :1, None] * PAGE
    keep = t <= (root + alen)[:, None, None]
    some = moved.any(-1)
    blk = s["table"].long().gather(1, page.clamp(0, s["table"].shape[1] - 1))
    layer = torch.arange(L, device=ctx.device)[:, None, None] * nb
    blk = (blk[None] + layer).view(L * B, T)
    keep, some, src = (x[None].expand(L, *x.shape).reshape(L * B, *x.shape[1:]) for x in (keep, some, src))
    scales = s["scales"].view(L * nb, -1, 2)
    for pool, which in ((s["k"], 0), (s["v"], 1)):
        pool = pool.view(L * nb, *pool.shape[2:])
        val = pool[blk].float() * scales[blk][..., which, None, None]          # [LB][T][Hkv][16][D]
        rows = val.transpose(2, 3).reshape(L * B, T * PAGE, *val.shape[2:3], val.shape[-1])
        rows = rows.gather(1, src.reshape(L * B, -1, 1, 1).expand(-1, -1, *rows.shape[2:]))
        val = rows.view(L * B, T, PAGE, *rows.shape[2:]).transpose(2, 3)
        _store8(pool, scales, which, blk, val, keep, some)
    return (root + 1 + alen).to(torch.int32)


# ------------------------------------------------------------------ exact values
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attend8":
        return _exact_attend8(s)
    lens = _lens(case)
    table = s["table"].cpu().tolist()
    if op == "commit8":
        k, v, sc = s["k"].double(), s["v"].double(), s["scales"].double()
        alen, path = _paths(case)
        for b, (c, a) in enumerate(zip(lens, alen)):
            root = c - case["N"]
            moves = {root + 1 + j: root + path[b][j] for j in range(a) if path[b][j] != j + 1}
            where = lambda u: (table[b][u // PAGE], u % PAGE)  # noqa: E731
            for which, pool in ((0, k), (1, v)):
                row = lambda u: pool[:, where(u)[0], :, where(u)[1]] * sc[:, where(u)[0], :, which, None]  # noqa: E731
                pages = {}
                for p in sorted({u // PAGE for u in moves}):
                    ts = [u for u in range(p * PAGE, p * PAGE + PAGE) if u <= root + a]
                    pages[p] = (ts, torch.stack([row(moves.get(u, u)) for u in ts], 2))   # [L][Hkv][rows][D]
                for p, (ts, val) in pages.items():
                    _exact_page(pool, sc, table[b][p], which, [u % PAGE for u in ts], val)
        ctx = torch.tensor([c - case["N"] + 1 + a for c, a in zip(lens, alen)], dtype=torch.int32)
        return {"ctx": ctx, "k": k, "v": v, "scales": sc}
    q_out, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
    sc = s["scales"].double()[None] if op == "append8" else None
    R, half = case["rotary"], case["half"]
    first = list(range(R // 2)) if half else list(range(0, R, 2))
    second = [j + R // 2 for j in first] if half else [j + 1 for j in first]
    turns = s["cos_sin"].double()
    for b, (c, n) in enumerate(zip(lens, _new_lens(case))):
        if not n:
            continue
        pos = torch.arange(c - n, c, device="cuda") if s["positions"] is None else s["positions"][b].long()
        z = torch.complex(turns[pos, :R // 2], turns[pos, R // 2:])[:, None]

        def turned(x):
            x = x[b, :n].double()
            w = torch.complex(x[..., first], x[..., second]) * z
            x[..., first], x[..., second] = w.real, w.imag
            return x

        q_out[b, :n] = turned(s["q"])
        for which, pool, rows in ((0, k, turned(s["kn"])), (1, v, s["vn"][b, :n].double())):
            for p in range((c - n) // PAGE, (c - 1) // PAGE + 1):
                lo, hi = max(p * PAGE, c - n), min(p * PAGE + PAGE, c)
                blk, val = table[b][p], rows[lo - (c - n):hi - (c - n)].transpose(0, 1)   # [Hkv][rows][D]
                if op == "append":
                    pool[blk, :, lo - p * PAGE:hi - p * PAGE] = val
                else:
                    old = pool[blk, :, :lo - p * PAGE] * sc[0, blk, :, which, None, None]
                    _exact_page(pool[None], sc, blk, which, list(range(hi - p * PAGE)),
                                torch.cat([old, val], 1)[None])
    out = {"q": q_out, "k": k, "v": v}
    if op == "append8":
        out["scales"] = sc[0]
    return out


def _exact_page(pool, sc, blk, which, at, val):
    """pool [L][nb][Hkv][16][D], val [L][Hkv][rows][D] in 64 bits: stored under the smallest fitting power of two."""
    top = val.abs().amax((-1, -2))
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(-100, 119)
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    e = torch.where((top <= 448 * torch.exp2(e - 1)) & (e > -100), e - 1, e)
    x = val / torch.exp2(e)[..., None, None]
    grid = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)  # e4m3: four significant bits
    pool[:, blk, :, at] = torch.round(x / grid) * grid                            # ties to even
    sc[:, blk, :, which] = torch.exp2(e)


def _exact_attend8(s):
    case = s["case"]
    N, Hq, Hkv, D = case["N"], case["Hq"], case["Hkv"], case["D"]
    out = torch.zeros((case["B"], N, Hq, D), dtype=torch.float64, device="cuda")
    for b, c in enumerate(_lens(case)):
        blk = s["table"][b, :-(-c // PAGE)].long()
        sc = s["scales"][blk].double()
        k = (s["k"][blk].double() * sc[..., 0, None, None]).transpose(0, 1).reshape(Hkv, -1, D)[:, :c]
        v = (s["v"][blk].double() * sc[..., 1, None, None]).transpose(0, 1).reshape(Hkv, -1, D)[:, :c]
        hidden = torch.zeros((N, c), dtype=torch.bool, device="cuda")
        for i in range(N):
            seen, j = [], i
            while j >= 0:
                seen.append(j)
                j = TREE[j] if case["tree"] else j - 1
            for j in range(N):
                hidden[i, c - N + j] = j not in seen
        for h in range(Hkv):
            G = Hq // Hkv
            q = s["q"][b, :, h * G:(h + 1) * G].double()                        # [N][G][D]
            w = torch.einsum("ngd,td->ngt", q, k[h]) / math.sqrt(D)
            w = torch.softmax(w.masked_fill(hidden[:, None], -math.inf), -1)
            out[b, :, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", w, v[h])
    return out
