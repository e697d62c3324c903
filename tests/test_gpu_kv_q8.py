"""The rotated append and the 8-bit KV cache on the GPU against tests/kv_reference.py: what append and commit leave
in memory bit for bit, the attention within the bound derived there."""
import math

import numpy as np
import pytest
import torch

import kv_reference as ref
import speculative_decoding_rl_b200 as sv
from speculative_decoding_rl_b200 import workloads as W
from speculative_decoding_rl_b200.session import AppendCall, AppendQ8Call, AttentionQ8Call, CommitQ8Call

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def same_bits(got, want):
    """NaN against NaN of any payload, all else bit for bit."""
    got, want = got.cpu(), want.cpu()
    nan = torch.isnan(want.float())
    assert torch.equal(torch.isnan(got.float()), nan)
    w = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[got.element_size()]
    eq = (got.contiguous().view(w) == want.contiguous().view(w)) | nan
    assert eq.all(), f"{int((~eq).sum())} of {eq.numel()} differ, first at {torch.nonzero(~eq)[0].tolist()}"


# ------------------------------------------------------------------ append
def run_append(q8, B, N, Hq, Hkv, D, R, interleaved, lens, seed, fused=False, positions=None, new_lens=None,
               with_q=True, spoil=None, rows=None):
    g, rng = gen(seed), np.random.default_rng(seed)
    mb = -(-max(lens) // 16) + 1
    table, nb = ref.table_for(lens, mb, rng)
    if q8:
        pools = list(ref.q8_pools(nb, Hkv, D, g))
    else:
        pools = [torch.randn((nb, Hkv, 16, D), generator=g).to(torch.bfloat16) for _ in range(2)]
    H = Hq + 2 * Hkv
    qkv = torch.randn((B, N, H, D), generator=g).to(torch.bfloat16)
    cs = ref.cos_sin(rows or max(lens), R) if R else None
    ctx = torch.tensor(lens, dtype=torch.int32)
    if spoil:
        spoil(qkv, pools, table, ctx, positions, nb)
    cut = lambda x: (x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:])  # noqa: E731
    q, k, v = cut(qkv)
    dq, dk, dv = cut(qkv.cuda())
    if not fused:
        dq, dk, dv = dq.contiguous(), dk.contiguous(), dv.contiguous()
    q_out = torch.full((B, N, Hq, D), 7.0, dtype=torch.bfloat16)
    dpos = None if positions is None else positions.cuda()
    dnl = None if new_lens is None else new_lens.cuda()
    dpools = [x.cuda() for x in pools]
    desc = sv.SvAttnDesc(B, N, Hq, Hkv, D, 16, mb, nb)
    rope = sv.make_rope_desc(None if cs is None else cs.cuda(), interleaved)
    call = (AppendQ8Call if q8 else AppendCall)(desc, rope, dpools, table.cuda(), ctx.cuda(), dq if with_q else None,
                                                dk, dv, positions=dpos, new_lens=dnl,
                                                q_out=q_out.cuda() if with_q else None)
    call.run()
    torch.cuda.synchronize()
    flags = ref.append(q if with_q else None, k, v, cs, interleaved, pools, table, ctx, q_out, positions, new_lens)
    assert call.status.tolist() == flags
    if with_q:
        same_bits(call.q_out, q_out)
        start = [c - (N if new_lens is None else int(new_lens[b])) for b, c in enumerate(lens)]
        if R and not any(flags):  # and against the formula in 64 bits
            for b in range(B):
                n = lens[b] - start[b]
                pos = torch.arange(start[b], lens[b]) if positions is None else positions[b, :n].long()
                y, mag = ref.rotate64(q[b, :n], cs[pos], interleaved)
                err = (call.q_out[b, :n].cpu().double() - y).abs()
                assert (err <= 2.0 ** -8 * y.abs() + 4 * 2.0 ** -24 * mag).all()
    for got, want in zip(dpools, pools):
        same_bits(got, want)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,R,interleaved,lens", [
    (1, 1, 4, 1, 64, 64, False, [1]),
    (1, 5, 28, 4, 128, 128, False, [6151]),
    (3, 5, 8, 2, 128, 128, True, [5, 16, 21]),
    (4, 9, 40, 8, 128, 64, False, [9, 32, 100, 17]),
    (2, 17, 4, 4, 64, 32, True, [17, 40]),
    (2, 33, 8, 1, 64, 16, False, [33, 64]),
    (2, 3, 16, 1, 128, 0, False, [3, 19]),
    (5, 64, 6, 2, 128, 112, False, [64, 65, 79, 80, 81]),
])
def test_append_leaves_the_formula(q8, B, N, Hq, Hkv, D, R, interleaved, lens):
    run_append(q8, B, N, Hq, Hkv, D, R, interleaved, lens, seed=100 + N)
    run_append(q8, B, N, Hq, Hkv, D, R, interleaved, lens, seed=200 + N, fused=True)


@pytest.mark.parametrize("D,R", [(8, 0), (48, 48), (80, 32), (256, 256), (200, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_other_head_sizes(D, R, interleaved):
    run_append(False, 2, 6, 6, 3, D, R, interleaved, [6, 40], seed=D)


@pytest.mark.parametrize("q8", [False, True])
def test_append_ragged_prompts_and_positions(q8):
    nl = torch.tensor([37, 0, 1, 16, 20], dtype=torch.int32)
    lens = [37, 50, 17, 16, 41]
    run_append(q8, 5, 37, 8, 2, 128, 128, False, lens, seed=1, new_lens=nl)
    pos = torch.randint(0, 500, (5, 37), generator=gen(2), dtype=torch.int32)
    run_append(q8, 5, 37, 8, 2, 128, 64, True, lens, seed=3, new_lens=nl, positions=pos, rows=500, fused=True)
    run_append(q8, 5, 37, 8, 2, 128, 64, True, lens, seed=4, new_lens=nl, with_q=False)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(256, 2, 1, 64), (300, 16, 2, 128), (259, 33, 3, 128)])
def test_append_long_ragged_prompts(q8, N, Hq, Hkv, D):
    # several groups of rows, or pages, to a CTA
    nl = torch.tensor([N, 0, N - 255, 17, N - 1], dtype=torch.int32)
    run_append(q8, 5, N, Hq, Hkv, D, D // 2, False, [N + 5, 30, N, 50, N - 1], seed=N, new_lens=nl, fused=True)


@pytest.mark.parametrize("q8", [False, True])
def test_append_flags_and_skips(q8):
    def spoil(qkv, pools, table, ctx, positions, nb):
        ctx[0] = 3                       # shorter than its new rows
        ctx[1] = table.shape[1] * 16 + 1  # longer than the table
        table[2, 1] = nb                 # one of its pages outside the pool
        table[3, 2] = -1
        positions[4, 18] = 500           # one row's position outside the table
        positions[5, 0] = -1
    pos = torch.randint(0, 500, (7, 20), generator=gen(5), dtype=torch.int32)
    run_append(q8, 7, 20, 8, 2, 64, 64, False, [25, 30, 36, 38, 30, 20, 30], seed=6, positions=pos, rows=500,
               spoil=spoil)
    nl = torch.tensor([-1, 21, 20], dtype=torch.int32)
    run_append(q8, 3, 20, 8, 2, 64, 64, False, [25, 30, 36], seed=7, new_lens=nl)


@pytest.mark.parametrize("q8", [False, True])
def test_append_nonfinite_and_extreme_rows(q8):
    def spoil(qkv, pools, table, ctx, positions, nb):
        qkv[0, 1] *= 3e38 / qkv[0, 1].abs().max()
        qkv[1, 0, :, 3] = math.inf
        qkv[1, 1, :, 5] = math.nan
        qkv[1, 2, 1] = -math.inf
        qkv[2] = 0
        qkv[3] *= 1e-36
        if q8:
            pools[0][:, :, 2, 1] = math.nan
            pools[2][0] = 2.0 ** -100
            pools[2][1] = 2.0 ** 60
    run_append(q8, 4, 4, 4, 2, 64, 0, False, [4, 22, 4, 9], seed=8, spoil=spoil)


def test_append_q8_takes_a_calibrated_cache():
    # scales that are no powers of two: kept rows come under one
    def spoil(qkv, pools, table, ctx, positions, nb):
        pools[2].copy_(torch.rand(pools[2].shape, generator=gen(11)) * 0.01 + 1e-4)
    run_append(True, 3, 5, 8, 2, 128, 128, False, [10, 24, 33], seed=12, spoil=spoil)


# ------------------------------------------------------------------ attention
def run_attend(N, Hq, Hkv, D, lens, seed, mask=None, spoil=None, q_scale=1.0, lo=-8, hi=-3, mb_more=0, stream=None):
    g, rng = gen(seed), np.random.default_rng(seed)
    B = len(lens)
    table, nb = ref.table_for(lens, -(-max(lens) // 16) + mb_more, rng)
    kv = list(ref.q8_pools(nb, Hkv, D, g, lo, hi))
    bytes_ = [x.view(torch.uint8) for x in kv[:2]]
    used = set()
    for b, C in enumerate(lens):  # entries behind the last row are NaN
        used.update(table[b, :-(-C // 16)].tolist())
        if C % 16:
            for x in bytes_:
                x[table[b, C // 16], :, C % 16:] = 0x7F
    for blk in set(range(nb)) - used:
        for x in bytes_:
            x[blk] = 0xFF
        kv[2][blk] = math.nan
    q = (torch.randn((B, N, Hq, D), generator=g) * q_scale).to(torch.bfloat16)
    ctx = torch.tensor(lens, dtype=torch.int32)
    if spoil:
        spoil(q, kv, table, ctx, nb)
    desc = sv.SvAttnDesc(B, N, Hq, Hkv, D, 16, table.shape[1], nb)
    call = AttentionQ8Call(desc, [x.cuda() for x in kv], table.cuda(), ctx.cuda(), q.cuda(),
                           None if mask is None else mask.cuda())
    call.out.fill_(7)
    call.workspace.fill_(255)
    call.run()
    torch.cuda.synchronize()
    want, tol = ref.attend64(q, kv, table, ctx, mask)
    return call, call.out.cpu().double(), want, tol


def check_attend(*a, **kw):
    call, got, want, tol = run_attend(*a, **kw)
    assert not call.status.any(), call.status
    assert torch.isfinite(got).all()
    err = (got - want).abs()
    assert (err <= tol).all(), f"worst {float((err / tol).max()):.3f} of the bound"
    assert torch.equal(call.run().cpu().double(), got)  # the same bits again
    return call


def tree_masks(parents, B):
    return torch.from_numpy(np.tile(W.ancestor_masks(parents), (B, 1)).view(np.int64).copy())


@pytest.mark.parametrize("N,Hq,Hkv,D,lens", [
    (1, 1, 1, 128, [1]), (1, 4, 1, 64, [1, 2, 16, 17]), (5, 28, 4, 128, [200, 1500, 5]),
    (9, 40, 8, 128, [9, 127, 128, 129, 1000]), (3, 16, 1, 128, [300]), (16, 8, 2, 64, [256, 255, 257, 16]),
    (16, 10, 2, 128, [700, 40]), (16, 10, 2, 64, [600]), (2, 8, 8, 128, [77]), (12, 16, 2, 128, [2049, 12]),
    (64, 8, 2, 128, [400, 64]), (64, 8, 2, 64, [90]), (1, 96, 1, 128, [333]), (4, 24, 1, 128, [150]),
    (7, 32, 8, 128, [513]), (13, 4, 1, 64, [1024]),
])
def test_attention_holds_its_bound(N, Hq, Hkv, D, lens):
    check_attend(N, Hq, Hkv, D, lens, seed=N * 7 + D)


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 4, 128), (8, 2, 64)])
def test_attention_tree_masks(Hq, Hkv, D):
    P = W.TREE_PARENTS_3221
    check_attend(len(P), Hq, Hkv, D, [700, 1031, len(P), 256], seed=31, mask=tree_masks(P, 4))


def test_attention_rows_that_see_nothing():
    m = torch.tensor([[1, 0, 2, 0], [0, 0, 0, 0], [0, 3, 0, 9]], dtype=torch.int64)
    call, got, want, tol = run_attend(4, 8, 2, 128, [4, 4, 60], seed=32, mask=m)
    assert not call.status.any()
    assert ((got - want).abs() <= tol).all()
    assert not got[1].any() and not got[0, 1].any() and not got[0, 3].any()


def test_attention_explicit_chain_equals_none():
    m = tree_masks(W.chain_parents(6), 2)
    a = run_attend(6, 8, 2, 128, [900, 333], seed=33)[1]
    b = run_attend(6, 8, 2, 128, [900, 333], seed=33, mask=m)[1]
    assert torch.equal(a, b)


def test_attention_long_split_units():
    check_attend(5, 16, 2, 128, [40000, 300], seed=34)
    check_attend(1, 4, 1, 64, [33333], seed=35)


def test_attention_many_short_sequences():
    lens = [1 + (37 * b) % 150 for b in range(512)]
    check_attend(1, 4, 2, 64, lens, seed=36)


@pytest.mark.parametrize("N,Hq,Hkv", [(3, 8, 2), (8, 12, 4), (10, 20, 4), (15, 8, 2), (11, 64, 8), (40, 12, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_several_units_to_a_range(N, Hq, Hkv, D):
    # 12 to 240 rows per KV head, units of one to three tiles, more of them than an SM's work ranges
    lens = [N + (53 * b) % 300 for b in range(200)]
    check_attend(N, Hq, Hkv, D, lens, seed=46)


@pytest.mark.parametrize("lo,hi,q_scale", [(-100, -99, 2.0 ** 90), (90, 101, 2.0 ** -105), (-60, 60, 2.0 ** -62)])
def test_attention_far_scales(lo, hi, q_scale):
    # scales at both ends of their range, and pages whose scales differ by up to 2^120
    check_attend(5, 8, 2, 128, [500, 33], seed=37, lo=lo, hi=hi, q_scale=q_scale)


def test_attention_scales_that_are_no_powers_of_two():
    def spoil(q, kv, table, ctx, nb):
        kv[2].copy_(torch.rand(kv[2].shape, generator=gen(1)) * 0.02 + 1e-3)
        kv[2][table[0, 1]] = 0.0          # counts as 2^-100
        kv[2][table[0, 2]] = 2.0 ** -120
    check_attend(5, 8, 2, 128, [500, 33], seed=38, spoil=spoil)


@pytest.mark.parametrize("q_scale", [20.0, 1e-6, 1e-30])
def test_attention_sharp_and_flat_softmax(q_scale):
    check_attend(5, 28, 4, 128, [900, 20], seed=39, q_scale=q_scale)


@pytest.mark.parametrize("gap", [8.0, 12.0, 15.0])
def test_attention_sink_over_a_flat_tail(gap):
    # one key far above thousands of equal ones, whose mass still counts: weights 2^-11 to 2^-21 of the largest
    def spoil(q, kv, table, ctx, nb):
        kv[0].copy_(torch.zeros(kv[0].shape).to(F8))
        kv[2].fill_(2.0 ** -6)
        q.fill_(1.0)
        kv[0][table[0, 3], :, 5, 0] = 448.0
        kv[2][table[0, 3], :, 0] = gap * math.sqrt(128) / 448
    check_attend(5, 8, 2, 128, [20000], seed=40, spoil=spoil)


@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 22, 2.0 ** 40])
@pytest.mark.parametrize("N,Hq,D", [(1, 4, 64), (5, 8, 128), (11, 16, 128)])
def test_attention_huge_scores_pick_one_key(size, N, Hq, D):
    # scores of `size` and more apart, to the end of what fp32 counts in: all weight on the largest
    def spoil(q, kv, table, ctx, nb):
        q.zero_()
        q[..., 0] = size
        kv[2][..., 0] = 1.0
        kv[0][..., 0] = torch.randint(-20, 20, kv[0].shape[:3], generator=gen(3)).float().to(F8)
        kv[0][table[0, 2], :, 9, 0] = 22.0
        kv[0][table[1, 0], :, 3, 0] = 22.0
    call, got, want, tol = run_attend(N, Hq, 2, D, [1500, 20], seed=47, spoil=spoil)
    assert not call.status.any()
    # exp(-2 * 2^10 / sqrt(D)) of the other keys is below 2^-180: the picked key's V, rounded once
    v = [call.pools[1][call.block_table[b, p], :, r].cpu().double() *
         call.pools[2][call.block_table[b, p], :, 1, None].cpu().double() for b, p, r in ((0, 2, 9), (1, 0, 3))]
    for b in range(2):
        pick = v[b].repeat_interleave(Hq // 2, 0)[None].expand(N, Hq, D)
        assert ((got[b] - pick).abs() <= (2.0 ** -8 + 2.0 ** -9) * pick.abs()).all()


def test_attention_rows_of_unlike_size():
    # a row's precision is its own, whatever the size of its neighbours
    def spoil(q, kv, table, ctx, nb):
        q[0, 0] *= 2.0 ** 40
        q[0, 1] *= 2.0 ** -40
        q[0, 2, 0] = 0
        q[0, 3, :, ::2] *= 2.0 ** -12
    check_attend(5, 8, 2, 128, [300], seed=41, spoil=spoil)


def test_attention_rising_scores():
    # every page's scores above the last one's: the running maximum rises all along
    def spoil(q, kv, table, ctx, nb):
        q.copy_(q.abs())
        kv[0].copy_(kv[0].float().abs().to(F8))
        for j in range(table.shape[1]):
            kv[2][table[0, j], :, 0] = 2.0 ** -9 * 1.09 ** j
    check_attend(5, 8, 2, 128, [1600], seed=42, spoil=spoil)


def test_attention_flags_invalid_sequences():
    def spoil(q, kv, table, ctx, nb):
        ctx[0] = 4
        ctx[1] = table.shape[1] * 16 + 1
        table[2, 3] = nb + 5
        table[2, 4] = -2
    call, got, want, tol = run_attend(5, 8, 2, 128, [300, 300, 300, 299], seed=43, spoil=spoil)
    assert call.status.tolist() == [2, 2, 8, 0]
    assert not got[0].any() and not got[1].any()
    assert ((got - want).abs() <= tol).all()


def test_attention_hidden_nan_stays_hidden():
    # a rejected branch's K and V may hold NaN: only rows that see the node see it
    P = W.TREE_PARENTS_3221

    def spoil(q, kv, table, ctx, nb):
        for b, C in enumerate(ctx.tolist()):
            for node in (2, 3):
                t = C - len(P) + node
                kv[0].view(torch.uint8)[table[b, t // 16], 0, t % 16, 7] = 0x7F
                kv[1].view(torch.uint8)[table[b, t // 16], :, t % 16, 11 + node] = 0xFF
    for D, Hkv in ((128, 4), (64, 2)):
        call, got, want, tol = run_attend(len(P), 32, Hkv, D, [500, 11, 140, 4000], seed=44,
                                          mask=tree_masks(P, 4), spoil=spoil)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        ok = ~torch.isnan(want)
        assert ((got - want).abs()[ok] <= tol[ok]).all()
        assert torch.isfinite(got[:, 1]).all() and torch.isnan(got[:, 2]).any()


def test_attention_nonfinite_queries_stay_in_their_row():
    def spoil(q, kv, table, ctx, nb):
        q[0, 1, 3, 5] = math.nan
        q[0, 2, 4, 6] = math.inf
    call, got, want, tol = run_attend(4, 8, 2, 128, [400], seed=45, spoil=spoil)
    bad = torch.zeros(4, 8, dtype=torch.bool)
    bad[1, 3] = bad[2, 4] = True
    assert torch.equal(torch.isnan(got[0]).all(-1), bad) and torch.equal(torch.isnan(got[0]).any(-1), bad)
    err = (got - want).abs()[0][~bad]
    assert (err <= tol[0][~bad]).all()


# ------------------------------------------------------------------ commit
def run_commit(parents, Hkv, D, lens, L, seed, spoil=None, max_len=None):
    g, rng = gen(seed), np.random.default_rng(seed)
    N, B = (5, len(lens)) if parents is None else (len(parents), len(lens))
    mb = -(-max(lens) // 16) + 1
    table, nb = ref.table_for(lens, mb, rng)
    layers = [list(ref.q8_pools(nb, Hkv, D, g)) for _ in range(L)]
    alen, path = W.make_accept_paths(N, parents, B, seed=seed, max_len=max_len)
    ctx = torch.tensor(lens, dtype=torch.int32)
    if spoil:
        spoil(layers, table, ctx, alen, path, nb)
    dev = [[x.cuda() for x in layer] for layer in layers]
    desc = sv.SvAttnDesc(B, N, Hkv, Hkv, D, 16, mb, nb)
    call = CommitQ8Call(desc, dev, table.cuda(), ctx.cuda(), alen.cuda(), path.cuda())
    got = call.run()
    torch.cuda.synchronize()
    new_ctx, flags = ref.commit_q8(layers, table, ctx, alen, path, N)
    assert got.tolist() == new_ctx and call.status.tolist() == flags
    for d, w in zip(dev, layers):
        for x, y in zip(d, w):
            same_bits(x, y)
    return flags


@pytest.mark.parametrize("parents,Hkv,D", [(None, 2, 128), ("tree", 4, 128), ("tree", 2, 64), ("random64", 2, 128),
                                           ("random64", 1, 64), ([-1], 1, 64)])
def test_commit_q8_leaves_the_formula(parents, Hkv, D):
    if parents == "tree":
        parents = W.TREE_PARENTS_3221
    elif parents == "random64":
        rng = np.random.default_rng(5)
        parents = [-1] + [int(rng.integers(max(0, c - 6), c)) for c in range(1, 64)]
    N = 5 if parents is None else len(parents)

    def spoil(layers, table, ctx, alen, path, nb):
        alen[0], path[0] = 0, -1
        for layer in layers:
            layer[0].view(torch.uint8)[:, :, 5, 3] = 0x7F
            layer[2][::3] *= 2.0 ** 20
    run_commit(parents, Hkv, D, [N, N + 1, N + 16, N + 17, N + 30, N + 7, N + 9, N + 100], 3, seed=61, spoil=spoil)


def test_commit_q8_flags():
    P = W.TREE_PARENTS_3221

    def spoil(layers, table, ctx, alen, path, nb):
        ctx[0] = 5
        ctx[1] = table.shape[1] * 16 + 1
        table[2, int(ctx[2] - 1) // 16] = nb
        alen[3] = 11
        alen[4], path[4, :3] = 3, torch.tensor([2, 2, 5], dtype=torch.int32)
        alen[5], path[5, :2] = 2, torch.tensor([3, 11], dtype=torch.int32)
    flags = run_commit(P, 2, 64, [200, 40, 60, 60, 60, 60, 70], 2, seed=62, spoil=spoil, max_len=3)
    assert flags == [2, 2, 8, 32, 32, 32, 0]


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 28, 4), (64, 8, 2)])
def test_steps_of_a_rollout(D, Hq, Hkv):
    """Prompts, then verify steps of a draft tree: append, attention, commit, captured in a graph and replayed."""
    P = W.TREE_PARENTS_3221
    N, B, L, R = len(P), 3, 2, D
    g, rng = gen(71), np.random.default_rng(71)
    prompts, mb = [40, 7, 29], 8
    nb = B * mb + 1
    table = torch.from_numpy(rng.permutation(nb)[:B * mb].reshape(B, mb).astype(np.int32))
    zeros = lambda: [torch.zeros((nb, Hkv, 16, D)).to(F8), torch.zeros((nb, Hkv, 16, D)).to(F8),  # noqa: E731
                     torch.ones((nb, Hkv, 2))]
    host = [zeros() for _ in range(L)]
    dev = [[x.cuda() for x in layer] for layer in host]
    cs = ref.cos_sin(256, R)
    rope = sv.make_rope_desc(cs.cuda())
    dtable, dctx = table.cuda(), torch.tensor(prompts, dtype=torch.int32).cuda()
    S = max(prompts)
    pq = [torch.randn((B, S, Hq + 2 * Hkv, D), generator=g).to(torch.bfloat16) for _ in range(L)]
    nl = torch.tensor(prompts, dtype=torch.int32)
    for layer in range(L):
        x = pq[layer].cuda()
        AppendQ8Call(sv.SvAttnDesc(B, S, Hq, Hkv, D, 16, mb, nb), rope, dev[layer], dtable, dctx, x[:, :, :Hq],
                     x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], new_lens=nl.cuda()).run()
        y = pq[layer]
        ref.append(None, y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:], cs, False, host[layer], table, prompts, None,
                   new_lens=nl)
    depth = [0] * N
    for c in range(1, N):
        depth[c] = depth[P[c]] + 1
    qkv = [torch.zeros((B, N, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(L)]
    pos = torch.zeros((B, N), dtype=torch.int32, device="cuda")
    ctx = torch.tensor([c + N for c in prompts], dtype=torch.int32).cuda()
    mask = tree_masks(P, B)
    desc = sv.SvAttnDesc(B, N, Hq, Hkv, D, 16, mb, nb)
    alen, path = torch.zeros(B, dtype=torch.int32).cuda(), torch.zeros((B, N - 1), dtype=torch.int32).cuda()
    calls = []
    for layer in range(L):
        x = qkv[layer]
        a = AppendQ8Call(desc, rope, dev[layer], dtable, ctx, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:],
                         positions=pos)
        calls += [a, AttentionQ8Call(desc, dev[layer], dtable, ctx, a.q_out, mask.cuda())]
    commit = CommitQ8Call(desc, dev, dtable, ctx, alen, path)
    calls.append(commit)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    saved = [[x.clone() for x in layer] for layer in dev]
    with torch.cuda.stream(side):
        for c in calls:
            c.run()
    torch.cuda.synchronize()
    for layer, old in zip(dev, saved):
        for x, y in zip(layer, old):
            x.copy_(y)
    with torch.cuda.graph(graph):
        for c in calls:
            c.run()
    lens = list(prompts)
    for step in range(3):
        rows = [torch.randn((B, N, Hq + 2 * Hkv, D), generator=g).to(torch.bfloat16) for _ in range(L)]
        hpos = torch.tensor([[c + d for d in depth] for c in lens], dtype=torch.int32)
        now = [c + N for c in lens]
        al, pa = W.make_accept_paths(N, P, B, seed=80 + step)
        for layer in range(L):
            qkv[layer].copy_(rows[layer])
        pos.copy_(hpos)
        ctx.copy_(torch.tensor(now, dtype=torch.int32))
        alen.copy_(al)
        path.copy_(pa)
        graph.replay()
        torch.cuda.synchronize()
        for layer in range(L):
            y = rows[layer]
            qo = torch.zeros((B, N, Hq, D), dtype=torch.bfloat16)
            assert ref.append(y[:, :, :Hq], y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:], cs, False, host[layer], table,
                              now, qo, positions=hpos) == [0] * B
            same_bits(calls[2 * layer].q_out, qo)
            want, tol = ref.attend64(qo, host[layer], table, now, mask)
            assert ((calls[2 * layer + 1].out.cpu().double() - want).abs() <= tol).all()
        lens, flags = ref.commit_q8(host, table, now, al, pa, N)
        assert commit.new_ctx_lens.tolist() == lens and not any(flags)
        for d, w in zip(dev, host):
            for x, y in zip(d, w):
                same_bits(x, y)


def test_calls_on_another_stream():
    side = torch.cuda.Stream()
    call, got, want, tol = run_attend(5, 8, 2, 128, [700], seed=91)
    torch.cuda.synchronize()
    call.out.fill_(3)
    torch.cuda.synchronize()
    call.run(stream=side)
    side.synchronize()
    assert torch.equal(call.out.cpu().double(), got)


def test_offsets_past_32_bits():
    """A cache of more than 4 GB to a pool: every call on its last blocks."""
    Hkv, D, N, Hq = 8, 128, 11, 8
    nb = (1 << 32) // (Hkv * 16 * D) + 70
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    g = gen(95)
    k, v = (torch.empty((nb, Hkv, 16, D), dtype=F8, device="cuda") for _ in range(2))
    scales = torch.empty((nb, Hkv, 2), device="cuda")
    last = torch.arange(nb - 64, nb)
    small = list(ref.q8_pools(64, Hkv, D, g))
    for big, part in zip((k, v, scales), small):
        big[nb - 64:] = part.cuda()
    table = torch.from_numpy(np.random.default_rng(95).permutation(64)[:60].reshape(2, 30).astype(np.int32))
    dtable = (table + (nb - 64)).to(torch.int32).cuda()
    lens = [470, 301]
    ctx = torch.tensor(lens, dtype=torch.int32)
    cs = ref.cos_sin(480, D)
    x = torch.randn((2, N, Hq + 2 * Hkv, D), generator=g).to(torch.bfloat16)
    dx = x.cuda()
    desc = sv.SvAttnDesc(2, N, Hq, Hkv, D, 16, 30, nb)
    cut = lambda t: (t[:, :, :Hq], t[:, :, Hq:Hq + Hkv], t[:, :, Hq + Hkv:])  # noqa: E731
    a = AppendQ8Call(desc, sv.make_rope_desc(cs.cuda()), (k, v, scales), dtable, ctx.cuda(), *cut(dx))
    mask = tree_masks(W.TREE_PARENTS_3221, 2)
    t = AttentionQ8Call(desc, (k, v, scales), dtable, ctx.cuda(), a.run(), mask.cuda())
    t.run()
    alen, path = W.make_accept_paths(N, W.TREE_PARENTS_3221, 2, seed=96)
    c = CommitQ8Call(desc, [(k, v, scales)], dtable, ctx.cuda(), alen.cuda(), path.cuda())
    c.run()
    torch.cuda.synchronize()
    qo = torch.zeros((2, N, Hq, D), dtype=torch.bfloat16)
    ref.append(*cut(x), cs, False, small, table, ctx, qo)
    want, tol = ref.attend64(qo, small, table, ctx, mask)
    same_bits(a.q_out, qo)
    assert ((t.out.cpu().double() - want).abs() <= tol).all()
    ref.commit_q8([small], table, ctx, alen, path, N)
    for big, part in zip((k, v, scales), small):
        same_bits(big[last.cuda()], part)
