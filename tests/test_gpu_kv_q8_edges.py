"""The 8-bit KV cache's calls where they are easily wrong. What append and commit leave in memory is compared bit for
bit, the attention within bounds that follow from its documented roundings."""
import math
import time

import numpy as np
import pytest
import torch

import kv_reference as ref
import speculative_decoding_rl_b200 as sv
from speculative_decoding_rl_b200.session import AppendQ8Call, CommitQ8Call
from test_gpu_kv_q8 import F8, gen, run_append, run_attend, same_bits

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("how", ["block", "position"])
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 2, 128), (64, 5, 64)])
def test_append_of_long_ragged_prompts_skips_pages_among_others(how, Hq, Hkv, D):
    # work enough for a CTA to go over four pages: of every four, one or two in the middle are skipped, in every pattern;
    # rows of unlike size, so that the halves of a page and its neighbours ask for different scales
    N, lens = 320, [320, 331, 325, 400, 322, 328] * 5
    nl = torch.tensor([320, 320, 300, 257, 320, 311] * 5, dtype=torch.int32)
    starts = [c - int(n) for c, n in zip(lens, nl)]
    pos = torch.randint(0, 500, (len(lens), N), generator=gen(5), dtype=torch.int32) if how == "position" else None

    def spoil(qkv, pools, table, ctx, positions, nb):
        qkv.mul_(torch.exp2(torch.randint(-8, 9, (len(lens), N, 1, 1), generator=gen(6)).float()).to(torch.bfloat16))
        for b, (c, start) in enumerate(zip(lens, starts)):
            skip = [(1,), (2,), (1, 2), (0, 2), (1, 3), (3,)][b % 6]
            for p in range(start // 16, (c - 1) // 16 + 1):
                if (p - start // 16) % 4 in skip:
                    if how == "block":
                        table[b, p] = -1 if p & 1 else nb + p
                    else:
                        positions[b, max(p * 16, start) - start + (p % 5 if p * 16 >= start else 0)] = -1 if p & 1 else 500
    run_append(True, len(lens), N, Hq, Hkv, D, D, False, lens, seed=51, positions=pos,
               new_lens=nl, spoil=spoil, rows=500, fused=True)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("B,N", [(17, 259), (1, 259)])
def test_append_of_long_prompts(q8, ragged, B, N):
    # many of them, several groups of rows or pages to a CTA; a single one
    lens = [N + 7 * b % 20 for b in range(B)]
    nl = torch.tensor([max(0, N - 31 * b) for b in range(B)], dtype=torch.int32) if ragged else None
    run_append(q8, B, N, 33, 3, 128, 64, False, lens, seed=56, new_lens=nl, fused=True)


@pytest.mark.parametrize("tiny", [0.0, 2.0 ** -120])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_below_the_smallest_count_as_it_to_append_and_commit(tiny, D):
    # to the attention such a page's entries stand for e4m3 value * 2^-100: written back they still do
    N, B, Hkv = 3, 3, 2
    lens = [8, 21, 19]
    table, nb = ref.table_for(lens, 3, np.random.default_rng(7))
    host = list(ref.q8_pools(nb, Hkv, D, gen(57)))
    dev = [x.cuda() for x in host]
    host[2].fill_(2.0 ** -100)
    dev[2].fill_(tiny)
    rows = torch.randn((B, N, Hkv, D), generator=gen(58))
    rows[0], rows[2] = 0, rows[2] * 2.0 ** -95           # all that is kept, and rows of its size
    rows = rows.to(torch.bfloat16)
    desc = sv.SvAttnDesc(B, N, Hkv, Hkv, D, 16, 3, nb)
    ctx = torch.tensor(lens, dtype=torch.int32)
    drows, dtable, dctx = rows.cuda(), table.cuda(), ctx.cuda()
    append = AppendQ8Call(desc, sv.make_rope_desc(None), dev, dtable, dctx, None, drows, drows)
    # a page that is not written keeps its scale; for the comparison it counts as the smallest
    append.run()
    assert ref.append(None, rows, rows, None, False, host, table, ctx, None) == append.status.tolist() == [0] * B
    for got, want in zip(dev, host):
        same_bits(got.clamp(min=2.0 ** -100) if got.dtype == torch.float32 else got, want)
    dev[2].copy_(torch.where(dev[2] == 2.0 ** -100, torch.full_like(dev[2], tiny), dev[2]))
    alen, path = torch.tensor([1, 1, 2], dtype=torch.int32), torch.tensor([[2, 0], [2, 0], [1, 2]], dtype=torch.int32)
    commit = CommitQ8Call(desc, [dev], dtable, dctx, alen.cuda(), path.cuda())
    new_ctx, flags = ref.commit_q8([host], table, ctx, alen, path, N)
    assert commit.run().tolist() == new_ctx and commit.status.tolist() == flags == [0] * B
    for got, want in zip(dev, host):
        same_bits(got.clamp(min=2.0 ** -100) if got.dtype == torch.float32 else got, want)


@pytest.mark.parametrize("outlier", [2.0 ** 4, 2.0 ** 10, 2.0 ** 20])
def test_what_a_rejected_outlier_leaves_in_its_page(outlier):
    # ten rows, a draft row far larger than they are, its rejection, an ordinary row: against the page that never held
    # the outlier
    D, Hkv = 128, 2
    rows = torch.randn((1, 12, Hkv, D), generator=gen(59)).to(torch.bfloat16)
    big = (rows[:, 11:] * outlier).to(torch.bfloat16)
    table = torch.tensor([[0]], dtype=torch.int32).cuda()

    def cache():
        return [torch.zeros((1, Hkv, 16, D)).to(F8).cuda(), torch.zeros((1, Hkv, 16, D)).to(F8).cuda(),
                torch.ones((1, Hkv, 2), device="cuda")]

    def append(kv, ctx, x):
        n = x.shape[1]
        x = x.cuda()
        AppendQ8Call(sv.SvAttnDesc(1, n, Hkv, Hkv, D, 16, 1, 1), sv.make_rope_desc(None), kv, table,
                     torch.tensor([ctx], dtype=torch.int32).cuda(), None, x, x).run()
        torch.cuda.synchronize()

    def values(kv):
        return (kv[0].cpu().double() * kv[2].cpu().double()[..., :1, None])[0, :, :11]
    plain, kv = cache(), cache()
    append(plain, 10, rows[:, :10])
    append(plain, 11, rows[:, 10:11])
    append(kv, 10, rows[:, :10])
    before = kv[2].cpu().clone()
    append(kv, 11, big)
    raised = kv[2].cpu().clone()
    top = big.abs().double().amax((1, 3))[0]                                   # [Hkv]
    assert (raised > before).all() and (top <= 448 * raised[0, :, 0]).all()
    commit = CommitQ8Call(sv.SvAttnDesc(1, 1, Hkv, Hkv, D, 16, 1, 1), [kv], table,
                          torch.tensor([10], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
                          torch.zeros((1, 1), dtype=torch.int32).cuda())
    assert commit.run().tolist() == [10]
    assert torch.equal(kv[2].cpu(), raised)                                    # nothing moved, nothing is written
    append(kv, 11, rows[:, 10:11])
    want, got, step = values(plain), values(kv), raised[0, :, :1, None].double() * 2.0 ** -9
    kept = want.abs() >= 2.0 ** -13 * top[:, None, None]
    assert torch.equal(got[kept], want[kept])
    # the rest were rounded once to the subnormals of the raised scale; the last row never was under it
    assert ((got - want).abs() <= step / 2).all() and torch.equal(got[:, 10], want[:, 10])


# ------------------------------------------------------------------ attention
def one_dim_scores(size, tops):
    """Scores along one dimension, whole numbers from -20 to 20 times `size`; the keys of `tops` (sequence, position)
    stand above them at 22 * size."""
    def spoil(q, kv, table, ctx, nb):
        q.zero_()
        q[..., 0] = size
        kv[2][..., 0] = 1.0
        kv[0].copy_(torch.zeros(kv[0].shape).to(F8))
        kv[0][..., 0] = torch.randint(-20, 20, kv[0].shape[:3], generator=gen(3)).float().to(F8)
        for b, t in tops:
            kv[0][table[b, t // 16], :, t % 16, 0] = 22.0
    return spoil


def value(call, b, t):
    """V of a key in 64 bits, [Hkv][D], and its scales."""
    blk = int(call.block_table[b, t // 16])
    sc = call.pools[2][blk, :, 1, None].cpu().double()
    return call.pools[1][blk, :, t % 16].cpu().double() * sc, sc


@pytest.mark.parametrize("size", [2.0 ** 17, 2.0 ** 23, 2.0 ** 28, 2.0 ** 30, 2.0 ** 60, 2.0 ** 120])
@pytest.mark.parametrize("lo,hi", [(1, 5), (-40, -24), (90, 101), (-100, -90)])
@pytest.mark.parametrize("N,Hq,D,lens", [(1, 4, 64, [1500, 20]), (5, 8, 128, [1500, 20]), (12, 8, 128, [60, 700]),
                                         (16, 8, 64, [400, 20]), (11, 16, 128, [300, 24000])])
def test_attention_huge_scores_whatever_the_scale_of_v(size, lo, hi, N, Hq, D, lens):
    # scores whose spacing is far beyond log2 of V's scale; all weight on one key
    tops = [(0, 41), (1, {20: 3, 700: 600, 24000: 17001}[lens[1]])]
    call, got, want, tol = run_attend(N, Hq, 2, D, lens, seed=52, spoil=one_dim_scores(size, tops), lo=lo, hi=hi)
    assert not call.status.any()
    # the next key is exp(-2 * 2^17 / sqrt(D)) < 2^-300 lower. What is left of the bound: the weight enters the
    # product rounded to 2^-9 of itself, the sum it is divided by is that weight in fp32 (2^-20 with the exponential),
    # the output is rounded to bf16
    for b, t in tops:
        v = value(call, b, t)[0].repeat_interleave(Hq // 2, 0)[None].expand(N, Hq, D)
        assert ((got[b] - v).abs() <= (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -19) * v.abs()).all()


@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 28, 2.0 ** 31, 2.0 ** 70])
@pytest.mark.parametrize("gap", [0, 8, 14, 60, 90])
def test_attention_equal_huge_scores_under_unlike_scales(size, gap):
    # two keys with the same score in tiles of different ranges, V's scales 2^gap apart: the mean of their values
    tops = [(0, 41), (0, 15000)]
    more = one_dim_scores(size, tops)

    def spoil(q, kv, table, ctx, nb):
        more(q, kv, table, ctx, nb)
        kv[2][table[0, 41 // 16], :, 1] = 2.0 ** (gap // 2)
        kv[2][table[0, 15000 // 16], :, 1] = 2.0 ** (gap // 2 - gap)
    call, got, want, tol = run_attend(5, 8, 2, 128, [20000], seed=53, spoil=spoil)
    assert not call.status.any()
    (v0, s0), (v1, s1) = (value(call, 0, t) for _, t in tops)
    # each weight is off by 2^-9 of itself or, far below the largest weight times scale, by 2^-24 of that
    bound = 2.0 ** -8 * (v0 + v1).abs() / 2 + (2.0 ** -9 + 2.0 ** -19) * (v0.abs() + v1.abs()) / 2 \
        + 2.0 ** -24 * s0 / 2 * (v1 / s1).abs()
    v, bound = (x.repeat_interleave(4, 0)[None].expand(5, 8, 128) for x in ((v0 + v1) / 2, bound))
    assert ((got[0] - v).abs() <= bound).all()


@pytest.mark.parametrize("gap", [120, 130, 160, 200])
@pytest.mark.parametrize("D,N,Hq,C", [(128, 5, 8, 300), (64, 1, 4, 700), (128, 11, 16, 400), (128, 5, 8, 20000)])
@pytest.mark.parametrize("last", [True, False])
def test_attention_scales_of_v_further_apart_than_fp32(gap, D, N, Hq, C, last):
    # keys of equal weight whose V scales differ by 2^gap: those of the small scale count in the sum of the weights
    # although their part of the output is nothing beside the others'
    def spoil(q, kv, table, ctx, nb):
        kv[0].copy_(torch.zeros(kv[0].shape).to(F8))
        kv[2][..., 1] = 2.0 ** -(gap // 2)
        for p in range(-(-C // 16)):
            if (p >= C // 32) == last:
                kv[2][table[0, p], :, 1] = 2.0 ** (gap - gap // 2)
    call, got, want, tol = run_attend(N, Hq, 2, D, [C], seed=54, spoil=spoil)
    assert not call.status.any()
    # every weight is 1 / (keys seen), exact but for 2^-20; what is left of the bound: the weights' 2^-9, 2^-24 of the
    # largest weight times scale for each of the others, and the output's rounding
    sc = call.pools[2][call.block_table[0].long(), :, 1].cpu().double()                        # [pages][Hkv]
    v = call.pools[1][call.block_table[0].long()].cpu().double() * sc[..., None, None]
    v = v.transpose(0, 1).reshape(2, -1, D)[:, :C]                                             # [Hkv][C][D]
    v8 = (v / sc.T.repeat_interleave(16, 1)[:, :C, None]).abs()
    for i in range(N):
        n = C - N + i + 1
        o, A = v[:, :n].sum(1) / n, v[:, :n].abs().sum(1) / n
        bound = 2.0 ** -8 * o.abs() + (2.0 ** -9 + 2.0 ** -19) * A + 2.0 ** -24 * sc.max() / n * v8[:, :n].sum(1)
        for h in range(Hq):
            kvh = h // (Hq // 2)
            assert ((got[0, i, h] - o[kvh]).abs() <= bound[kvh]).all()


@pytest.mark.parametrize("role", [sv.SV_STALL_SOFTMAX, sv.SV_STALL_MMA, sv.SV_STALL_LOADS, sv.SV_STALL_AUX])
@pytest.mark.parametrize("limit_ms", [5, 50])
@pytest.mark.parametrize("N,Hq,D,lens", [(1, 4, 64, [30, 9000]), (5, 8, 128, [900, 2100, 37, 40000, 640]),
                                         (9, 10, 128, [3000]), (16, 8, 64, [5000, 16]), (11, 16, 128, [11, 30000])])
def test_attention_wait_that_runs_out(role, limit_ms, N, Hq, D, lens):
    # one role of every CTA does nothing and the others' waits run out: the call returns within its limits, flags every
    # sequence, and leaves nothing behind that the next call would notice
    call, got, want, tol = run_attend(N, Hq, 2, D, lens, seed=55)
    status = torch.full((len(lens),), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    sv.sv_testing_verify_attention_q8_stalled(call.desc, call.q, call.kv, call.block_table, call.ctx_lens, call.mask,
                                              call.out, call.workspace, call.ws_bytes, status, limit_ms * 1_000_000,
                                              role)
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    assert (status.cpu() & sv.SV_FLAG_TIMEOUT).all(), status
    assert limit_ms / 1000 <= elapsed < 4.0, elapsed  # the limit, and 2 s at most for copies and products in flight
    assert torch.equal(call.run().cpu().double(), got)
    assert not call.status.any()


@pytest.mark.parametrize("N,Hq,D,lens", [(1, 4, 64, [300]), (5, 8, 128, [20000, 40]), (11, 16, 128, [700])])
@pytest.mark.parametrize("k_scale", [2.0 ** 60, 2.0 ** 100])
def test_attention_scores_past_fp32_are_nan_in_their_row_alone(N, Hq, D, lens, k_scale):
    def spoil(q, kv, table, ctx, nb):
        kv[2][..., 0] = k_scale
        q.mul_(1 / k_scale)
        q[0, N - 1, 1] = 2.0 ** 100       # a score of either sign beyond 2^128
    call, got, want, tol = run_attend(N, Hq, 2, D, lens, seed=65, spoil=spoil)
    bad = torch.zeros(got.shape[:3], dtype=torch.bool)
    bad[0, N - 1, 1] = True
    assert not call.status.any()
    assert torch.equal(torch.isnan(got).all(-1), bad) and torch.equal(torch.isnan(got).any(-1), bad)
    assert ((got - want).abs()[~bad] <= tol[~bad]).all()


# ------------------------------------------------------------------ scores that are whole numbers
# In test_gpu_kv_q8.py a score may be off by what fp32 may lose in a sum of D products, and large scores make that
# bound wide. Here q is a power of two in its first dimensions and zero elsewhere, and the first entries of a key add
# up to a whole number: every score is exact but for the factor log2(e) / sqrt(D), and little is left of the bound.
DIMS = 6


def whole_number_keys(n):
    """e4m3 entries [..., DIMS] whose sum is n, whole numbers of at most 2000 either way."""
    rest, parts = n.double().clone(), []
    for _ in range(DIMS):
        x = rest.clamp(-448, 448)
        unit = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=1))) - 3).clamp(min=1)
        x = torch.trunc(x / unit) * unit
        parts.append(x)
        rest = rest - x
    assert not rest.any()
    return torch.stack(parts, -1).float().to(F8)


def run_whole(N, Hq, D, levels, q_row, seed, mask=None, scales=None, **kw):
    """levels: for each sequence its keys' scores in powers of two (before q_row [N][Hq]'s factor), rounded to whole
    multiples of log2(e) / sqrt(D). Compares with the formula in 64 bits."""
    lens = [len(x) for x in levels]
    unit = math.log2(math.e) / math.sqrt(D)
    ns = [torch.round(torch.tensor(x, dtype=torch.float64) / unit) for x in levels]

    def spoil(q, kv, table, ctx, nb):
        q.zero_()
        q[..., :DIMS] = q_row[None, :, :, None]
        kv[0][:] = torch.zeros(kv[0].shape).to(F8)
        kv[2][..., 0] = 1.0
        for b, n in enumerate(ns):
            keys = whole_number_keys(n)
            for p in range(-(-len(n) // 16)):
                part = keys[p * 16:p * 16 + 16]
                kv[0][table[b, p], :, :len(part), :DIMS] = part
        if scales:
            scales(kv, table)
    call, got, _, _ = run_attend(N, Hq, 2, D, lens, seed=seed, spoil=spoil, mask=mask, **kw)
    assert not call.status.any()
    worst = 0.0
    for b, (C, n) in enumerate(zip(lens, ns)):
        blk = call.block_table[b, :-(-C // 16)].long().cpu()
        sc = call.pools[2].cpu().double()[blk][..., 1].T.repeat_interleave(16, 1)[:, :C]              # [Hkv][C]
        v8 = call.pools[1].cpu()[blk].double().transpose(0, 1).reshape(2, -1, D)[:, :C]
        for i in range(N):
            seen = torch.ones(C, dtype=torch.bool)
            for j in range(N):
                seen[C - N + j] = j <= i if mask is None else bool(int(mask[b, i]) >> j & 1)
            for h in range(Hq):
                s, kvh = n * float(q_row[i, h]) * unit, h // (Hq // 2)
                s = torch.where(seen, s, torch.full_like(s, -math.inf))
                top = s.max()
                w = torch.exp2(s - top)
                w = w / w.sum()
                o, A = w @ (v8[kvh] * sc[kvh, :, None]), w @ (v8[kvh].abs() * sc[kvh, :, None])
                # the score's three roundings and the factor's, 2^-24 each, and that of the difference; none where
                # all weight is on keys of one score
                d = 0.0 if bool((w[s < top] == 0).all()) else float(s[seen].abs().max()) * 2.0 ** -21 * math.log(2)
                bound = 2.0 ** -8 * o.abs() + (2.0 ** -9 + 2.0 ** -20 + 2 * math.expm1(d)) * A * 1.01 \
                    + 2.0 ** -24 * float((w * sc[kvh]).max()) * (seen.double() @ v8[kvh].abs())
                assert (bound <= 2.0 ** -6.5 * (v8[kvh].abs() * sc[kvh, :, None]).max()).all()  # it can fail
                err = (got[b, i, h] - o).abs()
                worst = max(worst, float((err / bound).max()))
                assert (err <= bound).all(), (b, i, h, float((err / bound).max()))
    return call, worst


SHAPES = [(1, 4, 64), (5, 8, 128), (9, 10, 128), (16, 8, 64), (11, 16, 128)]


@pytest.mark.parametrize("N,Hq,D", SHAPES)
@pytest.mark.parametrize("step", [4.0, 7.5, 8.5, 9.0, 12.0, 20.0])
def test_attention_maxima_that_rise_at_every_tile(N, Hq, D, step):
    # a tile's keys lie at the last tile's largest score, one of them `step` above: whenever the running maximum is
    # raised, the sums made before carry a good part of the answer
    def rising(C, at):
        x = [step * (t // 128) for t in range(C)]
        for t in range(at, C, 128):
            x[t] += step
        return x
    q_row = torch.exp2((torch.arange(N)[:, None] + torch.arange(Hq)[None]) % 3 - 1.0)
    run_whole(N, Hq, D, [rising(1500, 77), rising(130, 3), rising(max(N, 40), 5), rising(700, 127)], q_row, seed=60)


@pytest.mark.parametrize("N,Hq,D", SHAPES)
def test_attention_one_maximum_over_a_split_unit(N, Hq, D):
    # long sequences over many ranges, whose partials have maxima up to 60 powers of two apart
    g = gen(61)
    levels = [(torch.rand(30000, generator=g) * 4 + 56 * (torch.arange(30000) // 6000 == 3)).tolist(),
              (torch.rand(9000, generator=g) * 6).tolist()]
    q_row = torch.exp2((torch.arange(N)[:, None] + torch.arange(Hq)[None]) % 2 - 1.0)
    run_whole(N, Hq, D, levels, q_row, seed=62)


@pytest.mark.parametrize("N,Hq,D", SHAPES[1:])
def test_attention_rows_of_far_sizes(N, Hq, D):
    # a row's scores are its own: rows 2^80 apart in one unit, the large ones past 2^20 (one key, or equal ones, take
    # all weight), the small ones flat
    q_row = torch.exp2(torch.tensor([0.0, 40.0, -40.0, 1.0, 22.0])[torch.arange(N) % 5][:, None].expand(N, Hq))
    g = gen(63)
    levels = [(torch.rand(700, generator=g) * 8).tolist(), (torch.rand(max(N, 30), generator=g) * 8).tolist()]
    run_whole(N, Hq, D, levels, q_row, seed=64)


@pytest.mark.parametrize("N,Hq,D", SHAPES[1:])
@pytest.mark.parametrize("small", [2.0 ** -126, 2.0 ** -110, 2.0 ** -60, 1.0, 2.0 ** 10])
def test_attention_rows_beside_one_whose_scores_grow_past_2_20(N, Hq, D, small):
    # the first tile's scores are all 0, then one row's are huge: what the others have summed up under V's scales
    # of 2^4 to 2^8 stays
    q_row = torch.full((N, Hq), small)
    q_row[N // 2, 1] = 2.0 ** 30
    g = gen(66)
    levels = [[0.0] * 130 + (torch.rand(570, generator=g) * 8).tolist(), (torch.rand(max(N, 30), generator=g)).tolist()]
    run_whole(N, Hq, D, levels, q_row, seed=67, lo=4, hi=9)


@pytest.mark.parametrize("N,Hq,D", SHAPES[1:])
def test_attention_of_a_split_unit_in_two_parts_under_far_scales(N, Hq, D):
    # one row's scores pass 2^20, so that the unit's partials carry V's scales in their sums; of another row the largest
    # key, 2^200 above the rest, has V's smallest scale, and keys of the largest scale count as much
    C = 6000
    q_row = torch.ones((N, Hq))
    q_row[N // 2, 1] = 2.0 ** 25
    x = torch.rand(C, generator=gen(68)) * 6
    x[443] = 200

    def scales(kv, table):
        kv[2][..., 1] = 2.0 ** -100
        for p in range(C // 16):
            if p % 7 == 3 and p != 443 // 16:
                kv[2][table[0, p], :, 1] = 2.0 ** 99
    run_whole(N, Hq, D, [x.tolist()], q_row, seed=69, scales=scales)
