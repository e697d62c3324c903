"""Refusals of the append calls and the 8-bit cache's calls, and the argument helpers (no GPU): every error is
found on the host before any launch. Also pins the plain forms of tests/kv_reference.py."""
import math

import numpy as np
import pytest
import torch

import kv_reference as ref
import speculative_decoding_rl_b200 as sv

BASE = dict(num_seqs=2, num_q_rows=5, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
            max_blocks_per_seq=8, num_blocks=32)
Q, K, V, QO, TB, CL, ST, CS, KP, VP, SC = [0x1000000 * (i + 1) for i in range(11)]


def desc(**kw):
    return sv.SvAttnDesc(**{**BASE, **kw})


def append(q8=False, d=None, rope=None, rows=None, kv=None, table=TB, ctx=CL, q_out=QO, status=ST):
    d = d or desc()
    rope = rope or sv.SvRopeDesc(128, 0, 4096, CS)
    rows = rows or sv.SvNewRows(Q, K, V, 1024, 256, None, None)
    kv = kv or (sv.SvKVQ8(KP, VP, SC) if q8 else sv.SvKVLayer(KP, VP))
    (sv.sv_kv_append_q8 if q8 else sv.sv_kv_append)(d, rope, rows, kv, table, ctx, q_out, status, stream=0)


def refused(code, *a, **kw):
    with pytest.raises(sv.SvError) as e:
        append(*a, **kw)
    assert e.value.status == code, sv.sv_last_error()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-1), 1), (dict(num_seqs=65536), 1), (dict(num_q_rows=0), 1), (dict(num_q_rows=(1 << 20) + 1), 1),
    (dict(num_q_heads=0), 1), (dict(num_kv_heads=0), 1), (dict(num_kv_heads=65536), 1), (dict(head_dim=12), 2),
    (dict(head_dim=264), 2), (dict(block_size=32), 2), (dict(max_blocks_per_seq=0), 1), (dict(num_blocks=0), 1),
    (dict(max_blocks_per_seq=(1 << 26) + 1), 2),
])
def test_append_refuses_descriptors(q8, kw, status):
    refused(status, q8, d=desc(**kw))


def test_append_q8_takes_two_head_sizes():
    for D in (32, 96, 256):
        refused(2, True, d=desc(head_dim=D), rope=sv.SvRopeDesc(0, 0, 0, None))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("rope", [(8, 0, 64, CS), (144, 0, 64, CS), (-16, 0, 64, CS), (128, 2, 64, CS),
                                  (128, 0, 0, CS), (128, 0, 64, None), (128, 0, 64, CS + 4)])
def test_append_refuses_rotations(q8, rope):
    refused(2 if rope[0] in (8, 144, -16) else 1, q8, rope=sv.SvRopeDesc(*rope))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("rows", [
    (None, K, V, 1024, 256), (Q, None, V, 1024, 256), (Q, K, None, 1024, 256), (Q + 8, K, V, 1024, 256),
    (Q, K + 2, V, 1024, 256), (Q, K, V + 8, 1024, 256), (Q, K, V, 1016, 256), (Q, K, V, 1028, 256),
    (Q, K, V, 1024, 248), (Q, K, V, 1024, 260), (Q, K, V, -1024, 256), (Q, K, V, 1 << 41, 256),
])
def test_append_refuses_rows(q8, rows):
    refused(1, q8, rows=sv.SvNewRows(*rows, None, None))


@pytest.mark.parametrize("q8", [False, True])
def test_append_refuses_pointers(q8):
    for kw in (dict(table=None), dict(ctx=None), dict(q_out=None), dict(q_out=QO + 2), dict(table=TB + 2),
               dict(ctx=CL + 1), dict(status=ST + 2)):
        refused(1, q8, **kw)
    bad = [sv.SvKVQ8(None, VP, SC), sv.SvKVQ8(KP, VP, None), sv.SvKVQ8(KP, VP + 8, SC), sv.SvKVQ8(KP, VP, SC + 4)] \
        if q8 else [sv.SvKVLayer(None, VP), sv.SvKVLayer(KP + 8, VP)]
    for kv in bad:
        refused(1, q8, kv=kv)
    rows = sv.SvNewRows(Q, K, V, 1024, 256, 0x7001, None)
    refused(1, q8, rows=rows)


@pytest.mark.parametrize("q8", [False, True])
def test_append_refuses_outputs_over_inputs(q8):
    # q_out is 2*5*8*128 bf16 = 20480 bytes; in-place rotation of q is refused too
    for at in (Q, K, V, TB, CL, CS, Q + 20464):
        refused(1, q8, q_out=at)
        assert "overlap" in sv.sv_last_error()
    for at in (TB, CL + 4, K):
        refused(1, q8, status=at)
    refused(1, q8, status=QO + 64)


@pytest.mark.parametrize("q8", [False, True])
def test_append_refuses_a_cache_over_other_arguments(q8):
    pools = 32 * 2 * 16 * 128 * (1 if q8 else 2)
    for at in (Q, K, V, QO, TB, CL, ST, CS):
        for kv in ((at, VP, SC), (KP, at, SC), (KP, KP + pools - 16, SC)) + (((KP, VP, at),) if q8 else ()):
            refused(1, q8, kv=sv.SvKVQ8(*kv) if q8 else sv.SvKVLayer(*kv[:2]))
            assert "overlap" in sv.sv_last_error()


def test_append_with_no_sequences_is_a_no_op():
    for q8 in (False, True):
        append(q8, d=desc(num_seqs=0), rows=sv.SvNewRows(None, None, None, 0, 0, None, None), table=None, ctx=None,
               q_out=None, status=None, kv=sv.SvKVQ8(None, None, None) if q8 else sv.SvKVLayer(None, None))


@pytest.mark.parametrize("kw,status", [
    (dict(num_q_rows=0), 1), (dict(num_q_rows=65), 1), (dict(num_q_heads=6, num_kv_heads=4), 1),
    (dict(head_dim=96), 2), (dict(block_size=32), 2), (dict(num_seqs=-1), 1), (dict(num_seqs=513), 2),
    (dict(num_blocks=0), 1), (dict(num_q_heads=194, num_kv_heads=2), 2),
])
def test_attention_q8_refuses_descriptors(kw, status):
    d = desc(**kw)
    with pytest.raises(sv.SvError) as e:
        sv.sv_verify_attention_q8(d, Q, sv.SvKVQ8(KP, VP, SC), TB, CL, None, QO, 256, 1 << 20, stream=0)
    assert e.value.status == status
    assert sv.sv_verify_attention_q8_workspace_size(d) == 0


def test_attention_q8_refuses_pointers():
    good = dict(q=Q, kv=(KP, VP, SC), table=TB, ctx=CL, mask=None, out=QO, status=ST)
    for kw in (dict(q=None), dict(q=Q + 8), dict(kv=(None, VP, SC)), dict(kv=(KP, VP, None)),
               dict(kv=(KP + 8, VP, SC)), dict(kv=(KP, VP, SC + 4)), dict(table=None), dict(ctx=None),
               dict(out=None), dict(out=QO + 8), dict(mask=0x9004)):
        a = {**good, **kw}
        with pytest.raises(sv.SvError) as e:
            sv.sv_verify_attention_q8(desc(), a["q"], sv.SvKVQ8(*a["kv"]), a["table"], a["ctx"], a["mask"], a["out"],
                                      256, 1 << 20, a["status"], stream=0)
        assert e.value.status == 1
    sv.sv_verify_attention_q8(desc(num_seqs=0), None, sv.SvKVQ8(None, None, None), None, None, None, None, None, 0,
                              stream=0)


@pytest.mark.parametrize("kw,layers,status", [
    (dict(num_q_rows=0), 1, 1), (dict(num_q_rows=65), 1, 1), (dict(head_dim=96), 1, 2), (dict(block_size=32), 1, 2),
    (dict(num_kv_heads=0), 1, 1), (dict(num_blocks=0), 1, 1), ({}, 0, 1), ({}, 129, 1),
])
def test_commit_q8_refuses_arguments(kw, layers, status):
    with pytest.raises(sv.SvError) as e:
        sv.sv_kv_commit_q8(desc(**kw), [(KP, VP, SC)] * layers, TB, CL, Q, K, QO, stream=0)
    assert e.value.status == status


def test_commit_q8_refuses_pointers_and_aliases():
    base = dict(table=TB, ctx=CL, alen=Q, path=K, new=QO, status=ST)
    for layers, kw in [([(KP, VP + 8, SC)], {}), ([(KP, VP, SC + 4)], {}), ([(KP, VP, None)], {}),
                       ([(KP, VP, SC)], dict(table=None)), ([(KP, VP, SC)], dict(new=None)),
                       ([(KP, VP, SC)], dict(new=CL + 4)), ([(KP, VP, SC)], dict(status=Q)),
                       ([(KP, VP, SC)], dict(status=QO))]:
        a = {**base, **kw}
        with pytest.raises(sv.SvError) as e:
            sv.sv_kv_commit_q8(desc(), layers, a["table"], a["ctx"], a["alen"], a["path"], a["new"], a["status"],
                               stream=0)
        assert e.value.status == 1


def test_row_strides_of_fused_projections():
    qkv = torch.zeros((2, 3, 12, 64), dtype=torch.bfloat16)
    assert sv._row_stride(qkv[:, :, :8], "q") == sv._row_stride(qkv[:, :, 8:10], "k") == 12 * 64
    one = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16)
    assert sv._row_stride(one, "k") == 4 * 64
    assert sv._row_stride(qkv[:1, :1, :5], "k") == 5 * 64  # a single row's stride is not read
    for bad in (qkv[:, :, :, :32], qkv[:, :, ::2], qkv.transpose(1, 2), qkv[:, :2], qkv.float()):
        with pytest.raises(ValueError):
            sv.make_new_rows(None, bad, bad)
    k = qkv[:, :, 8:10]
    for kw in (dict(positions=torch.zeros((2, 3))), dict(positions=torch.zeros((3, 2), dtype=torch.int32)),
               dict(new_lens=torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            sv.make_new_rows(None, k, k, **kw)
    with pytest.raises(ValueError):
        sv.make_new_rows(qkv[:1, :, :8], k, k)
    with pytest.raises(ValueError):
        sv.make_rope_desc(torch.zeros((4, 64), dtype=torch.float64))
    with pytest.raises(ValueError):
        sv.make_kv_q8(one, one, one)
    assert sv.make_rope_desc(None).rotary_dim == 0


def test_attention_q8_refuses_outputs_over_inputs():
    ws, need = 0x100000000, 1 << 20
    for kw in (dict(out=Q), dict(out=Q + 20464), dict(out=KP), dict(ws=VP), dict(out=ws + 256), dict(status=CL + 4),
               dict(status=TB), dict(ws=0x100000000, out=0x100000000 + need - 16)):
        a = {**dict(out=QO, ws=ws, status=ST), **kw}
        with pytest.raises(sv.SvError) as e:
            sv.sv_verify_attention_q8(desc(), Q, sv.SvKVQ8(KP, VP, SC), TB, CL, None, a["out"], a["ws"], need,
                                      a["status"], stream=0)
        assert e.value.status == 1 and "overlap" in sv.sv_last_error()


def test_call_objects_refuse_other_layouts():
    from speculative_decoding_rl_b200.session import AppendCall, AppendQ8Call, AttentionQ8Call, CommitQ8Call
    B, N, Hq, Hkv, D, mb, nb = 2, 3, 4, 2, 64, 4, 9
    d = sv.SvAttnDesc(B, N, Hq, Hkv, D, 16, mb, nb)
    f8 = torch.float8_e4m3fn
    pool, sc = torch.zeros((nb, Hkv, 16, D)).to(f8), torch.zeros((nb, Hkv, 2))
    wide = torch.zeros((B, mb + 1), dtype=torch.int32)
    table, ctx = wide[:, :mb].contiguous(), torch.zeros(B, dtype=torch.int32)
    q = torch.zeros((B, N, Hq, D), dtype=torch.bfloat16)
    k = torch.zeros((B, N, Hkv, D), dtype=torch.bfloat16)
    mask = torch.zeros((B, N), dtype=torch.int64)
    kv, rope = (pool, pool, sc), sv.make_rope_desc(None)

    def bad(call):
        with pytest.raises(ValueError):
            call()
    for kv2 in ((pool, pool), (pool[:8], pool, sc), (pool, pool.float(), sc), (pool, pool, sc.double()),
                (pool, pool, sc[..., :1]), (pool.transpose(1, 2), pool, sc)):
        bad(lambda: AttentionQ8Call(d, kv2, table, ctx, q))
        bad(lambda: AppendQ8Call(d, rope, kv2, table, ctx, q, k, k))
        bad(lambda: CommitQ8Call(d, [kv, kv2], table, ctx, ctx, torch.zeros((B, N - 1), dtype=torch.int32)))
    for t2, c2 in ((wide[:, :mb], ctx), (table.long(), ctx), (table, ctx.long()), (table, ctx[:1])):
        bad(lambda: AttentionQ8Call(d, kv, t2, c2, q))
        bad(lambda: AppendQ8Call(d, rope, kv, t2, c2, q, k, k))
        bad(lambda: AppendCall(d, rope, (k, k), t2, c2, q, k, k))
    bad(lambda: AttentionQ8Call(d, kv, table, ctx, q.float()))
    bad(lambda: AttentionQ8Call(d, kv, table, ctx, q.transpose(1, 2)))
    bad(lambda: AttentionQ8Call(d, kv, table, ctx, q, mask.int()))
    bad(lambda: AttentionQ8Call(d, kv, table, ctx, q, out=q[:, :2]))
    bad(lambda: AppendQ8Call(d, rope, kv, table, ctx, None, k, k, q_out=q))
    bad(lambda: AppendQ8Call(d, rope, kv, table, ctx, q, k, k[:, :2]))
    bad(lambda: CommitQ8Call(d, [kv], table, ctx, ctx, torch.zeros((B, N), dtype=torch.int32)))
    bad(lambda: AttentionQ8Call(d, kv, table, ctx, q))  # all well but the device


# ------------------------------------------------------------------ the plain forms themselves
def test_page_exponent_is_the_smallest_that_holds():
    rng = np.random.default_rng(1)
    for x in list(rng.lognormal(0, 20, 200)) + [448.0, 448.0 * (1 + 2 ** -23), 224.0, 1e-35, 3e38]:
        x = float(np.float32(x))
        e = ref.page_exponent(x)
        assert -100 <= e <= 119
        assert x <= 448 * 2.0 ** e or e == 119
        assert e == -100 or x > 448 * 2.0 ** (e - 1)
    assert 448 * 2.0 ** 119 >= torch.finfo(torch.bfloat16).max / 2 ** 0.9


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotations_agree(interleaved):
    g = torch.Generator().manual_seed(2)
    x = torch.randn((7, 3, 64), generator=g).to(torch.bfloat16)
    cs = ref.cos_sin(7, 32)
    y32 = ref.rotate32(x, cs, interleaved)
    y64, mag = ref.rotate64(x, cs, interleaved)
    assert ((y32.double() - y64).abs() <= 3 * 2.0 ** -24 * mag).all()
    assert torch.equal(y32[..., 32:], x[..., 32:].float())


def test_attend64_matches_softmax():
    g = torch.Generator().manual_seed(3)
    rng = np.random.default_rng(3)
    lens = [37, 3]
    t, nb = ref.table_for(lens, 4, rng)
    kv = ref.q8_pools(nb, 2, 64, g)
    q = torch.randn((2, 3, 4, 64), generator=g).to(torch.bfloat16)
    out, tol = ref.attend64(q, kv, t, lens)
    for b, C in enumerate(lens):
        for hq in range(4):
            k = torch.stack([kv[0][t[b, u // 16], hq // 2, u % 16].double() * kv[2][t[b, u // 16], hq // 2, 0]
                             for u in range(C)])
            v = torch.stack([kv[1][t[b, u // 16], hq // 2, u % 16].double() * kv[2][t[b, u // 16], hq // 2, 1]
                             for u in range(C)])
            for i in range(3):
                n = C - 3 + i + 1
                w = torch.softmax(q[b, i, hq].double() @ k[:n].T / math.sqrt(64), 0)
                assert torch.allclose(w @ v[:n], out[b, i, hq], rtol=1e-12, atol=1e-14)
    assert (tol > 0).all()
