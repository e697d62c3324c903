"""The 8-bit KV cache's calls where they are easily wrong. What append and commit leave in memory is compared bit for
bit, the attention within bounds that follow from its documented roundings."""
import pytest
import torch

from test_gpu_kv_q8 import gen, run_append

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("how", ["block", "position"])
@pytest.mark.parametrize("D,Hkv", [(128, 2), (64, 5)])
def test_append_of_long_ragged_prompts_skips_pages_among_others(how, D, Hkv):
    # a CTA goes over four pages: of every four, one or two in the middle are skipped, in every pattern; rows of
    # unlike size, so that the halves of a page and its neighbours ask for different scales
    N, lens = 320, [320, 331, 325, 400, 322, 328]
    nl = torch.tensor([320, 320, 300, 257, 320, 311], dtype=torch.int32)
    starts = [c - int(n) for c, n in zip(lens, nl)]
    pos = torch.randint(0, 500, (len(lens), N), generator=gen(5), dtype=torch.int32) if how == "position" else None

    def spoil(qkv, pools, table, ctx, positions, nb):
        qkv.mul_(torch.exp2(torch.randint(-8, 9, (len(lens), N, 1, 1), generator=gen(6)).float()).to(torch.bfloat16))
        for b, (c, start) in enumerate(zip(lens, starts)):
            skip = [(1,), (2,), (1, 2), (0, 2), (1, 3), (3,)][b]
            for p in range(start // 16, (c - 1) // 16 + 1):
                if (p - start // 16) % 4 in skip:
                    if how == "block":
                        table[b, p] = -1 if p & 1 else nb + p
                    else:
                        positions[b, max(p * 16, start) - start + (p % 5 if p * 16 >= start else 0)] = -1 if p & 1 else 500
    run_append(True, len(lens), N, 4 if D == 128 else 5, Hkv, D, D, False, lens, seed=51, positions=pos,
               new_lens=nl, spoil=spoil, rows=500, fused=True)
