"""Plain CPU forms of the rotated append and the 8-bit KV cache's calls.

Writes are emulated rounding by rounding, so what a call leaves in memory has
to match bit for bit; `rotate64` and `attend64` are the formulas in 64 bits.
"""
import math

import numpy as np
import torch

PAGE = 16


def rotate32(x, cs, interleaved):
    """x bf16 [n][H][D], cs fp32 [n][R]: every product and sum rounded once to fp32 (elementwise CPU operations
    do not contract)."""
    y = x.float().clone()
    R = cs.shape[1]
    c, s = cs[:, None, :R // 2], cs[:, None, R // 2:]
    a, b = (y[..., 0:R:2].clone(), y[..., 1:R:2].clone()) if interleaved else \
        (y[..., :R // 2].clone(), y[..., R // 2:R].clone())
    ac, bs, bc, as_ = a * c, b * s, b * c, a * s
    lo, hi = ac - bs, bc + as_
    if interleaved:
        y[..., 0:R:2], y[..., 1:R:2] = lo, hi
    else:
        y[..., :R // 2], y[..., R // 2:R] = lo, hi
    return y


def rotate64(x, cs, interleaved):
    """The same by complex numbers in 64 bits, and the sum of the products' magnitudes."""
    y = x.double().clone()
    mag = y.abs()
    R = cs.shape[1]
    z = torch.complex(cs[:, :R // 2].double(), cs[:, R // 2:].double())[:, None]
    first = list(range(0, R, 2)) if interleaved else list(range(R // 2))
    second = [j + 1 for j in first] if interleaved else [j + R // 2 for j in first]
    a, b = y[..., first], y[..., second]
    w = torch.complex(a, b) * z
    y[..., first], y[..., second] = w.real, w.imag
    mag[..., first] = (a * z.real).abs() + (b * z.imag).abs()
    mag[..., second] = (b * z.real).abs() + (a * z.imag).abs()
    return y, mag


def page_exponent(top: float) -> int:
    """Smallest e in [-100, 119] with top <= 448 * 2^e."""
    if top == 0:
        return -100
    m, x = math.frexp(top)          # top = m * 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    return max(-100, min(119, x - 9 if m <= 0.875 else x - 8))


def store_page(pool, scales, blk, h, which, val):
    """val fp32 [rows][D]: the rows kept, written under their power of two."""
    fin = val[torch.isfinite(val)]
    e = page_exponent(float(fin.abs().max()) if fin.numel() else 0.0)
    x = torch.where(torch.isfinite(val), val.double() * 2.0 ** -e, torch.full_like(val, math.nan).double())
    pool[blk, h, :val.shape[0]] = x.float().to(torch.float8_e4m3fn)
    scales[blk, h, which] = 2.0 ** e


def load_row(pool, scales, blk, h, which, r):
    return pool[blk, h, r].float() * scales[blk, h, which]


def append(q, k, v, cs, interleaved, pools, table, ctx, q_out, positions=None, new_lens=None, R=None):
    """Emulates sv_kv_append (pools: (k, v)) and sv_kv_append_q8 (pools: (k, v, scales)) in place. Returns flags."""
    B, N, Hkv, D = k.shape
    mb, nb = table.shape[1], pools[0].shape[0]
    R = (0 if cs is None else cs.shape[1]) if R is None else R
    flags = []
    for b in range(B):
        C, n = int(ctx[b]), N if new_lens is None else int(new_lens[b])
        if n < 0 or n > N or C < n or C > mb * PAGE:
            flags.append(2)
            continue
        f = 0
        start = C - n
        pos = [start + i if positions is None else int(positions[b, i]) for i in range(n)]
        bad_row = [R > 0 and not 0 <= t < cs.shape[0] for t in pos]
        if any(bad_row):
            f |= 2
        if n:
            cst = None if R == 0 else cs[torch.tensor([t if not bad else 0 for t, bad in zip(pos, bad_row)])]
            rot = (lambda x: x.float()) if R == 0 else (lambda x: rotate32(x, cst, interleaved))
            rk, rv = rot(k[b, :n]), v[b, :n].float()
            rq = None if q is None else rot(q[b, :n])
            for p in range(start // PAGE, (C - 1) // PAGE + 1):
                lo, hi = max(p * PAGE, start), min(p * PAGE + PAGE, C)
                blk = int(table[b, p])
                if not 0 <= blk < nb:
                    f |= 8
                    continue
                if any(bad_row[lo - start:hi - start]):
                    continue
                if q is not None:
                    q_out[b, lo - start:hi - start] = rq[lo - start:hi - start].to(torch.bfloat16)
                for which, rows in ((0, rk), (1, rv)):
                    new = rows[lo - start:hi - start]
                    for h in range(Hkv):
                        if len(pools) == 2:
                            pools[which][blk, h, lo - p * PAGE:hi - p * PAGE] = new[:, h].to(torch.bfloat16)
                        else:
                            old = [load_row(pools[which], pools[2], blk, h, which, r) for r in range(lo - p * PAGE)]
                            store_page(pools[which], pools[2], blk, h, which, torch.stack(old + list(new[:, h])))
        flags.append(f)
    return flags


def commit_q8(layers, table, ctx, alen, path, N):
    """Emulates sv_kv_commit_q8 in place; returns (new lengths, flags)."""
    mb, nb = table.shape[1], layers[0][0].shape[0]
    new_ctx, flags = [], []
    for b in range(len(ctx)):
        C, a = int(ctx[b]), int(alen[b])
        f = 0
        if C < N or C > mb * PAGE:
            f |= 2
        elif any(not 0 <= int(table[b, p]) < nb for p in range((C - N) // PAGE, (C - 1) // PAGE + 1)):
            f |= 8
        nodes = [int(x) for x in path[b, :a]] if 0 <= a <= N - 1 else None
        if nodes is None or any(not p < x <= N - 1 for p, x in zip([0] + nodes, nodes)):
            f |= 32
        flags.append(f)
        new_ctx.append(C if f else C - N + 1 + a)
        if f or nodes == list(range(1, a + 1)):
            continue
        root = C - N
        k0 = next(j for j in range(a) if nodes[j] != j + 1)
        src = {t: t for t in range(root + 1 + k0)}
        src.update({root + 1 + j: root + nodes[j] for j in range(k0, a)})
        for pools in layers:
            old = [x.clone() for x in pools]
            for p in range((root + 1 + k0) // PAGE, (root + a) // PAGE + 1):
                ts = range(p * PAGE, min(p * PAGE + PAGE, root + a + 1))
                for which in (0, 1):
                    for h in range(pools[0].shape[1]):
                        rows = [load_row(old[which], old[2], int(table[b, src[t] // PAGE]), h, which, src[t] % PAGE)
                                for t in ts]
                        store_page(pools[which], pools[2], int(table[b, p]), h, which, torch.stack(rows))
    return new_ctx, flags


def attend64(q, kv, table, ctx, mask=None):
    """Verify attention over the 8-bit cache in 64 bits. Returns (out, tol): tol bounds what the call's documented
    roundings can move each entry by.

    With w the softmax weights, A = sum w |v|: each weight enters the product with V rounded to at least 9 bits
    (2^-9 of itself; half a step of a 3 x 3-bit expansion), or, where it is so small that the pieces' exponents end,
    to half of e5m2's smallest step, 2^-17, on a scale on which the row's largest weight times V's scale is at least
    2^7: 2^-24 of that largest. Its exponential adds 2^-20, and a score off by d moves it by e^d - 1, and the sum it is
    divided by likewise: 2 (e^d - 1) in all. The score is a sum of D products, exact in fp32 but for its additions
    (D roundings of at most 2^-23 of the sum of the magnitudes, an extra bit for adders that cut off), of q held in two
    4-bit pieces on a scale on which its row's largest entry is above 224: off by at most half of e4m3's smallest step,
    2^-10, which is less than 2^-17 of that entry. The output is rounded to bf16 (2^-8 of itself)."""
    k_pool, v_pool, scales = kv
    B, N, Hq, D = q.shape
    Hkv, nb = k_pool.shape[1], k_pool.shape[0]
    out, tol = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for b in range(B):
        C = int(ctx[b])
        if C < N or C > table.shape[1] * PAGE:
            continue
        blk = table[b, :-(-C // PAGE)].long()
        good = (blk >= 0) & (blk < nb)
        at = torch.where(good, blk, torch.zeros_like(blk))
        sc = scales[at].double().clamp(min=2.0 ** -100)
        ok = good[:, None, None, None]

        def whole(pool, which):
            x = pool[at].float().double() * sc[..., which, None, None]
            return torch.where(ok, x, torch.zeros_like(x)).transpose(0, 1).reshape(Hkv, -1, D)[:, :C]

        k, v = whole(k_pool, 0), whole(v_pool, 1)
        seen = torch.ones((N, C), dtype=torch.bool)
        for i in range(N):
            for j in range(N):
                bit = j <= i if mask is None else bool((int(mask[b, i]) >> j) & 1)
                seen[i, C - N + j] = bit
        for hq in range(Hq):
            h = hq // (Hq // Hkv)
            qd = q[b, :, hq].double()
            s = (qd @ k[h].T) / math.sqrt(D)
            s = torch.where(seen, s, torch.full_like(s, -math.inf))
            m = s.amax(1, keepdim=True)
            w = torch.where(seen, torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m)),
                            torch.zeros_like(s))
            tot = w.sum(1, keepdim=True)
            w = torch.where(tot > 0, w / tot, w)
            if torch.isnan(v[h]).any():
                vv = torch.where(seen[..., None], v[h][None], torch.zeros((), dtype=torch.float64))
                o, A = torch.einsum("nt,ntd->nd", w, vv), torch.einsum("nt,ntd->nd", w, vv.abs())
            else:
                o, A = w @ v[h], w @ v[h].abs()
            kk = k[h].abs().nan_to_num(0.0)
            d = ((qd.abs() @ kk.T) * D * 2.0 ** -22 +
                 qd.abs().amax(1, keepdim=True) * kk.sum(-1) * 2.0 ** -17) / math.sqrt(D)
            d = torch.where(seen, d, torch.zeros_like(d))
            d = d.amax(1, keepdim=True)
            # the floor of a weight, in the units of the e4m3 values it multiplies
            sv = torch.where(good[:, None], sc[:, h, 1:], torch.ones_like(sc[:, h, 1:])).repeat(1, PAGE).reshape(-1)[:C]
            v8 = (v[h] / sv[:, None]).abs().nan_to_num(0.0)
            floor = 2.0 ** -24 * (w * sv).amax(1, keepdim=True) * (seen.double() @ v8)
            out[b, :, hq] = o
            tol[b, :, hq] = 2.0 ** -8 * o.abs() + (2.0 ** -9 + 2.0 ** -20 + 2 * torch.expm1(d)) * A * 1.01 + floor + 1e-37
    return out, tol


# ------------------------------------------------------------------ inputs
def table_for(lens, mb, rng, spare=2):
    """Block table [B][mb] over a random permutation; unused entries point at a spare block."""
    need = [-(-c // PAGE) for c in lens]
    nb = sum(need) + spare
    perm = rng.permutation(nb)
    t = np.full((len(lens), mb), perm[-1], dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(t), nb


def q8_pools(nb, Hkv, D, g, lo=-8, hi=-3):
    """Pools with entries over the format's whole range under powers of two."""
    def pool():
        return (torch.randn((nb, Hkv, PAGE, D), generator=g) * 64).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return pool(), pool(), torch.exp2(torch.randint(lo, hi, (nb, Hkv, 2), generator=g).float())


def cos_sin(rows, R, theta=1e4):
    freq = theta ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()
