// sv_verify_attention_q8: GQA attention of every active sequence's N draft
// query rows over its paged 8-bit KV cache (e4m3 pages, one scale each for K
// and V of a KV head), split over the context and combined.
//
// Units, tiles, schedule, partials and the combine kernel are the bf16 cache's
// (sv_attention.cu). The stream of K and V bounds the call; it is half the bf16
// cache's, so nothing may be spent on widening it: K and V go from HBM through
// shared memory into the tensor cores as the 8-bit values they are
// (kind::f8f6f4), and the other operand of each product is cut into 8-bit
// pieces whose sum holds it:
//   S^T = K Q^T  q, scaled by a power of two of its row, is the sum of two e4m3
//                values: bf16 has 8 significant bits, e4m3 four, so the sum is
//                exact down to 2^-18 of the row's largest entry. Two products
//                over the same K accumulate into S.
//   O^T = V^T P  the weights p, rounded to fp16, are cut into three e5m2 values
//                (3 significant bits each, fp16's own exponent range): at least
//                9 bits, 2^-9 of the weight, down to 2^-17 of the running
//                maximum and 2^-29 of the maximum below, so that a long flat
//                tail under one large weight keeps its mass. One product takes
//                the pieces side by side (N = 3 x rows) and the epilogue adds
//                the three sums.
// A key is a lane of the softmax warps, so a page's scales are one factor per
// thread: K's joins the exponent, V's the weight before it is cut.
//
// Inside a CTA (tcgen05 + TMA, one persistent CTA per SM):
//   warps 0 .. MATH_WARPS-1  softmax warpgroups, as in the bf16 kernel; at the
//                start they also cut the first unit's query rows;
//   WARP_K, WARP_V  TMA producers: per tile, 8 boxes of one page each;
//   WARP_MMA     TMEM allocator and MMA issuer;
//   WARP_ST      status flags; then the V ring: rows past ctx_len and NaN of new
//                keys (a row of a draft tree must not meet what its mask hides)
//                are zeroed before a tile goes to its product;
//   WARP_Q       query pieces of the units to come, and the pages' scales, four
//                tiles at a time, for the softmax.
#include <string.h>

#include "sv_page8.cuh"
#include "sv_q8.h"
#include "sv_schedule.cuh"

namespace sv {

using namespace tc;

namespace {

// Softmax warpgroups as in the bf16 kernel: each owns q8_cw(RP) row columns.
__host__ __device__ constexpr int q8_cw(int RP) { return RP == 96 ? 32 : 16; }
__host__ __device__ constexpr int q8_nwg(int RP) { return RP / q8_cw(RP); }
__host__ __device__ constexpr int q8_threads(int RP) { return 32 * (4 * q8_nwg(RP) + 5); }

constexpr int SC_BATCH = 4;    // tiles whose page scales are fetched together
constexpr int SC_RING = 4;     // batches in shared memory
constexpr int PAGES_TILE = TILE_KEYS / PAGE;
constexpr int UNIT_RING = 32;  // units whose NaN mark is kept
// Units whose row scales are kept. Unit u is cut once unit u - 2 is through
// Q.K; the softmax has then loaded S of unit u - 4 at least, may still be using
// that unit's scales, and is past unit u - 5: five are enough.
constexpr int QS_RING = 8;
constexpr int MAX_RING = 8;    // K or V slots at most
// p is held as p * 2^P_SHIFT / (V's scale): the running maximum's weight is
// 2^12, a raise waits until one passes 2^(12 + RESCALE_LOG2), below fp16's and
// e5m2's largest values, and fp16's smallest step is 2^-36 of the maximum.
constexpr float P_SCALE = 4096.f, P_UNSCALE = 1.f / 4096.f;
constexpr float RESCALE_LOG2 = 3.f;

struct Q8Layout {
    uint32_t tile_bytes, off_k, off_q, q_bytes, off_p, p_bytes, off_bar, off_tp, off_cl, off_red, off_ms, off_as,
        off_lred, off_rowi, off_umask, off_vote, off_fin, off_mfin, off_qs, off_sc, off_vnan, off_misc, total;
};

__host__ __device__ constexpr int q8_barriers(int RP, int NK, int NV) {
    return 2 * NK + 3 * NV + 2 * 2 /*q*/ + 2 * 2 /*s*/ + 2 /*p*/ + 2 * 2 /*o*/ + 1 /*done*/ + q8_nwg(RP) +
           2 * SC_RING;
}

__host__ __device__ inline Q8Layout q8_layout(int D, int RP, int NK, int NV, int B) {
    Q8Layout L;
    const int NWG = q8_nwg(RP), CW = q8_cw(RP);
    L.tile_bytes = (uint32_t)TILE_KEYS * D;
    L.off_k = NV * L.tile_bytes;
    L.off_q = L.off_k + NK * L.tile_bytes;
    L.q_bytes = 2u * RP * D;  // two pieces
    L.off_p = L.off_q + 2 * L.q_bytes;
    L.p_bytes = 3u * RP * TILE_KEYS;  // three pieces
    L.off_bar = L.off_p + 2 * L.p_bytes;
    L.off_tp = L.off_bar + 8u * q8_barriers(RP, NK, NV);
    L.off_cl = L.off_tp + 4u * (B + 1);
    L.off_red = (L.off_cl + 4u * B + 15u) & ~15u;
    L.off_ms = L.off_red + 4u * 2 * NWG * 4 * CW;   // [par][wg][warp][CW] tile column maxima
    L.off_as = L.off_ms + 4u * 2 * RP;              // [par][RP] running maxima
    L.off_lred = L.off_as + 4u * 2 * RP;            // [par][RP] rescale factors
    L.off_rowi = L.off_lred + 4u * NWG * 4 * CW;    // [wg][warp][CW] row-sum partials
    L.off_umask = (L.off_rowi + 4u * RP + 15u) & ~15u;
    L.off_vote = L.off_umask + 8u * NWG * 64;       // [wg][64] mask words of the unit
    L.off_fin = L.off_vote + 4u * 2 * NWG * 4;      // [par][wg][warp] rescale votes
    L.off_mfin = L.off_fin + 4u * RP;               // [RP] row sums of a finished unit
    L.off_qs = (L.off_mfin + 4u * RP + 15u) & ~15u;
    L.off_sc = L.off_qs + 4u * QS_RING * RP;        // [QS_RING][RP] query row scales
    L.off_vnan = L.off_sc + 8u * SC_RING * SC_BATCH * PAGES_TILE;  // page scales (K, V)
    L.off_misc = L.off_vnan + 4u * UNIT_RING;
    L.total = L.off_misc + 16u + 4u * 32;
    return L;
}

struct Q8Params {
    CUtensorMap tm_k;
    CUtensorMap tm_v;
    AttnParams a;
    const float2 *scales;
    int NK, NV, Nc;
};

// Cuts row r of a unit's queries into two e4m3 pieces in shared memory (128- or
// 64-byte swizzled rows of D bytes, the second piece's RP rows after the
// first's) and writes the row's scale; one warp. A row with an entry that is
// not finite gets the scale NaN, and with it NaN outputs.
template <int D, int RP>
SV_DEV void cut_query_row(const uint16_t *src, uint8_t *qbuf, float *qs, int r, int lane) {
    constexpr int E = D / 32;  // entries per lane
    float x[E];
    if constexpr (E == 4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(src) + lane);
        x[0] = __uint_as_float(w.x << 16); x[1] = __uint_as_float(w.x & 0xFFFF0000u);
        x[2] = __uint_as_float(w.y << 16); x[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(src) + lane);
        x[0] = __uint_as_float(w << 16); x[1] = __uint_as_float(w & 0xFFFF0000u);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xffffffffu, top);
    const bool finite = top < 0x7F800000u;
    // |x| <= 448 * 2^e. e stays where 2^-e and 2^e are normal.
    const int ex = (int)(top >> 23) - 127;
    const int e = max(-126, (top & 0x7FFFFFu) <= 0x600000u ? ex - 8 : ex - 7);
    const float inv = exp2_int(-e);
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        const float a = finite ? x[i] * inv : 0.f, b = finite ? x[i + 1] * inv : 0.f;
        const uint32_t h = float2_to_e4m3x2(a, b);
        const float2 back = e4m3x2_to_float2(h);
        hi |= h << (8 * i);
        lo |= float2_to_e4m3x2(a - back.x, b - back.y) << (8 * i);
    }
    const int at = lane * E;  // byte of the row
    const int sw = D == 128 ? r & 7 : (r >> 1) & 3;
    uint8_t *dst = qbuf + r * D + (((at >> 4) ^ sw) << 4) + (at & 15);
    if constexpr (E == 4) {
        *reinterpret_cast<uint32_t *>(dst) = hi;
        *reinterpret_cast<uint32_t *>(dst + RP * D) = lo;
    } else {
        *reinterpret_cast<uint16_t *>(dst) = (uint16_t)hi;
        *reinterpret_cast<uint16_t *>(dst + RP * D) = (uint16_t)lo;
    }
    if (lane == 0) qs[r] = finite ? exp2_int(e) : NAN;
}

// fp16 pairs of four weights -> the bytes of their first 3-bit pieces (cut off
// or, for the last piece, rounded); h is left with the remainders.
SV_DEV uint32_t cut_piece(uint32_t *h, bool last) {
    if (last) {
        // half of the e5m2 step added to the magnitude: rounds to nearest
        return __byte_perm(h[0] + 0x00800080u, h[1] + 0x00800080u, 0x7531);
    }
    const uint32_t bytes = __byte_perm(h[0], h[1], 0x7531);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t t = h[i] & 0xFF00FF00u;
        const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&h[i]), *reinterpret_cast<const __half2 *>(&t));
        h[i] = *reinterpret_cast<const uint32_t *>(&d);
    }
    return bytes;
}

template <int D, int RP>
__global__ void __launch_bounds__(q8_threads(RP), 1) attn_q8_kernel(const __grid_constant__ Q8Params P) {
    constexpr int NWG = q8_nwg(RP);
    constexpr int CW = q8_cw(RP);
    constexpr int MATH_WARPS = 4 * NWG;
    constexpr int NTHREADS = q8_threads(RP);
    constexpr int WARP_K = MATH_WARPS, WARP_MMA = MATH_WARPS + 1, WARP_V = MATH_WARPS + 2, WARP_ST = MATH_WARPS + 3,
                  WARP_Q = MATH_WARPS + 4;
    // The three pieces side by side in one product's N while two O buffers of
    // that width fit TMEM beside S (and N = 288 is past a product's 256); for 96
    // rows the pieces go one after the other into the same columns.
    constexpr bool SIDE = RP <= 64;
    constexpr int ON = SIDE ? 3 * RP : RP;           // columns of an O buffer
    constexpr int S_COLS = (RP + 31) / 32 * 32;      // TMEM columns per S buffer
    constexpr int O_COLS = (ON + 31) / 32 * 32;      // and per O buffer
    constexpr int TM_O = 2 * S_COLS;
    static_assert(TM_O + 2 * O_COLS <= 512, "TMEM");
    constexpr int SW = D == 128 ? 2 : 4;             // swizzle of K, V and Q rows
    constexpr uint32_t PIECE = 16u * TILE_KEYS;      // bytes of one piece of 16 columns
    const AttnParams &p = P.a;
    const int NK = P.NK, NV = P.NV;
    auto qphase = [](int u) -> uint32_t { return (u >> 1) & 1; };

    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const Q8Layout L = q8_layout(D, RP, NK, NV, p.B);
    uint64_t *bar = reinterpret_cast<uint64_t *>(base + L.off_bar);
    uint64_t *k_full = bar, *k_empty = bar + NK;
    uint64_t *v_full = bar + 2 * NK, *v_empty = v_full + NV, *vz = v_empty + NV;
    uint64_t *q_full = vz + NV, *q_empty = q_full + 2;
    uint64_t *s_full = q_empty + 2, *s_empty = s_full + 2;
    uint64_t *p_full = s_empty + 2;
    uint64_t *o_full = p_full + 2;     // [2] by tile parity: the tile's PV has completed, its P buffer is free
    uint64_t *o_free = o_full + 2;     // [2] by unit parity: the unit's O buffer has been read out
    uint64_t *sc_full = o_free + 2, *sc_empty = sc_full + SC_RING;
    uint64_t *done_bar = sc_empty + SC_RING;
    uint64_t *wg_bar = done_bar + 1;
    int *TP = reinterpret_cast<int *>(base + L.off_tp);
    int *CL = reinterpret_cast<int *>(base + L.off_cl);
    float *red = reinterpret_cast<float *>(base + L.off_red);
    float *mS = reinterpret_cast<float *>(base + L.off_ms);
    float *aS = reinterpret_cast<float *>(base + L.off_as);
    float *lred = reinterpret_cast<float *>(base + L.off_lred);
    int *rowi = reinterpret_cast<int *>(base + L.off_rowi);
    uint64_t *umask = reinterpret_cast<uint64_t *>(base + L.off_umask);
    int *vote = reinterpret_cast<int *>(base + L.off_vote);
    float *lfin = reinterpret_cast<float *>(base + L.off_fin);
    float *mfin = reinterpret_cast<float *>(base + L.off_mfin);
    float *qs = reinterpret_cast<float *>(base + L.off_qs);
    float2 *scr = reinterpret_cast<float2 *>(base + L.off_sc);
    int *vnan = reinterpret_cast<int *>(base + L.off_vnan);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + L.off_misc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(base + L.off_misc + 4);
    int *scratch = reinterpret_cast<int *>(base + L.off_misc + 16);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < NK; ++s) { mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], 1); }
        for (int s = 0; s < NV; ++s) { mbar_init(&v_full[s], 1); mbar_init(&v_empty[s], 1); mbar_init(&vz[s], 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], MATH_WARPS); mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], MATH_WARPS);
            mbar_init(&p_full[i], MATH_WARPS);
            mbar_init(&o_full[i], 1); mbar_init(&o_free[i], MATH_WARPS);
        }
        for (int i = 0; i < SC_RING; ++i) { mbar_init(&sc_full[i], 1); mbar_init(&sc_empty[i], MATH_WARPS); }
        mbar_init(done_bar, 1);
        for (int g = 0; g < NWG; ++g) mbar_init(&wg_bar[g], 4);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == WARP_MMA) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == WARP_K && lane == 0) {
        tma_prefetch_desc(&P.tm_k);
        tma_prefetch_desc(&P.tm_v);
    }
    for (int r = tid; r < RP; r += NTHREADS) {
        rowi[r] = r / p.G;
        for (int i = 0; i < QS_RING; ++i) qs[i * RP + r] = 1.f;
    }
    {  // zero both query buffers: rows past a unit's real rows stay zero
        uint4 *q4 = reinterpret_cast<uint4 *>(base + L.off_q);
        for (uint32_t e = tid; e < 2 * L.q_bytes / 16u; e += NTHREADS) q4[e] = make_uint4(0, 0, 0, 0);
    }
    griddep_wait();  // no input is read, and nothing written, before this wait
    griddep_launch_dependents();
    tile_prefix(p, TP, scratch, CL);  // contains __syncthreads
    const int ups = p.Hkv * p.RC;
    const int total = ups * TP[p.B];
    const int W = total > 0 ? (total + p.num_ctas - 1) / p.num_ctas : 1;
    if (tid == 0) {
        const int v0 = min((int)blockIdx.x * W, total), v1 = min(v0 + W, total);
        int n;
        const TileInfo t0 = cta_tiles(TP, p.B, ups, v0, v1, &n);
        scratch[0] = t0.b; scratch[1] = t0.hr; scratch[2] = t0.j; scratch[3] = t0.Tb; scratch[4] = n;
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const TileInfo t_first{scratch[0], scratch[1], scratch[2], scratch[3]};
    const int ntiles = scratch[4];

    // query rows of tile ti's unit, the CTA's u-th, every `step`-th from `r0` on
    auto cut_queries = [&](const TileInfo &ti, int u, int r0, int step) {
        const int h = ti.hr / p.RC, rc = ti.hr - h * p.RC;
        const int rows = min(p.rows_unit, p.R - rc * p.rows_unit);
        const uint16_t *q = p.q + (((size_t)ti.b * p.N + rc * P.Nc) * p.Hq + h * p.G) * D;
#pragma unroll 4
        for (int r = r0; r < rows; r += step) {
            const int i = rowi[r];
            cut_query_row<D, RP>(q + ((size_t)i * p.Hq + (r - i * p.G)) * D, base + L.off_q + (u & 1) * L.q_bytes,
                                 qs + u % QS_RING * RP, r, lane);
        }
    };

    if (warp == WARP_K || warp == WARP_V) {
        // ------------------------- TMA producers --------------------------
        if (lane == 0) {
            const bool is_k = warp == WARP_K;
            const int NR = is_k ? NK : NV;
            uint64_t *full = is_k ? k_full : v_full;
            uint64_t *empty = is_k ? k_empty : v_empty;
            const CUtensorMap *tm = is_k ? &P.tm_k : &P.tm_v;
            uint8_t *ring = base + (is_k ? L.off_k : 0u);
            int issued_tiles = 0, rs = 0;
            uint32_t rph = 0;
            TileInfo ti = t_first;
            for (int lt = 0; lt < ntiles; ++lt, next_tile(ti, TP, p.B, ups)) {
                const int h = ti.hr / p.RC;
                const int C = CL[ti.b];
                int blks[PAGES_TILE];
#pragma unroll
                for (int pg = 0; pg < PAGES_TILE; ++pg) {
                    const int page = ti.j * PAGES_TILE + pg;
                    blks[pg] = page * PAGE < C ? __ldg(p.block_table + (size_t)ti.b * p.max_blocks + page) : -1;
                }
                const int s = rs;
                if (!mbar_wait(&empty[s], rph ^ 1u, abort_flag, p.wait_limit_ns)) break;
                if (++rs == NR) { rs = 0; rph ^= 1u; }
                mbar_arrive_expect_tx(&full[s], L.tile_bytes);
                uint8_t *dst = ring + s * L.tile_bytes;
#pragma unroll
                for (int pg = 0; pg < PAGES_TILE; ++pg) {
                    // out of range (or past ctx_len): a coordinate past the pool, which the TMA unit fills with zeros
                    const int blk = (blks[pg] >= 0 && blks[pg] < p.num_blocks) ? blks[pg] : p.num_blocks;
                    tma_load_4d(dst + pg * (PAGE * D), tm, &full[s], 0, 0, h, blk);
                }
                issued_tiles = lt + 1;
            }
            if (*abort_flag)  // this CTA's own copies land before it can exit
                for (int lt = max(0, issued_tiles - NR); lt < issued_tiles; ++lt)
                    mbar_wait_time(&full[lt % NR], (lt / NR) & 1, WAIT_LIMIT_NS);
        }
    } else if (warp == WARP_ST) {
        // ---------------- per-sequence status (and invalid sequences) ----------------
        for (int b = blockIdx.x; b < p.B; b += p.num_ctas) {
            const int C = CL[b];
            const bool ctx_ok = C >= p.N && C <= p.max_blocks * PAGE;
            int bad = 0;
            if (ctx_ok) {
                for (int jb = lane; jb < (C + PAGE - 1) / PAGE; jb += 32) {
                    const int blk = __ldg(p.block_table + (size_t)b * p.max_blocks + jb);
                    bad |= (blk < 0 || blk >= p.num_blocks);
                }
            } else {
                uint4 *o4 = reinterpret_cast<uint4 *>(p.out + (size_t)b * p.N * p.Hq * D);
                for (int e = lane; e < p.N * p.Hq * D / 8; e += 32) o4[e] = make_uint4(0, 0, 0, 0);
            }
            bad = __any_sync(0xffffffffu, bad);
            if (p.status && lane == 0)
                p.status[b] = (ctx_ok ? 0 : SV_FLAG_BAD_CONTEXT) | (bad ? SV_FLAG_BAD_BLOCK : 0);
        }
        // ------------------- V rows past ctx_len, NaN of new keys -------------------
        // 0 * NaN is NaN: rows past ctx_len hold whatever the pool holds, and a new
        // key that some rows must not see may hold NaN. Both are zeroed here once
        // the tile has landed. Where NaN was zeroed the unit is marked, and its
        // read-out puts it back for the rows that see the key.
        TileInfo ti = t_first;
        int vs = 0, u = -1;
        uint32_t vph = 0;
        for (int lt = 0; lt < ntiles; ++lt, next_tile(ti, TP, p.B, ups)) {
            const int s = vs;
            const uint32_t par = vph;
            if (++vs == NV) { vs = 0; vph ^= 1u; }
            if (lt == 0 || ti.j == 0) {
                ++u;
                // the ring outlasts the units between this warp and the read-out
                if (lane == 0) vnan[u % UNIT_RING] = 0;
            }
            const bool landed = mbar_test(&v_full[s], par) || mbar_wait(&v_full[s], par, abort_flag, p.wait_limit_ns);
            if (!__all_sync(0xffffffffu, landed)) break;
            const int C = CL[ti.b];
            // keys of the tile from the first new one on, and from ctx_len on
            // (pages wholly past ctx_len were loaded as zeros by the TMA unit)
            const int kn = max(0, C - p.N - ti.j * TILE_KEYS), k0 = max(0, C - ti.j * TILE_KEYS);
            const int k1 = min(TILE_KEYS, (k0 + PAGE - 1) / PAGE * PAGE);
            if (kn < k1) {
                uint8_t *vt = base + s * L.tile_bytes;
                bool hit = false;
                for (int e = kn * (D / 16) + lane; e < k1 * (D / 16); e += 32) {
                    uint4 *at = reinterpret_cast<uint4 *>(vt) + e;
                    if (e >= k0 * (D / 16)) {
                        *at = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    uint4 w = *at;
                    uint32_t *wp = reinterpret_cast<uint32_t *>(&w);
                    uint32_t any = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // 0xFF in each byte that is NaN (all but the sign set)
                        const uint32_t is = __vcmpeq4(wp[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                        any |= is;
                        wp[i] &= ~is;
                    }
                    if (any) {
                        *at = w;
                        hit = true;
                    }
                }
                if (__any_sync(0xffffffffu, hit) && lane == 0) vnan[u % UNIT_RING] = 1;
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&vz[s]);
        }
    } else if (warp == WARP_Q) {
        // ------------- query pieces and page scales, ahead of their use -------------
        TileInfo ti = t_first;
        int u = -1, batch = 0;
        bool ok = true;
        for (int lt = 0; lt < ntiles && ok; ++lt, next_tile(ti, TP, p.B, ups)) {
            if (lt % SC_BATCH == 0) {
                // tile lt + lane / 8, page lane % 8 of it
                TileInfo w = ti, mine = ti;
#pragma unroll
                for (int j = 1; j < SC_BATCH; ++j) {
                    next_tile(w, TP, p.B, ups);
                    if (lane / PAGES_TILE >= j) mine = w;
                }
                const int page = mine.j * PAGES_TILE + lane % PAGES_TILE;
                float2 sc = make_float2(1.f, 1.f);
                if (lt + lane / PAGES_TILE < ntiles && page * PAGE < CL[mine.b]) {
                    const int blk = __ldg(p.block_table + (size_t)mine.b * p.max_blocks + page);
                    if (blk >= 0 && blk < p.num_blocks) {
                        sc = __ldg(P.scales + (size_t)blk * p.Hkv + mine.hr / p.RC);
                        sc.x = fmaxf(sc.x, PAGE8_SCALE_MIN);
                        sc.y = fmaxf(sc.y, PAGE8_SCALE_MIN);
                    }
                }
                const int slot = batch % SC_RING;
                const bool free = mbar_test(&sc_empty[slot], (batch / SC_RING & 1) ^ 1) ||
                                  mbar_wait(&sc_empty[slot], (batch / SC_RING & 1) ^ 1, abort_flag, p.wait_limit_ns);
                if (!(ok = __all_sync(0xffffffffu, free))) break;
                scr[slot * 32 + lane] = sc;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_full[slot]);
                ++batch;
            }
            if (lt == 0 || ti.j == 0) {
                ++u;
                if (u == 0) continue;  // the softmax warps cut the first unit's rows
                const bool free = mbar_test(&q_empty[u & 1], qphase(u) ^ 1) ||
                                  mbar_wait(&q_empty[u & 1], qphase(u) ^ 1, abort_flag, p.wait_limit_ns);
                if (!(ok = __all_sync(0xffffffffu, free))) break;
                cut_queries(ti, u, 0, 1);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_n(&q_full[u & 1], MATH_WARPS);
            }
        }
    } else if (warp == WARP_MMA) {
        // -------------------------- MMA issuer ----------------------------
        // Polls both queues and issues whichever product is ready, as in the bf16 kernel.
        if (lane == 0) {
            constexpr uint32_t idq = idesc_f8(128, RP, 0, 0, false, false);
            constexpr uint32_t idp = idesc_f8(128, ON, 0, 1, true, true);
            int nq = 0, np = 0, lu = -1, lup = -1;
            int ks = 0, vs = 0;
            uint32_t kph = 0, vph = 0;
            const uint64_t kdesc = smem_desc(smem_u32(base + L.off_k), 16, 8 * D, SW);
            const uint64_t qdesc = smem_desc(smem_u32(base + L.off_q), 16, 8 * D, SW);
            // D = 64: dims 64..127 of the 128-row product read bytes of other keys and are not read out
            const uint64_t vdesc = smem_desc(smem_u32(base), 8 * D, 8 * D, SW);
            const uint64_t pdesc = smem_desc(smem_u32(base + L.off_p), 128, SIDE ? PIECE : 3 * PIECE, 0);
            TileInfo tq = t_first;
            TileInfo tp = tq;
            uint32_t idle = 0;
            uint64_t idle_since = 0;
            while (np < ntiles) {
                bool progressed = false;
                if (nq < ntiles) {
                    const bool newu = (nq == 0 || tq.j == 0);
                    const int lu_n = newu ? lu + 1 : lu;
                    const int sb = nq & 1;
                    if ((!newu || mbar_test(&q_full[lu_n & 1], qphase(lu_n))) && mbar_test(&k_full[ks], kph) &&
                        mbar_test(&s_empty[sb], ((nq >> 1) & 1) ^ 1)) {
                        lu = lu_n;
                        tc_fence_after();
                        const uint64_t ka = kdesc + ((ks * L.tile_bytes) >> 4);
                        const uint64_t qa = qdesc + (((lu & 1) * L.q_bytes) >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 32; ++kk)
#pragma unroll
                            for (int piece = 0; piece < 2; ++piece)
                                mma_f8_ss(tmem + sb * S_COLS, ka + ((kk * 32) >> 4),
                                          qa + ((piece * RP * D + kk * 32) >> 4), idq, kk + piece > 0);
                        mma_commit(&s_full[sb]);
                        mma_commit(&k_empty[ks]);
                        if (nq == ntiles - 1 || tq.j == tq.Tb - 1) mma_commit(&q_empty[lu & 1]);
                        if (++ks == NK) { ks = 0; kph ^= 1u; }
                        ++nq;
                        if (nq < ntiles) next_tile(tq, TP, p.B, ups);
                        progressed = true;
                    }
                }
                if (np < nq) {
                    const bool newu = (np == 0 || tp.j == 0);
                    const int lup_n = newu ? lup + 1 : lup;
                    const int pb = np & 1, ob = lup_n & 1;
                    if (mbar_test(&p_full[pb], (np >> 1) & 1) && mbar_test(&vz[vs], vph) &&
                        (!newu || mbar_test(&o_free[ob], ((lup_n >> 1) & 1) ^ 1))) {
                        lup = lup_n;
                        tc_fence_after();
                        const uint64_t va = vdesc + ((vs * L.tile_bytes) >> 4);
                        const uint64_t pa = pdesc + ((pb * L.p_bytes) >> 4);
                        constexpr int NPROD = SIDE ? 1 : 3;
#pragma unroll
                        for (int kk = 0; kk < TILE_KEYS / 32; ++kk)
#pragma unroll
                            for (int piece = 0; piece < NPROD; ++piece)
                                mma_f8_ss(tmem + TM_O + ob * O_COLS, va + ((kk * 32 * D) >> 4),
                                          pa + ((piece * PIECE + kk * 512) >> 4), idp,
                                          (kk + piece > 0 || !newu) ? 1u : 0u);
                        mma_commit(&o_full[pb]);
                        mma_commit(&v_empty[vs]);
                        if (++vs == NV) { vs = 0; vph ^= 1u; }
                        ++np;
                        if (np < ntiles) next_tile(tp, TP, p.B, ups);
                        progressed = true;
                    }
                }
                if (progressed) {
                    idle = 0;
                } else if (++idle > 8 && (__nanosleep(20), (idle & 63) == 0)) {
                    if (*abort_flag) break;
                    const uint64_t now = globaltimer_ns();
                    if (idle == 64) idle_since = now;
                    else if (now - idle_since > p.wait_limit_ns) { *abort_flag = 1; break; }
                }
            }
            mma_commit(done_bar);  // every MMA of this CTA has finished before TMEM is freed
            mbar_wait_time(done_bar, 0, WAIT_LIMIT_NS);
        }
    } else {
        // ------------------------------ softmax ------------------------------
        const int wg = warp >> 2;          // warpgroup: owns row columns [wg*CW, wg*CW + CW)
        const int wiw = warp & 3;          // warp within the warpgroup = TMEM lane quadrant
        const int ell = wiw * 32 + lane;   // key (S) / head dim (O) lane
        const int col0 = wg * CW;
        uint32_t wg_phase = 0;
        const uint32_t lane_base = tmem + ((uint32_t)(wiw * 32) << 16);
        float lsum[CW];
#pragma unroll
        for (int c = 0; c < CW; ++c) lsum[c] = 0.f;
        const size_t slot_floats = slot_stride(p.rows_unit, D);
        bool ok = true;

        int cur_u = -1, last_par = 0, lu = -1;
        int ub = 0, uh = 0, urc = 0, uC = 0, urows = 0;

        auto warp_arrive = [&](uint64_t *b) {
            __syncwarp();
            if (lane == 0) mbar_arrive(b);
        };
        auto wait_w = [&](uint64_t *b, uint32_t parity) -> bool {
            const bool r = mbar_test(b, parity) || mbar_wait(b, parity, abort_flag, p.wait_limit_ns);
            return __all_sync(0xffffffffu, r);
        };
        auto wg_sync = [&]() -> bool {
            warp_arrive(&wg_bar[wg]);
            const bool r = wait_w(&wg_bar[wg], wg_phase);
            wg_phase ^= 1;
            return r;
        };

        if (ntiles > 0) {
            cut_queries(t_first, 0, warp, MATH_WARPS);
            fence_proxy_async_smem();
            warp_arrive(&q_full[0]);
        }

        // Unit ends as in the bf16 kernel: close_unit reduces the row sums,
        // finish_unit reads O out once the next unit's first tile is through softmax.
        bool pending = false;
        int pend_u = 0, pend_lu = 0, pend_jt = 0;
        auto close_unit = [&](int jt_last) -> bool {
#pragma unroll
            for (int c = 0; c < CW; ++c) {
                const float v = warp_sum(lsum[c]);
                if (lane == 0) lred[(wg * 4 + wiw) * CW + c] = v;
                lsum[c] = 0.f;
            }
            if (!wg_sync()) return false;
            if (wiw == 0 && lane < CW) {
                float l = 0.f;
                for (int w = 0; w < 4; ++w) l += lred[(wg * 4 + w) * CW + lane];
                lfin[col0 + lane] = l;
                mfin[col0 + lane] = mS[last_par * RP + col0 + lane];
            }
            if (!wg_sync()) return false;
            pending = true;
            pend_u = cur_u;
            pend_lu = lu;
            pend_jt = jt_last;
            return true;
        };
        auto finish_unit = [&]() -> bool {
            pending = false;
            if (!wait_w(&o_full[pend_jt & 1], (pend_jt >> 1) & 1)) return false;
            tc_fence_after();
            const int fb = pend_u / ups, fhr = pend_u - fb * ups;
            const int fh = fhr / p.RC, frc = fhr - fh * p.RC;
            const int frows = min(p.rows_unit, p.R - frc * p.rows_unit);
            const int Tb = real_tiles(TP[fb + 1] - TP[fb]);
            const int tpre = ups * TP[fb] + fhr * (Tb + UNIT_COST);  // the unit's first position
            const int first_cta = tpre / W;
            const int nseg = (tpre + Tb - 1) / W - first_cta + 1;
            const bool to_slot = nseg > 1;
            const bool marked = vnan[pend_lu % UNIT_RING] != 0;
            float *slot = p.ws_partial + (size_t)(pend_u + blockIdx.x) * slot_floats;
#pragma unroll 1
            for (int c0 = 0; c0 < CW; c0 += 16) {
                float o[16];
                const uint32_t oaddr = lane_base + TM_O + (pend_lu & 1) * O_COLS + (col0 + c0) * (SIDE ? 3 : 1);
                tmem_ld16(oaddr, o);
                if constexpr (SIDE) {
                    float o1[16], o2[16];
                    tmem_ld16(oaddr + 16, o1);
                    tmem_ld16(oaddr + 32, o2);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] = (o[c] + (o1[c] + o2[c])) * P_UNSCALE;
                } else {
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] *= P_UNSCALE;
                }
                if (ell >= D) continue;
                if (marked) {
                    // NaN among the new keys' V, zeroed for the product: back to the rows that see the key
#pragma unroll 1
                    for (int n = 0; n < p.N; ++n) {
                        const int t = CL[fb] - p.N + n;
                        const int blk = __ldg(p.block_table + (size_t)fb * p.max_blocks + t / PAGE);
                        if (blk < 0 || blk >= p.num_blocks) continue;
                        const uint8_t *vp = reinterpret_cast<const uint8_t *>(p.v_pool) +
                                            (((size_t)blk * p.Hkv + fh) * PAGE + t % PAGE) * D;
                        if ((vp[ell] & 0x7F) != 0x7F) continue;
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const int i = frc * P.Nc + rowi[col0 + c0 + c];
                            if (col0 + c0 + c < frows &&
                                (p.mask ? (__ldg(p.mask + (size_t)fb * p.N + i) >> n & 1) != 0 : n <= i))
                                o[c] = NAN;
                        }
                    }
                }
                if (!to_slot) {
                    uint16_t *orow = p.out + (((size_t)fb * p.N + frc * P.Nc) * p.Hq + fh * p.G) * D + ell;
                    const size_t hqd = (size_t)p.Hq * D;
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const int r = col0 + c0 + c;
                        if (r < frows) {
                            const int i = rowi[r];
                            const float l = lfin[r];
                            const __nv_bfloat16 v = __float2bfloat16_rn(l > 0.f || l != l ? __fdividef(o[c], l) : 0.f);
                            orow[i * hqd + (size_t)(r - i * p.G) * D] = *reinterpret_cast<const uint16_t *>(&v);
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (col0 + c0 + c < frows) slot[(size_t)(col0 + c0 + c) * D + ell] = o[c];
                }
            }
            tc_fence_before();
            warp_arrive(&o_free[pend_lu & 1]);
            if (to_slot && wiw == 0 && lane < CW && col0 + lane < frows) {
                slot[(size_t)p.rows_unit * D + col0 + lane] = mfin[col0 + lane];
                slot[(size_t)p.rows_unit * D + p.rows_unit + col0 + lane] = lfin[col0 + lane];
            }
            return true;
        };

        // one pass past the last tile closes and finishes the CTA's last unit
        TileInfo tnext = t_first;
        for (int lt = 0; lt <= ntiles && ok; ++lt) {
            const bool end = lt == ntiles;
            const TileInfo ti = end ? TileInfo{0, 0, 0, 1} : tnext;
            if (!end) next_tile(tnext, TP, p.B, ups);
            const bool first = (lt == 0 || ti.j == 0 || end);
            if (first) {
                if (lt > 0 && !(ok = close_unit(lt - 1))) break;
                if (end) {
                    if (pending) ok = finish_unit();
                    break;
                }
                ++lu;
                cur_u = ti.b * ups + ti.hr;
                ub = ti.b;
                uh = ti.hr / p.RC;
                urc = ti.hr - uh * p.RC;
                uC = CL[ub];
                urows = min(p.rows_unit, p.R - urc * p.rows_unit);
                if (p.mask) {
                    for (int k = wiw * 32 + lane; k < p.N; k += 128)
                        umask[wg * 64 + k] = __ldg(p.mask + (size_t)ub * p.N + k);
                    if (!(ok = wg_sync())) break;
                }
            }
            const int sb = lt & 1, par = lt & 1;
            // the page's scales: K's in the exponent's unit, V's
            const int batch = lt / SC_BATCH;
            if (!(ok = wait_w(&sc_full[batch % SC_RING], batch / SC_RING & 1))) break;
            const float2 scl = scr[(batch % SC_RING) * 32 + lt % SC_BATCH * PAGES_TILE + ell / PAGE];
            if (lt % SC_BATCH == SC_BATCH - 1) warp_arrive(&sc_empty[batch % SC_RING]);
            const float ksc = scl.x * p.scale_log2, vsc = scl.y * P_SCALE, lv = __log2f(scl.y);
            if (!(ok = wait_w(&s_full[sb], (lt >> 1) & 1))) break;
            tc_fence_after();
            float sv[CW];
            tmem_ld_cols<CW>(lane_base + sb * S_COLS + col0, sv);
            tmem_wait_ld();
            tc_fence_before();
            warp_arrive(&s_empty[sb]);

            const int key = ti.j * TILE_KEYS + ell;
            const bool valid = key < uC;
            const int newk = key - (uC - p.N);
#pragma unroll
            for (int c = 0; c < CW; ++c) sv[c] *= ksc;
            if (__any_sync(0xffffffffu, !valid || newk >= 0)) {
                // tile holds keys past ctx_len or new (masked) keys: per-element visibility
                const int ibase = urc * P.Nc;
#pragma unroll
                for (int c = 0; c < CW; ++c) {
                    bool vis = valid;
                    if (valid && newk >= 0 && col0 + c < urows) {
                        const int i = ibase + rowi[col0 + c];
                        vis = p.mask ? ((umask[wg * 64 + i] >> newk) & 1ull) != 0 : newk <= i;
                    }
                    if (!vis) sv[c] = -INFINITY;
                }
            }

            // x = s * qs is the exponent (log2 units, without the maximum); the
            // running maximum is of x + log2(V's scale), the weight that enters
            // the product with V. It is raised only when one passes it by
            // 2^RESCALE_LOG2, by a vote of the warpgroup, as in the bf16 kernel.
            const float4 *qs4 = reinterpret_cast<const float4 *>(qs + lu % QS_RING * RP + col0);
            const float4 *mo4 = reinterpret_cast<const float4 *>(mS + (par ^ 1) * RP + col0);
            bool need = first;
            if (!first) {
                const float thr = RESCALE_LOG2 - lv;
#pragma unroll
                for (int c4 = 0; c4 < CW / 4; ++c4) {
                    const float4 m4 = mo4[c4], q4 = qs4[c4];
                    need |= fmaf(sv[c4 * 4 + 0], q4.x, -m4.x) > thr;
                    need |= fmaf(sv[c4 * 4 + 1], q4.y, -m4.y) > thr;
                    need |= fmaf(sv[c4 * 4 + 2], q4.z, -m4.z) > thr;
                    need |= fmaf(sv[c4 * 4 + 3], q4.w, -m4.w) > thr;
                }
            }
            const bool wneed = __any_sync(0xffffffffu, need);
            if (lane == 0) vote[(par * NWG + wg) * 4 + wiw] = wneed;
            if (!(ok = wg_sync())) break;
            const int *vt = vote + (par * NWG + wg) * 4;
            const bool rescale = (vt[0] | vt[1] | vt[2] | vt[3]) != 0;
            if (rescale) {
                float *rd = red + ((par * NWG + wg) * 4 + wiw) * CW;
                const float *qr = qs + lu % QS_RING * RP + col0;
#pragma unroll
                for (int c = 0; c < CW; ++c) {
                    float m;
                    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(fmaf(sv[c], qr[c], lv)));
                    if (lane == c) rd[c] = m;
                }
                if (!(ok = wg_sync())) break;
                if (wiw == 0 && lane < CW) {
                    const int c = lane;
                    const float m_old = first ? M_NONE : mS[(par ^ 1) * RP + col0 + c];
                    float rmax = -INFINITY;
                    for (int w = 0; w < 4; ++w) rmax = fmaxf(rmax, red[((par * NWG + wg) * 4 + w) * CW + c]);
                    const float mx = fmaxf(m_old, rmax);  // stays M_NONE while nothing is visible
                    mS[par * RP + col0 + c] = mx;
                    aS[par * RP + col0 + c] = ex2_approx(m_old - mx);  // M_NONE - finite underflows to 0
                }
                if (!(ok = wg_sync())) break;
                {
                    const float4 *an4 = reinterpret_cast<const float4 *>(aS + par * RP + col0);
#pragma unroll
                    for (int c4 = 0; c4 < CW / 4; ++c4) {
                        const float4 a4 = an4[c4];
                        lsum[c4 * 4 + 0] *= a4.x;
                        lsum[c4 * 4 + 1] *= a4.y;
                        lsum[c4 * 4 + 2] *= a4.z;
                        lsum[c4 * 4 + 3] *= a4.w;
                    }
                }
                if (!first) {
                    // scale the unit's O^T columns once the previous tile's PV has landed
                    if (!(ok = wait_w(&o_full[(lt - 1) & 1], ((lt - 1) >> 1) & 1))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < CW; c0 += 16) {
#pragma unroll 1
                        for (int piece = 0; piece < (SIDE ? 3 : 1); ++piece) {
                            float o[16];
                            const uint32_t oaddr = lane_base + TM_O + (lu & 1) * O_COLS +
                                                   (col0 + c0) * (SIDE ? 3 : 1) + piece * 16;
                            tmem_ld16(oaddr, o);
                            tmem_wait_ld();
                            const float4 *a4p = reinterpret_cast<const float4 *>(aS + par * RP + col0 + c0);
#pragma unroll
                            for (int c4 = 0; c4 < 4; ++c4) {
                                const float4 a4 = a4p[c4];
                                o[c4 * 4 + 0] *= a4.x;
                                o[c4 * 4 + 1] *= a4.y;
                                o[c4 * 4 + 2] *= a4.z;
                                o[c4 * 4 + 3] *= a4.w;
                            }
                            tmem_st16(oaddr, o);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
            } else if (wiw == 0 && lane < CW) {
                // keep the maxima: readers of these slots are past the next tile's vote sync
                mS[par * RP + col0 + lane] = mS[(par ^ 1) * RP + col0 + lane];
            }
            last_par = par;
            const float4 *ms4 = reinterpret_cast<const float4 *>(mS + (rescale ? par : par ^ 1) * RP + col0);
            if (!(ok = wait_w(&o_full[sb], ((lt >> 1) & 1) ^ 1))) break;  // P buffer sb is free
            uint8_t *pbuf = base + L.off_p + sb * L.p_bytes + ell * 16;
#pragma unroll
            for (int c16 = 0; c16 < CW; c16 += 16) {
                uint32_t piece[3][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c4 = c16 / 4 + k;
                    const float4 m4 = ms4[c4], q4 = qs4[c4];
                    const float mm[4] = {m4.x, m4.y, m4.z, m4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
                    float pp[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = c4 * 4 + i;
                        const float w = ex2_approx(fmaf(sv[c], qq[i], -mm[i]));
                        lsum[c] += w;
                        pp[i] = w * vsc;
                    }
                    const __half2 h0 = __floats2half2_rn(pp[0], pp[1]), h1 = __floats2half2_rn(pp[2], pp[3]);
                    uint32_t h[2] = {*reinterpret_cast<const uint32_t *>(&h0), *reinterpret_cast<const uint32_t *>(&h1)};
                    piece[0][k] = cut_piece(h, false);
                    piece[1][k] = cut_piece(h, false);
                    piece[2][k] = cut_piece(h, true);
                }
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    *reinterpret_cast<uint4 *>(pbuf + ((col0 + c16) / 16 * 3 + j) * PIECE) =
                        make_uint4(piece[j][0], piece[j][1], piece[j][2], piece[j][3]);
            }
            fence_proxy_async_smem();
            warp_arrive(&p_full[sb]);
            // the previous unit's last PV was issued before this tile's
            if (pending && !(ok = finish_unit())) break;
        }
    }

    // ----------------------------- teardown -------------------------------
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && p.status)
        for (int b = tid; b < p.B; b += NTHREADS) atomicOr(p.status + b, SV_FLAG_TIMEOUT);
    if (warp == WARP_MMA) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Map of an e4m3 pool [num_blocks][Hkv][16][D]: boxes of one head's page,
// swizzled by rows of D bytes.
bool encode_pool_q8(CUtensorMap *m, const void *pool, int num_blocks, int Hkv, int D) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)PAGE, (cuuint64_t)Hkv, (cuuint64_t)num_blocks};
    const cuuint64_t strides[3] = {(cuuint64_t)D, (cuuint64_t)PAGE * D, (cuuint64_t)Hkv * PAGE * D};
    const cuuint32_t box[4] = {(cuuint32_t)D, PAGE, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(pool), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int RP>
cudaError_t launch_q8(Q8Params &P, cudaStream_t stream) {
    // as many K and V slots as fit, V's the larger half (its slots are held longer)
    int NK = MAX_RING, NV = MAX_RING;
    while (q8_layout(D, RP, NK, NV, P.a.B).total + 1024 > (uint32_t)SMEM_LIMIT) {
        if (NK >= NV) --NK; else --NV;
        if (NK < 2) return cudaErrorInvalidConfiguration;
    }
    P.NK = NK;
    P.NV = NV;
    const size_t smem = q8_layout(D, RP, NK, NV, P.a.B).total + 1024;
    auto kfn = attn_q8_kernel<D, RP>;
    cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_programmatic(kfn, dim3(P.a.num_ctas), dim3(q8_threads(RP)), smem, stream, P);
}

template <int D>
cudaError_t launch_q8_rp(Q8Params &P, int RP, cudaStream_t stream) {
    switch (RP) {
        case 16: return launch_q8<D, 16>(P, stream);
        case 32: return launch_q8<D, 32>(P, stream);
        case 48: return launch_q8<D, 48>(P, stream);
        case 64: return launch_q8<D, 64>(P, stream);
        case 96: return launch_q8<D, 96>(P, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

size_t attention_q8_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int num_ctas) {
    return attention_workspace_bytes(B, N, Hq, Hkv, D, num_ctas);
}

cudaError_t launch_attention_q8(const AttnParams &p, const float *scales, cudaStream_t stream) {
    Q8Params P;
    memset(&P, 0, sizeof P);
    P.a = p;
    P.scales = reinterpret_cast<const float2 *>(scales);
    int RU, RC;
    row_chunks(p.N, p.G, &RU, &RC, &P.Nc);
    if (!encode_pool_q8(&P.tm_k, p.k_pool, p.num_blocks, p.Hkv, p.D) ||
        !encode_pool_q8(&P.tm_v, p.v_pool, p.num_blocks, p.Hkv, p.D))
        return cudaErrorInvalidValue;
    const int RP = RU > 64 ? 96 : (RU + 15) / 16 * 16;
    cudaError_t e = p.D == 128 ? launch_q8_rp<128>(P, RP, stream) : launch_q8_rp<64>(P, RP, stream);
    return e != cudaSuccess ? e : launch_combine(p, stream);
}

}  // namespace sv
