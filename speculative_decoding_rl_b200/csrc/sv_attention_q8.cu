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
//                exact down to 2^-17 of the row's largest entry. Two products
//                over the same K accumulate into S.
//   O^T = V^T P  the weights p, rounded to fp16, are cut into three e5m2 values
//                (3 significant bits each, fp16's own exponent range): at least
//                9 bits, 2^-9 of the weight, down to 2^-15 of the running
//                maximum and 2^-24 of the maximum below, so that a long flat
//                tail under one large weight keeps its mass. One product takes
//                the pieces side by side (N = 3 x rows) and the epilogue adds
//                the three sums.
// A key is a lane of the softmax warps, so a page's scales are one factor per
// thread: K's joins the exponent, V's the weight before it is cut.
//
// What the stream leaves per tile is less than the softmax's chain (scores out
// of TMEM, vote, exponentials, cut, back to shared memory) takes, so a CTA works
// on NT tiles at once: it stands for NT work ranges of the schedule, each with
// its own warps, rings, S, P and O. Code is kept short as well, since warps in
// different places of a long loop wait for instructions: columns are taken 16 at
// a time in rolled loops, and what they carry from tile to tile, the row sums,
// stays in TMEM beside S.
//
// Inside a CTA (tcgen05 + TMA, one persistent CTA per SM), for each range:
//   softmax      NG warpgroups of CW row columns; a thread is one key of the
//                tile. They also cut their units' query rows;
//   WARP_LD      TMA producer of K and V: per tile, 8 boxes of one page each;
//   WARP_MMA     MMA issuer;
//   WARP_AUX     status flags; the V ring: rows past ctx_len and NaN of new keys
//                (a row of a draft tree must not meet what its mask hides) are
//                zeroed before a tile goes to its product; the pages' scales.
//
// Measured at D = 128: 64 sequences of 512 to 32768 tokens, 45 rows a unit (1.05
// GB) 255 us in short runs (4.1 TB/s; the loads alone would take 160 us), of which
// a range's tile takes 1.9 us and a unit's start and end 7 us; 16 trees of 88 rows
// over 24576 tokens (0.41 GB) 173 us; 294 and 183 us one after the other under the
// power cap. What bounds it is the softmax's chain of 3580 warp instructions a tile,
// two tiles in flight: no unit is full (issue 49 %, memory 50 %, tensor unit 49 %).
#include <string.h>

#include <type_traits>

#include "../../include/specverify_testing.h"
#include "sv_page8.cuh"
#include "sv_q8.h"
#include "sv_schedule.cuh"

namespace sv {

using namespace tc;

namespace {

// Shape of the kernel for RP padded rows per unit. Two ranges everywhere but at 96
// rows, whose sums fill TMEM: three took 1.1 to 1.5 times as long (fewer registers
// a thread), one left the chain of a tile exposed (64 sequences: 786 us). As many
// columns to a warpgroup as keep its loop within 128 registers: 24 in place of 48
// measured the same, 16 took 1.3 to 2 times as long; 64 rows (32 sequences of 512 to
// 16384 tokens, 8 rows of 32/4 heads) take 66 us in one warpgroup, 85 in two of 32
// columns, whose 704 threads leave 80 registers, and 76 in two of a single range.
constexpr int CH = 16;  // columns taken at a time
template <int RP>
struct Q8Shape {
    static constexpr int CW = RP > 64 ? 32 : RP;               // row columns per warpgroup
    static constexpr int NG = RP / CW;                         // warpgroups per range
    static_assert(CW % CH == 0, "whole chunks of columns");
    static constexpr int NT = RP == 96 ? 1 : 2;                // ranges
    // O accumulators side by side: P's pieces enter a product's N together as far
    // as TMEM has room for their sums, the last one goes into the last sum.
    static constexpr int ACC = RP == 64 ? 1 : RP >= 48 ? 2 : 3;
    static constexpr int SB = 2;                  // S buffers per range
    static constexpr int PB = NT == 1 ? 2 : 1;    // P buffers per range
    static constexpr int NQ = RP == 64 ? 1 : 2;   // query buffers per range
    static constexpr int TM_S = (ACC * RP + 31) / 32 * 32;    // of a range's TMEM columns: O, S, row sums
    static constexpr int TM_L = TM_S + SB * RP;
    static constexpr int R_COLS = 512 / NT / 32 * 32;
    static_assert(TM_L + RP <= R_COLS, "TMEM");
    static constexpr int WGS = NT * NG;
    static constexpr int MATH_WARPS = 4 * WGS;
    static constexpr int THREADS = 32 * (MATH_WARPS + 3 * NT);
};

constexpr int UC = UNIT_COST_Q8;
constexpr int SC_BATCH = 4;    // tiles whose page scales are fetched together
constexpr int SC_RING = 4;     // batches of a range in shared memory
constexpr int PAGES_TILE = TILE_KEYS / PAGE;
constexpr int UNIT_RING = 32;  // units of a range whose NaN mark is kept
// Units whose row scales are kept: the warpgroups of a range cut unit u + 1
// while the slower one may still use the scales of unit u - 1.
constexpr int QS_RING = 4;
constexpr int MAX_RING = 16;   // K and V slots of a range at most
// p is held as p * P_SCALE * (V's scale): the running maximum's weight is 2^7, a
// raise waits until one passes P_MAX = 2^15, below fp16's and e5m2's largest
// values; half of e5m2's smallest step is 2^-24 of the maximum.
constexpr float P_SCALE = 128.f, P_UNSCALE = 1.f / 128.f, P_MAX = 32768.f;
// A maximum is of score + log2(V's scale). From here on a score's spacing (2^-3)
// would round that sum, and past 2^28 lose the scale or overshoot by more than the
// weights have room for: the maximum is then kept in two parts, hi + lo, hi the
// largest score alone and lo the largest (score - hi) + log2(V's scale), neither
// of which rounds. Such a unit is rare: its tiles' scores are rewritten as
// score - hi, so that the pass that makes the weights is the same.
constexpr float TWO_PARTS_FROM = 1048576.f;
// A range is at least this long: on small calls, shorter ranges would cost the
// combine more partials than they save (one sequence of 6151 tokens: 17.4 us at 2,
// 16.7 at 4, 18.5 at 6).
constexpr int MIN_WIDTH = 4;

struct Q8Layout {
    uint32_t tile_bytes, off_k, off_q, q_bytes, off_p, p_bytes, off_bar, off_tp, off_cl, off_red, off_nm, off_as,
        off_rowi, off_rowoff, off_umask, off_nh, off_qs, off_sc, off_vnan, off_misc, total;
};

template <int D, int RP>
__host__ __device__ inline Q8Layout q8_layout(int NK, int NV, int B) {
    using S = Q8Shape<RP>;
    Q8Layout L;
    L.tile_bytes = (uint32_t)TILE_KEYS * D;
    L.off_k = S::NT * NV * L.tile_bytes;           // [range][NV]
    L.off_q = L.off_k + S::NT * NK * L.tile_bytes; // [range][NK]
    L.q_bytes = 2u * RP * D;                       // [range][NQ]: two pieces
    L.off_p = L.off_q + S::NT * S::NQ * L.q_bytes;
    L.p_bytes = 3u * RP * TILE_KEYS;               // [range][PB]: three pieces
    L.off_bar = L.off_p + S::NT * S::PB * L.p_bytes;
    const int nbar = S::NT * (2 * NK + 3 * NV + S::NQ + 2 * S::SB + 2 * S::PB + 1 + 2 * SC_RING);
    L.off_tp = L.off_bar + 8u * nbar;
    L.off_cl = L.off_tp + 4u * (B + 1);
    L.off_red = (L.off_cl + 4u * B + 15u) & ~15u;
    L.off_nm = L.off_red + 4u * 4 * S::NT * RP;    // [range][warp][RP] tile column maxima, or row sums
    L.off_as = L.off_nm + 4u * S::NT * RP;         // [range][RP] running maxima (or second parts), negated
    L.off_rowi = L.off_as + 4u * S::NT * RP;       // [range][RP] roots of the rescale factors
    L.off_rowoff = (L.off_rowi + 4u * RP + 15u) & ~15u;
    L.off_umask = L.off_rowoff + 4u * RP;
    L.off_nh = L.off_umask + 8u * S::WGS * 64;     // [wg][64] mask words of the unit
    // [range][RP] first parts of maxima in two parts, negated; factors of a finished unit
    L.off_qs = (L.off_nh + 4u * S::NT * RP + 15u) & ~15u;
    L.off_sc = L.off_qs + 4u * S::NT * QS_RING * RP;        // [range][QS_RING][RP] query row scales
    L.off_vnan = L.off_sc + 8u * S::NT * SC_RING * SC_BATCH * PAGES_TILE;  // [range][batch][32] page scales (K, V)
    L.off_misc = L.off_vnan + 4u * S::NT * UNIT_RING;
    L.total = L.off_misc + 16u + 4u * 40;
    return L;
}

struct Q8Params {
    CUtensorMap tm_k;
    CUtensorMap tm_v;
    AttnParams a;  // num_ctas counts ranges
    const float2 *scales;
    int NK, NV, Nc;
    uint32_t wait_ns;  // bound of a wait
};

// A lane's D/16 entries of a query row, in bf16 bits, as two 8-bit words' worth of
// registers: 16 lanes hold a row.
template <int D>
struct QueryLane {
    static constexpr int E = D / 16;
    using Half = typename std::conditional<D == 128, uint2, uint32_t>::type;  // E bytes
    using Raw = typename std::conditional<D == 128, uint4, uint2>::type;      // 2 E bytes
};

// Cuts the entries a lane holds of row r (raw bf16 bits, the low half of them at
// `a`, the high half at `b`) into two e4m3 pieces, the first written to `a`, the
// second to `b`, and writes the row's scale. The 16 lanes of a half warp hold a
// row. A row with an entry that is not finite gets the scale NaN, and with it
// NaN outputs.
template <int D>
SV_DEV void cut_query_row(uint8_t *a, uint8_t *b, float *scale, int lane) {
    constexpr int E = QueryLane<D>::E;
    using Half = typename QueryLane<D>::Half;
    const Half ra = *reinterpret_cast<const Half *>(a), rb = *reinterpret_cast<const Half *>(b);
    const uint32_t *wa = reinterpret_cast<const uint32_t *>(&ra), *wb = reinterpret_cast<const uint32_t *>(&rb);
    float x[E];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        const uint32_t w = i < E / 4 ? wa[i] : wb[i - E / 4];
        x[2 * i] = __uint_as_float(w << 16);
        x[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
        top = max(top, max((w << 16) & 0x7FFFFFFFu, w & 0x7FFF0000u));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool finite = top < 0x7F800000u;
    // |x| <= 448 * 2^e, e no smaller than -119: a unit in two parts divides differences
    // of scores, up to 2^7 for a row this small, by 2^e. The smallest rows are then held
    // to 2^-129, which moves a score by 2^-16 at most (448 * 2^100 the largest key entry).
    const int ex = (int)(top >> 23) - 127;
    const int e = max(-119, (top & 0x7FFFFFu) <= 0x600000u ? ex - 8 : ex - 7);
    const float inv = finite ? exp2_int(-e) : 0.f;
    uint32_t hi[E / 4] = {}, lo[E / 4] = {};
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        const float y0 = x[i] * inv, y1 = x[i + 1] * inv;
        const uint32_t h = float2_to_e4m3x2(y0, y1);
        const float2 back = e4m3x2_to_float2(h);
        hi[i / 4] |= h << (8 * (i % 4));
        lo[i / 4] |= float2_to_e4m3x2(y0 - back.x, y1 - back.y) << (8 * (i % 4));
    }
    *reinterpret_cast<Half *>(a) = *reinterpret_cast<const Half *>(hi);
    *reinterpret_cast<Half *>(b) = *reinterpret_cast<const Half *>(lo);
    if (lane % 16 == 0) *scale = finite ? exp2_int(e) : NAN;
}

// Sums (or maxima) of CH values over the warp's lanes: the lane returns that of
// value lane / 2. Each step halves the values a lane carries: 16 shuffles in place
// of 80.
template <bool MAX = false>
SV_DEV float warp_reduce(float *v, int lane) {
    auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
    for (int half = CH / 2, bit = 16; half > 0; half >>= 1, bit >>= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
            v[i] = join(keep, __shfl_xor_sync(0xffffffffu, send, bit));
        }
    }
    return join(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
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

// Two fp32 operations per instruction.
SV_DEV uint64_t pack2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
SV_DEV void unpack2(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
SV_DEV uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
SV_DEV uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
SV_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Bounded wait on a phase, in few instructions (there are two dozen of them in
// the kernel): gives up limit_ns after its first try, or once another thread has raised
// *abort; raises it then. (A count of tries would be no bound: a try takes 80 ns to 4 us.)
SV_DEV uint32_t clock_ns() {
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}
SV_DEV bool wait_phase(uint64_t *b, uint32_t parity, volatile int *abort, uint32_t limit_ns) {
    if (mbar_try_wait(b, parity)) return true;
    const uint32_t t0 = clock_ns();
    bool done;
#pragma unroll 1
    do done = mbar_try_wait(b, parity);
    while (!done && !*abort && clock_ns() - t0 <= limit_ns);
    if (!done) *abort = 1;
    return done;
}

// Barrier of the 128 threads of a warpgroup, plain and with the or of a predicate.
SV_DEV void wg_sync(int id) { named_bar_sync(id, 128); }
SV_DEV bool wg_any(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id)
        : "memory");
    return r != 0;
}

template <int D, int RP>
__global__ void __launch_bounds__(Q8Shape<RP>::THREADS, 1) attn_q8_kernel(const __grid_constant__ Q8Params P) {
    using S = Q8Shape<RP>;
    constexpr int CW = S::CW, NG = S::NG, NT = S::NT, SB = S::SB, PB = S::PB, NQ = S::NQ;
    constexpr int ACC = S::ACC;
    constexpr int MATH_WARPS = S::MATH_WARPS, NTHREADS = S::THREADS;
    constexpr int WARP_LD = MATH_WARPS, WARP_MMA = MATH_WARPS + NT, WARP_AUX = MATH_WARPS + 2 * NT;
    constexpr int SW = D == 128 ? 2 : 4;             // swizzle of K, V and Q rows
    constexpr uint32_t GROUP = 16u * TILE_KEYS;      // bytes of 16 columns of one piece of P
    const AttnParams &p = P.a;
    const int NK = P.NK, NV = P.NV;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const Q8Layout L = q8_layout<D, RP>(NK, NV, p.B);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the range this warp works for, and its barriers
    const int r = warp < MATH_WARPS ? warp / (4 * NG) : (warp - MATH_WARPS) % NT;
    const int nrb = 2 * NK + 3 * NV + NQ + 2 * SB + 2 * PB + 1 + 2 * SC_RING;
    uint64_t *bar = reinterpret_cast<uint64_t *>(base + L.off_bar);
    uint64_t *k_full = bar + r * nrb, *k_empty = k_full + NK;
    uint64_t *v_full = k_empty + NK, *v_empty = v_full + NV;
    uint64_t *vz = v_empty + NV;        // [NV] the tile's V is ready for its PV
    uint64_t *q_full = vz + NV;         // [NQ]
    uint64_t *s_full = q_full + NQ, *s_empty = s_full + SB;
    uint64_t *p_full = s_empty + SB;    // [PB]
    uint64_t *o_full = p_full + PB;     // [PB] the tile's PV has completed, its P is free
    uint64_t *sc_full = o_full + PB, *sc_empty = sc_full + SC_RING;
    uint64_t *done_bar = sc_empty + SC_RING;
    int *TP = reinterpret_cast<int *>(base + L.off_tp);
    int *CL = reinterpret_cast<int *>(base + L.off_cl);
    int *rowi = reinterpret_cast<int *>(base + L.off_rowi);      // [RP] row r -> r / G
    int *rowoff = reinterpret_cast<int *>(base + L.off_rowoff);  // [RP] entries from a unit's first row to row r
    float2 *scr = reinterpret_cast<float2 *>(base + L.off_sc) + r * SC_RING * 32;
    int *vnan = reinterpret_cast<int *>(base + L.off_vnan) + r * UNIT_RING;
    uint8_t *k_ring = base + L.off_k + r * NK * L.tile_bytes, *v_ring = base + r * NV * L.tile_bytes;
    uint8_t *q_buf = base + L.off_q + r * NQ * L.q_bytes, *p_buf = base + L.off_p + r * PB * L.p_bytes;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + L.off_misc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(base + L.off_misc + 4);
    int *scratch = reinterpret_cast<int *>(base + L.off_misc + 16);

    if (lane == 0 && warp >= WARP_AUX) {  // each range's barriers, by its AUX warp
#pragma unroll 1
        for (int s = 0; s < NK; ++s) { mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], 1); }
#pragma unroll 1
        for (int s = 0; s < NV; ++s) { mbar_init(&v_full[s], 1); mbar_init(&v_empty[s], 1); mbar_init(&vz[s], 1); }
        for (int i = 0; i < NQ; ++i) mbar_init(&q_full[i], 4 * NG);
        for (int i = 0; i < SB; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 4 * NG); }
        for (int i = 0; i < PB; ++i) { mbar_init(&p_full[i], 4 * NG); mbar_init(&o_full[i], 1); }
        for (int i = 0; i < SC_RING; ++i) { mbar_init(&sc_full[i], 1); mbar_init(&sc_empty[i], 4 * NG); }
        mbar_init(done_bar, 1);
        if (r == 0) *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == WARP_MMA) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == WARP_LD && lane == 0) {
        tma_prefetch_desc(&P.tm_k);
        tma_prefetch_desc(&P.tm_v);
    }
#pragma unroll 1
    for (int i = tid; i < RP; i += NTHREADS) {
        rowi[i] = i / p.G;
        rowoff[i] = (i / p.G * p.Hq + i % p.G) * D;
    }
    griddep_wait();  // no input is read, and nothing written, before this wait
    griddep_launch_dependents();
    tile_prefix<UC>(p, TP, scratch, CL);  // contains __syncthreads
    const int ups = p.Hkv * p.RC;
    const int total = ups * TP[p.B];
    const int W = schedule_width(p, total);
    // range r of this CTA is the schedule's range blockIdx.x + r * gridDim.x
    if (tid < NT) {
        const int v0 = (int)min((long long)(blockIdx.x + tid * gridDim.x) * W, (long long)total);
        const int v1 = min(v0 + W, total);
        int n;
        const TileInfo t0 = cta_tiles<UC>(TP, p.B, ups, v0, v1, &n);
        int *o = scratch + 8 * tid;
        o[0] = t0.b; o[1] = t0.hr; o[2] = t0.j; o[3] = t0.Tb; o[4] = n;
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot + r * S::R_COLS;
    const TileInfo t_first{scratch[8 * r], scratch[8 * r + 1], scratch[8 * r + 2], scratch[8 * r + 3]};
    // Test hook: to one role of the CTA's first range there are no tiles, so that the
    // others wait for what never comes.
    const int role = warp < WARP_LD ? SV_STALL_SOFTMAX
                                    : warp < WARP_MMA ? SV_STALL_LOADS : warp < WARP_AUX ? SV_STALL_MMA : SV_STALL_AUX;
    const int ntiles = p.stall == role && r == 0 ? 0 : scratch[8 * r + 4];

    auto wait_w = [&](uint64_t *b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait_phase(b, parity, abort_flag, P.wait_ns));
    };

    if (warp >= WARP_AUX) {
        // ---------------- per-sequence status (and invalid sequences) ----------------
        if (r == 0)
#pragma unroll 1
            for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
                const int C = CL[b];
                const bool ctx_ok = C >= p.N && C <= p.max_blocks * PAGE;
                int bad = 0;
                if (ctx_ok) {
#pragma unroll 1
                    for (int jb = lane; jb < (C + PAGE - 1) / PAGE; jb += 32) {
                        const int blk = __ldg(p.block_table + (size_t)b * p.max_blocks + jb);
                        bad |= (blk < 0 || blk >= p.num_blocks);
                    }
                } else {
                    uint4 *o4 = reinterpret_cast<uint4 *>(p.out + (size_t)b * p.N * p.Hq * D);
#pragma unroll 1
                    for (int e = lane; e < p.N * p.Hq * D / 8; e += 32) o4[e] = make_uint4(0, 0, 0, 0);
                }
                bad = __any_sync(0xffffffffu, bad);
                if (p.status && lane == 0)
                    p.status[b] = (ctx_ok ? 0 : SV_FLAG_BAD_CONTEXT) | (bad ? SV_FLAG_BAD_BLOCK : 0);
            }
        // Page scales come in batches of SC_BATCH tiles: lane l has tile l / 8's page
        // l % 8. The next batch is fetched while this one's tiles are cleaned.
        TileInfo ta = t_first;
        int blk = -1, head = 0;
        auto batch_ids = [&](int t) {  // of the batch whose first tile, the range's t-th, is ta
            TileInfo mine = ta;
#pragma unroll 1
            for (int j = 1; j <= SC_BATCH; ++j) {
                next_tile<UC>(ta, TP, p.B, ups);
                if (lane / PAGES_TILE >= j) mine = ta;
            }
            const int page = mine.j * PAGES_TILE + lane % PAGES_TILE;
            head = mine.hr / p.RC;
            blk = -1;
            if (t + lane / PAGES_TILE < ntiles && page * PAGE < CL[mine.b])
                blk = __ldg(p.block_table + (size_t)mine.b * p.max_blocks + page);
        };
        float2 sc = make_float2(1.f, 1.f);
        auto batch_scales = [&]() {
            sc = make_float2(1.f, 1.f);
            if (blk >= 0 && blk < p.num_blocks) sc = __ldg(P.scales + (size_t)blk * p.Hkv + head);
        };
        auto batch_publish = [&](int batch) -> bool {
            const int slot = batch % SC_RING;
            if (!wait_w(&sc_empty[slot], (batch / SC_RING & 1) ^ 1)) return false;
            scr[slot * 32 + lane] = make_float2(page8_scale(sc.x), page8_scale(sc.y));
            __syncwarp();
            if (lane == 0) mbar_arrive(&sc_full[slot]);
            return true;
        };
        bool ok = true;
        if (ntiles > 0) {
            batch_ids(0);
            batch_scales();
            ok = batch_publish(0);
        }
        // V rows past ctx_len, NaN of new keys. 0 * NaN is NaN: rows past ctx_len
        // hold whatever the pool holds, and a new key that some rows must not see
        // may hold NaN. Both are zeroed once the tile has landed. Where NaN was
        // zeroed the unit is marked, and its read-out puts it back for the rows that
        // see the key.
        TileInfo ti = t_first;
        int vs = 0, u = -1;
        uint32_t vph = 0;
#pragma unroll 1
        for (int lt = 0; lt < ntiles && ok; ++lt) {
            const bool more = lt % SC_BATCH == 0 && lt + SC_BATCH < ntiles;
            if (more) batch_ids(lt + SC_BATCH);
            if (lt == 0 || ti.j == 0) {
                ++u;
                // the ring outlasts the units between this warp and the read-out
                if (lane == 0) vnan[u % UNIT_RING] = 0;
            }
            const int C = CL[ti.b];
            // keys of the tile from the first new one on, and from ctx_len on
            // (pages wholly past ctx_len were loaded as zeros by the TMA unit)
            const int kn = max(0, C - p.N - ti.j * TILE_KEYS), k0 = max(0, C - ti.j * TILE_KEYS);
            const int k1 = min(TILE_KEYS, (k0 + PAGE - 1) / PAGE * PAGE);
            next_tile<UC>(ti, TP, p.B, ups);
            if (!(ok = wait_w(&v_full[vs], vph))) break;
            if (kn < k1) {
                uint8_t *vt = v_ring + vs * L.tile_bytes;
                bool hit = false;
#pragma unroll 1
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
            if (lane == 0) mbar_arrive(&vz[vs]);
            if (++vs == NV) { vs = 0; vph ^= 1u; }
            if (more) batch_scales();
            if (lt % SC_BATCH == 2 && lt + 2 < ntiles) ok = batch_publish(lt / SC_BATCH + 1);
        }
    } else if (warp >= WARP_MMA) {
        // -------------------------- MMA issuer ----------------------------
        // The range's products in order.
        if (lane == 0) {
            constexpr uint32_t idq = idesc_f8(128, RP, 0, 0, false, false);
            constexpr uint32_t idp = idesc_f8(128, ACC * RP, 0, 1, true, true), idp1 = idesc_f8(128, RP, 0, 1, true, true);
            const uint64_t kdesc = smem_desc(smem_u32(k_ring), 16, 8 * D, SW);
            const uint64_t qdesc = smem_desc(smem_u32(q_buf), 16, 8 * D, SW);
            // D = 64: dims 64..127 of the 128-row product read bytes of other keys and are not read out
            const uint64_t vdesc = smem_desc(smem_u32(v_ring), 8 * D, 8 * D, SW);
            const uint64_t pdesc = smem_desc(smem_u32(p_buf), 128, GROUP, 0);
            // addresses stay in a descriptor's low word; the high words (K's and Q's are alike) are fixed
            const uint32_t khi = (uint32_t)(kdesc >> 32), vhi = (uint32_t)(vdesc >> 32), phi = (uint32_t)(pdesc >> 32);
            int ks = 0, vs = 0;
            uint32_t kph = 0, vph = 0;
            TileInfo tq = t_first, tp = tq;
            int lu = -1;
            auto wait1 = [&](uint64_t *b, uint32_t parity) {
                return wait_phase(b, parity, abort_flag, P.wait_ns);
            };
            auto issue_qk = [&](int t) -> bool {
                if (t == 0 || tq.j == 0) {
                    ++lu;
                    if (!wait1(&q_full[lu % NQ], (lu / NQ) & 1)) return false;
                }
                if (!wait1(&k_full[ks], kph) || !wait1(&s_empty[t % SB], ((t / SB) & 1) ^ 1)) return false;
                tc_fence_after();
                const uint32_t ka = (uint32_t)kdesc + ((ks * L.tile_bytes) >> 4);
                const uint32_t qa = (uint32_t)qdesc + ((lu % NQ * L.q_bytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
#pragma unroll
                    for (int piece = 0; piece < 2; ++piece)
                        mma_f8_ss(tmem + S::TM_S + t % SB * RP, ka + ((kk * 32) >> 4), khi,
                                  qa + ((piece * RP * D + kk * 32) >> 4), khi, idq, kk + piece > 0);
                mma_commit(&s_full[t % SB]);
                mma_commit(&k_empty[ks]);
                if (++ks == NK) { ks = 0; kph ^= 1u; }
                next_tile<UC>(tq, TP, p.B, ups);
                return true;
            };
            auto issue_pv = [&](int t) -> bool {
                const bool newu = t == 0 || tp.j == 0;
                if (!wait1(&p_full[t % PB], (t / PB) & 1) || !wait1(&vz[vs], vph)) return false;
                tc_fence_after();
                const uint32_t va = (uint32_t)vdesc + ((vs * L.tile_bytes) >> 4);
                const uint32_t pa = (uint32_t)pdesc + ((t % PB * L.p_bytes) >> 4);
                // the first ACC pieces side by side, the others into the last sum
#pragma unroll
                for (int kk = 0; kk < TILE_KEYS / 32; ++kk) {
                    mma_f8_ss(tmem, va + ((kk * 32 * D) >> 4), vhi, pa + ((kk * 512) >> 4), phi, idp,
                              (kk > 0 || !newu) ? 1u : 0u);
#pragma unroll
                    for (int piece = ACC; piece < 3; ++piece)
                        mma_f8_ss(tmem + (ACC - 1) * RP, va + ((kk * 32 * D) >> 4), vhi,
                                  pa + ((piece * (RP / 16) * GROUP + kk * 512) >> 4), phi, idp1, 1u);
                }
                mma_commit(&o_full[t % PB]);
                mma_commit(&v_empty[vs]);
                if (++vs == NV) { vs = 0; vph ^= 1u; }
                next_tile<UC>(tp, TP, p.B, ups);
                return true;
            };
            // Q.K of tile q runs up to SB tiles ahead of P.V of tile v. With one query
            // buffer a unit's rows are cut after the last unit is read out: its last
            // P.V comes first.
            int q = 0, v = 0;
            bool ok = true;
#pragma unroll 1
            while (v < ntiles && ok) {
                const bool behind = NQ == 1 && tq.j == 0 && q > v;
                if (q < ntiles && q < v + SB && !behind)
                    ok = issue_qk(q++);
                else
                    ok = issue_pv(v++);
            }
            mma_commit(done_bar);  // every MMA of this range has finished before TMEM is freed
            mbar_wait_time(done_bar, 0, WAIT_LIMIT_NS);
        }
    } else if (warp >= WARP_LD) {
        // -------------------------- TMA producer --------------------------
        // K one tile ahead of V. Page ids of a tile, one per lane 0..7; num_blocks
        // (a coordinate past the pool, which the TMA unit fills with zeros) for ids
        // out of range and pages past ctx_len.
        TileInfo ti = t_first;  // the tile after the last one whose ids were fetched
        auto page_ids = [&]() -> int {
            const int page = ti.j * PAGES_TILE + lane;
            int blk = -1;
            if (lane < PAGES_TILE && page * PAGE < CL[ti.b])
                blk = __ldg(p.block_table + (size_t)ti.b * p.max_blocks + page);
            return blk;
        };
        int slot[2] = {0, 0}, issued[2] = {0, 0};
        uint32_t ph[2] = {0, 0};
        bool ok = true;
        auto load = [&](int kv, int ids, int h) -> bool {
            uint64_t *full = kv ? v_full : k_full, *empty = kv ? v_empty : k_empty;
            const int s = slot[kv], NR = kv ? NV : NK;
            if (!wait_w(&empty[s], ph[kv] ^ 1u)) return false;
            uint8_t *dst = (kv ? v_ring : k_ring) + s * L.tile_bytes;
            if (lane == 0) mbar_arrive_expect_tx(&full[s], L.tile_bytes);
            __syncwarp();
            const int blk = ids >= 0 && ids < p.num_blocks ? ids : p.num_blocks;
            if (lane < PAGES_TILE)
                tma_load_4d(dst + lane * (PAGE * D), kv ? &P.tm_v : &P.tm_k, &full[s], 0, 0, h, blk);
            ++issued[kv];
            if (++slot[kv] == NR) { slot[kv] = 0; ph[kv] ^= 1u; }
            return true;
        };
        int idv = 0, hv = 0;  // of the tile whose V comes next
        int idk = 0;
        if (ntiles > 0) idk = page_ids();
#pragma unroll 1
        for (int lt = 0; lt <= ntiles && ok; ++lt) {
            const int h = ti.hr / p.RC, ids = idk;
            if (lt < ntiles) next_tile<UC>(ti, TP, p.B, ups);
            if (lt + 1 < ntiles) idk = page_ids();  // in flight while this tile waits for its slots
            if (lt < ntiles) ok = load(0, ids, h);
            if (lt > 0 && ok) ok = load(1, idv, hv);
            idv = ids;
            hv = h;
        }
        if (lane == 0) {  // for the teardown
            scratch[8 * r + 5] = issued[0];
            scratch[8 * r + 6] = issued[1];
        }
    } else {
        // ------------------------------ softmax ------------------------------
        // A wait that runs out leaves `ok` false; the warp goes on to the next vote
        // without work, past every barrier on the way, and the warpgroup leaves
        // together from there, so that no warp is missing at a barrier.
        const int wg = warp >> 2, cg = wg - r * NG;
        const int wiw = warp & 3;          // warp within the warpgroup = TMEM lane quadrant
        const int ell = wiw * 32 + lane;   // key (S) / head dim (O) lane
        const int col0 = cg * CW;
        const int seg = blockIdx.x + r * gridDim.x;
        const uint32_t tm_o = tmem + ((uint32_t)(wiw * 32) << 16) + col0;
        const uint32_t tm_s = tmem + ((uint32_t)(wiw * 32) << 16) + S::TM_S + col0, tm_l = tm_s + SB * RP;
        float *red = reinterpret_cast<float *>(base + L.off_red) + r * 4 * RP + col0;  // [warp] * RP
        float *nm = reinterpret_cast<float *>(base + L.off_nm) + r * RP + col0;
        float *as = reinterpret_cast<float *>(base + L.off_as) + r * RP + col0;
        float *nh = reinterpret_cast<float *>(base + L.off_nh) + r * RP + col0;
        uint64_t *umask = reinterpret_cast<uint64_t *>(base + L.off_umask) + wg * 64;
        float *qs_ring = reinterpret_cast<float *>(base + L.off_qs) + r * QS_RING * RP;
        const size_t slot_floats = slot_stride(p.rows_unit, D);
        bool ok = true, split = false;  // split: the unit's maxima are in two parts
        int lu = -1, ub = 0, uhr = 0, uC = 0;

        auto warp_arrive = [&](uint64_t *b) {
            __syncwarp();
            if (lane == 0) mbar_arrive(b);
        };
        // this warpgroup's share of the query rows of tile ti's unit, the range's u-th
        auto cut_queries = [&](const TileInfo &ti, int u) {
            const int h = ti.hr / p.RC, rc = ti.hr - h * p.RC;
            const int rows = min(p.rows_unit, p.R - rc * p.rows_unit);
            const uint16_t *q = p.q + (((size_t)ti.b * p.N + rc * P.Nc) * p.Hq + h * p.G) * D;
            // half a warp to a row; all loads in flight, then the raw bits to where the
            // lane's pieces go, then (rolled, for the code's size) the cut in place
            constexpr int E = QueryLane<D>::E;
            using Raw = typename QueryLane<D>::Raw;
            using Half = typename QueryLane<D>::Half;
            const int row0 = (cg * 4 + wiw) * 2 + (lane >> 4), l16 = lane & 15;
            uint8_t *qb = q_buf + u % NQ * L.q_bytes;
            auto place = [&](int row) -> uint8_t * {
                const int at = l16 * E, sw = D == 128 ? row & 7 : (row >> 1) & 3;
                return qb + row * D + (((at >> 4) ^ sw) << 4) + (at & 15);
            };
            constexpr int PER = (RP / 2 + 4 * NG - 1) / (4 * NG);  // rows of a half warp
            Raw raw[PER];
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int row = row0 + k * 8 * NG;
                if (row < rows) raw[k] = __ldg(reinterpret_cast<const Raw *>(q + rowoff[row]) + l16);
                else memset(&raw[k], 0, sizeof(Raw));
            }
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                if (RP % (8 * NG) && row0 + k * 8 * NG >= RP) break;
                uint8_t *at = place(row0 + k * 8 * NG);
                *reinterpret_cast<Half *>(at) = reinterpret_cast<const Half *>(&raw[k])[0];
                *reinterpret_cast<Half *>(at + RP * D) = reinterpret_cast<const Half *>(&raw[k])[1];
            }
#pragma unroll 1
            for (int k = 0; k < PER; ++k) {
                const int row = row0 + k * 8 * NG;
                if (RP % (8 * NG) && row - (lane >> 4) >= RP) break;  // the warp's two rows are even and odd, RP is even
                uint8_t *at = place(row);
                cut_query_row<D>(at, at + RP * D, qs_ring + u % QS_RING * RP + row, lane);
            }
            fence_proxy_async_smem();
            warp_arrive(&q_full[u % NQ]);
        };
        // The unit is through: its row sums over the 128 key lanes, then O^T (lane =
        // head dim, column = row) out of TMEM; normalised and written out if this
        // range covered the unit whole, else a partial for the combine kernel.
        auto finish_unit = [&](int tlast) -> bool {
#pragma unroll 1
            for (int c0 = 0; c0 < CW; c0 += CH) {
                float l[CH];
                tmem_ld16(tm_l + c0, l);
                tmem_wait_ld();
                const float v = warp_reduce<>(l, lane);
                if (lane % 2 == 0) red[wiw * RP + c0 + lane / 2] = v;
            }
            wg_sync(1 + wg);
            const int fh = uhr / p.RC, frc = uhr - fh * p.RC;
            const int frows = min(p.rows_unit, p.R - frc * p.rows_unit) - col0;  // of this warpgroup's columns
            const int Tb = real_tiles<UC>(TP[ub + 1] - TP[ub]);
            const int tpre = ups * TP[ub] + uhr * (Tb + UC);  // the unit's first position
            const bool to_slot = (tpre + Tb - 1) / W != tpre / W;
            float *slot = p.ws_partial + (size_t)(ub * ups + uhr + seg) * slot_floats;
            if (ell < CW) {
                const float l = (red[ell] + red[RP + ell]) + (red[2 * RP + ell] + red[3 * RP + ell]);
                // in a slot the maximum is hi alone: lo, at most 100 either way, goes into the
                // sums, which stay below 2^100 a key and 2^109 times the keys
                const float back = split ? ex2_approx(-nm[ell]) : 1.f;
                if (to_slot && ell < frows) {
                    slot[(size_t)p.rows_unit * D + col0 + ell] = split ? -nh[ell] : -nm[ell];
                    slot[(size_t)p.rows_unit * D + p.rows_unit + col0 + ell] = l * back;
                }
                // what O is multiplied by, in nh's place: a row that saw nothing gives 0
                nh[ell] = to_slot ? back : l > 0.f || l != l ? 1.f / l : 0.f;
            }
            wg_sync(1 + wg);
            if (!wait_w(&o_full[tlast % PB], (tlast / PB) & 1)) return false;
            tc_fence_after();
            const bool marked = vnan[lu % UNIT_RING] != 0;
            uint16_t *ounit = p.out + (((size_t)ub * p.N + frc * P.Nc) * p.Hq + fh * p.G) * D + ell;
            float *sunit = slot + (size_t)col0 * D + ell;
#pragma unroll 1
            for (int c0 = 0; c0 < CW; c0 += CH) {
                float o[CH];
                tmem_ld16(tm_o + c0, o);
#pragma unroll
                for (int i = 1; i < ACC; ++i) {
                    float o1[CH];
                    tmem_ld16(tm_o + i * RP + c0, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < CH; ++c) o[c] += o1[c];
                }
                tmem_wait_ld();
#pragma unroll
                for (int c4 = 0; c4 < CH / 4; ++c4) {
                    const float4 f = reinterpret_cast<const float4 *>(nh + c0)[c4];
                    o[c4 * 4] = o[c4 * 4] * P_UNSCALE * f.x;
                    o[c4 * 4 + 1] = o[c4 * 4 + 1] * P_UNSCALE * f.y;
                    o[c4 * 4 + 2] = o[c4 * 4 + 2] * P_UNSCALE * f.z;
                    o[c4 * 4 + 3] = o[c4 * 4 + 3] * P_UNSCALE * f.w;
                }
                if (ell >= D) continue;
                if (marked) {
                    // NaN among the new keys' V, zeroed for the product: back to the rows that see the key
#pragma unroll 1
                    for (int k = 0; k < p.N; ++k) {
                        const int t = uC - p.N + k;
                        const int blk = __ldg(p.block_table + (size_t)ub * p.max_blocks + t / PAGE);
                        if (blk < 0 || blk >= p.num_blocks) continue;
                        const uint8_t *vp = reinterpret_cast<const uint8_t *>(p.v_pool) +
                                            (((size_t)blk * p.Hkv + fh) * PAGE + t % PAGE) * D;
                        if ((vp[ell] & 0x7F) != 0x7F) continue;
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            const int i = frc * P.Nc + rowi[col0 + c0 + c];
                            if (c0 + c < frows &&
                                (p.mask ? (__ldg(p.mask + (size_t)ub * p.N + i) >> k & 1) != 0 : k <= i))
                                o[c] = NAN;
                        }
                    }
                    __syncwarp();
                }
                if (to_slot) {
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        if (c0 + c < frows) sunit[(c0 + c) * D] = o[c];
                } else {
#pragma unroll
                    for (int c4 = 0; c4 < CH / 4; ++c4) {
                        const int4 at = reinterpret_cast<const int4 *>(rowoff + col0 + c0)[c4];
                        const int off[4] = {at.x, at.y, at.z, at.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const __nv_bfloat16 v = __float2bfloat16_rn(o[c4 * 4 + i]);
                            if (c0 + c4 * 4 + i < frows) ounit[off[i]] = *reinterpret_cast<const uint16_t *>(&v);
                        }
                    }
                }
            }
            tc_fence_before();  // the next unit's first P.V, after this warpgroup's P, overwrites O
            return true;
        };

        if (ntiles > 0) cut_queries(t_first, 0);
        TileInfo tnext = t_first;
#pragma unroll 1
        for (int lt = 0; lt <= ntiles; ++lt) {
            const bool end = lt == ntiles;
            const TileInfo ti = tnext;
            const bool first = lt == 0 || end || ti.j == 0;
            if (first) {
                if (lt > 0) {
                    if (wg_any(1 + wg, !ok)) break;
                    ok = finish_unit(lt - 1);
                }
                if (end) break;
                ++lu;
                ub = ti.b;
                uhr = ti.hr;
                uC = CL[ub];
                if (NQ == 1 && lu > 0) cut_queries(ti, lu);
                if (p.mask) {
#pragma unroll 1
                    for (int k = ell; k < p.N; k += 128) umask[k] = __ldg(p.mask + (size_t)ub * p.N + k);
                    wg_sync(1 + wg);
                }
            }
            next_tile<UC>(tnext, TP, p.B, ups);
            // the page's scales: K's in the exponent's unit, V's
            const int sslot = lt / SC_BATCH % SC_RING;
            if (ok) ok = wait_w(&sc_full[sslot], lt / (SC_BATCH * SC_RING) & 1);
            const float2 scl = scr[sslot * 32 + lt % SC_BATCH * PAGES_TILE + ell / PAGE];
            if (lt % SC_BATCH == SC_BATCH - 1) warp_arrive(&sc_empty[sslot]);
            const float lv = __log2f(scl.y), ks1 = scl.x * p.scale_log2;
            uint64_t ksc = pack2(ks1, ks1);
            const uint64_t vsc = pack2(scl.y * P_SCALE, scl.y * P_SCALE);
            const float *qs = qs_ring + lu % QS_RING * RP + col0;
            const int sb = lt % SB;
            const uint32_t saddr = tm_s + sb * RP;
            if (ok) ok = wait_w(&s_full[sb], (lt / SB) & 1);
            tc_fence_after();

            // Tiles with keys past ctx_len or new (masked) keys: -inf, back into S, for
            // the columns that do not see this key.
            const int key = ti.j * TILE_KEYS + ell;
            const int newk = key - (uC - p.N);
            if (ok && __any_sync(0xffffffffu, newk >= 0)) {
                const int ibase = (uhr % p.RC) * P.Nc;
#pragma unroll 1
                for (int c0 = 0; c0 < CW; c0 += CH) {
                    float x[CH];
                    tmem_ld16(saddr + c0, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        // columns past the unit's rows: any answer will do
                        const int i = min(ibase + rowi[col0 + c0 + c], p.N - 1);
                        const bool bit = p.mask ? (umask[i] >> (newk & 63) & 1ull) != 0 : newk <= i;
                        if (newk >= 0 && !(bit && key < uC)) x[c] = -INFINITY;
                    }
                    tmem_st16(saddr + c0, x);
                }
                tmem_wait_st();
            }

            // x = s * qs is the exponent (log2 units, without the maximum); the
            // running maximum is of x + log2(V's scale), the weight that enters the
            // product with V. It is raised only when one passes it by 2^8
            // (P_MAX). That is rare after a unit's first tile, so the tile's
            // weights are made against the maxima there are, and only then does the
            // warpgroup vote; if one was too large the maxima are raised and the tile
            // is done again, its weights taken out of the row sums first.
            const int pb = lt % PB;
            uint8_t *pdst = p_buf + pb * L.p_bytes + ell * 16;
            auto p_at = [&](int c0) { return (col0 + c0) / 16 * GROUP; };
            if (lt >= PB && ok) ok = wait_w(&o_full[pb], ((lt - PB) / PB) & 1);  // P is free
            const bool fresh = first;  // a unit in two parts raises at every tile, before its weights are made
            bool raise = first || split, leave = false;
            // a second raise in a row cannot come: the maxima are the tile's own then
#pragma unroll 1
            for (int tries = 0;; ++tries) {
                if (!raise) {
                    __half2 top2 = __float2half2_rn(0.f);
                    if (ok) {
#pragma unroll 1
                        for (int c0 = 0; c0 < CW; c0 += CH) {
                            float x[CH], l[CH];
                            tmem_ld16(saddr + c0, x);
                            tmem_wait_ld();
                            tmem_ld16(tm_l + c0, l);
                            // in phases over the chunk, so that no value waits for the one before
                            uint64_t w[CH / 2];
                            uint32_t h[CH / 2], piece[3][CH / 4];
#pragma unroll
                            for (int c4 = 0; c4 < CH / 4; ++c4) {
                                const ulonglong2 q4 = reinterpret_cast<const ulonglong2 *>(qs + c0)[c4];
                                const ulonglong2 m4 = reinterpret_cast<const ulonglong2 *>(nm + c0)[c4];
                                // a row's scale is a power of two, so that its product is exact and the sum
                                // with the maximum rounds the same score that the maximum was made from
                                w[2 * c4] = fma2(mul2(pack2(x[c4 * 4], x[c4 * 4 + 1]), ksc), q4.x, m4.x);
                                w[2 * c4 + 1] = fma2(mul2(pack2(x[c4 * 4 + 2], x[c4 * 4 + 3]), ksc), q4.y, m4.y);
                            }
#pragma unroll
                            for (int i = 0; i < CH / 2; ++i) {
                                float a, b;
                                unpack2(w[i], a, b);
                                w[i] = pack2(ex2_approx(a), ex2_approx(b));
                            }
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < CH / 2; ++i) {
                                float a, b;
                                unpack2(add2(pack2(l[2 * i], l[2 * i + 1]), w[i]), l[2 * i], l[2 * i + 1]);
                                unpack2(mul2(w[i], vsc), a, b);
                                const __half2 hh = __floats2half2_rn(a, b);
                                h[i] = *reinterpret_cast<const uint32_t *>(&hh);
                            }
                            {
                                __half2 t[CH / 2];
#pragma unroll
                                for (int i = 0; i < CH / 2; ++i) t[i] = *reinterpret_cast<const __half2 *>(&h[i]);
#pragma unroll
                                for (int o = CH / 4; o > 0; o >>= 1)
#pragma unroll
                                    for (int i = 0; i < o; ++i) t[i] = __hmax2(t[i], t[i + o]);
                                top2 = __hmax2(top2, t[0]);
                            }
#pragma unroll
                            for (int j = 0; j < 3; ++j)
#pragma unroll
                                for (int c4 = 0; c4 < CH / 4; ++c4) piece[j][c4] = cut_piece(h + 2 * c4, j == 2);
                            tmem_st16(tm_l + c0, l);
#pragma unroll
                            for (int j = 0; j < 3; ++j)
                                *reinterpret_cast<uint4 *>(pdst + (j * (RP / 16) * GROUP + p_at(c0))) =
                                    make_uint4(piece[j][0], piece[j][1], piece[j][2], piece[j][3]);
                        }
                        tmem_wait_st();
                    }
                    raise = wg_any(1 + wg, !ok || (tries < 2 && !__hble2(top2, __float2half2_rn(P_MAX))));
                    if (!raise) break;
                }
                if ((leave = wg_any(1 + wg, !ok))) break;
                // tile column maxima over the 128 keys; this tile's weights out of the row sums (the
                // weights of a unit in two parts are made after this)
                const bool were = split && !fresh;
                bool big = were;
#pragma unroll 1
                for (int c0 = 0; c0 < CW && !were; c0 += CH) {
                    float y[CH], l[CH];
                    tmem_ld16(saddr + c0, y);
                    if (!fresh) tmem_ld16(tm_l + c0, l);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        const float e = __fmul_rn(y[c] * ks1, qs[c0 + c]);
                        // a sum that overflowed held nothing that counts beside the weight that made it so
                        l[c] = fresh || l[c] == INFINITY ? 0.f : l[c] - ex2_approx(__fadd_rn(e, nm[c0 + c]));
                        y[c] = __fadd_rn(e, lv);
                    }
                    tmem_st16(tm_l + c0, l);
                    const float m = warp_reduce<true>(y, lane);
                    big |= fabsf(m) >= TWO_PARTS_FROM && fabsf(m) < INFINITY;
                    if (lane % 2 == 0) red[wiw * RP + c0 + lane / 2] = m;
                }
                tmem_wait_st();
                auto tile_max = [&]() {  // of column ell
                    return fmaxf(fmaxf(red[ell], red[RP + ell]), fmaxf(red[2 * RP + ell], red[3 * RP + ell]));
                };
                // once a unit's maxima have two parts, all its tiles' have
                split = wg_any(1 + wg, big);
                float hi = 0.f, lo = 0.f;
                if (ell < CW && !split) hi = tile_max();
                if (__builtin_expect(split, 0)) {  // hi: the largest score; lo: what the scales add to it
#pragma unroll 1
                    for (int part = 0; part < 2; ++part) {
#pragma unroll 1
                        for (int c0 = 0; c0 < CW; c0 += CH) {
                            float y[CH];
                            tmem_ld16(saddr + c0, y);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < CH; ++c) {
                                const float e = __fmul_rn(y[c] * ks1, qs[c0 + c]);
                                y[c] = part ? __fadd_rn(__fsub_rn(e, as[c0 + c]), lv) : e;
                            }
                            const float m = warp_reduce<true>(y, lane);
                            if (lane % 2 == 0) red[wiw * RP + c0 + lane / 2] = m;
                        }
                        wg_sync(1 + wg);
                        if (ell < CW) (part ? lo : hi) = tile_max();
                        if (part) break;
                        if (ell < CW) as[ell] = hi;
                        wg_sync(1 + wg);
                    }
                }
                if (ell < CW) {
                    // h1 stays M_NONE while nothing is visible; M_NONE - finite underflows to 0
                    const float h0 = fresh ? M_NONE : were ? -nh[ell] : -nm[ell], l0 = were ? -nm[ell] : 0.f;
                    const float h1 = fmaxf(h0, hi), l1 = fmaxf((h0 - h1) + l0, (hi - h1) + lo);
                    // a score past fp32's range: NaN for the row (the fused product would pass over it)
                    nm[ell] = h1 == INFINITY ? NAN : split ? -l1 : -h1;
                    nh[ell] = -h1;
                    // the factor's root: V's scales may be 2^200 apart, and a row sum as large
                    as[ell] = ex2_approx(0.5f * ((h0 - h1) + (split ? l0 - l1 : 0.f)));
                }
                wg_sync(1 + wg);
                if (!fresh) {
                    // the row sums and O^T's columns follow, once the previous tile's PV has landed
                    if (ok) ok = wait_w(&o_full[(lt - 1) % PB], ((lt - 1) / PB) & 1);
                    tc_fence_after();
                    if (ok) {
#pragma unroll 1
                        for (int i = 0; i < CW / CH * (ACC + 1); ++i) {
                            const int c0 = i / (ACC + 1) * CH, k = i % (ACC + 1);
                            const uint32_t at = k == ACC ? tm_l + c0 : tm_o + k * RP + c0;
                            float o[CH];
                            tmem_ld16(at, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < CH; ++c) o[c] = o[c] * as[c0 + c] * as[c0 + c];
                            tmem_st16(at, o);
                        }
                        tmem_wait_st();
                    }
                }
                if (__builtin_expect(split, 0)) {
                    // in the scores' place what gives score - hi, exact where it counts, when
                    // multiplied by the row's scale, a power of two (a NaN stays one)
#pragma unroll 1
                    for (int c0 = 0; c0 < CW; c0 += CH) {
                        float y[CH];
                        tmem_ld16(saddr + c0, y);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            const float e = __fmul_rn(y[c] * ks1, qs[c0 + c]);
                            y[c] = __fadd_rn(e, nh[c0 + c]) * __int_as_float(0x7F000000 - __float_as_int(qs[c0 + c]));
                        }
                        tmem_st16(saddr + c0, y);
                    }
                    tmem_wait_st();
                    ksc = pack2(1.f, 1.f);
                }
                raise = false;
            }
            if (leave) break;
            tc_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s_empty[sb]);
                mbar_arrive(&p_full[pb]);
            }
            if (NQ == 2 && first && lt + ti.Tb - ti.j < ntiles) {
                // the next unit's query rows; the buffer's last products are those of the unit before this one
                TileInfo nu = ti;
                nu.j = nu.Tb - 1;
                next_tile<UC>(nu, TP, p.B, ups);
                cut_queries(nu, lu + 1);
            }
        }
    }

    // ----------------------------- teardown -------------------------------
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && tid < NT * (NK + NV)) {
        // someone gave up: copies that nobody waited for land before the CTA exits. One
        // thread to a slot of K and V of each range.
        const int rr = tid / (NK + NV), at = tid % (NK + NV), ring = at < NK ? NK : NV, slot = at < NK ? at : at - NK;
        const int uses = (scratch[8 * rr + (at < NK ? 5 : 6)] - slot + ring - 1) / ring;
        uint64_t *full = reinterpret_cast<uint64_t *>(base + L.off_bar) + rr * nrb + (at < NK ? slot : 2 * NK + slot);
        if (uses > 0) mbar_wait_time(full, (uses - 1) & 1, WAIT_LIMIT_NS);
    }
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
    using S = Q8Shape<RP>;
    // as many K and V slots as fit, V's the larger half (its slots are held longer)
    int slots = MAX_RING;
    while (q8_layout<D, RP>(slots / 2, slots - slots / 2, P.a.B).total + 1024 > (uint32_t)SMEM_LIMIT)
        if (--slots < 2) return cudaErrorInvalidConfiguration;
    P.NK = slots / 2;
    P.NV = slots - slots / 2;
    const size_t smem = q8_layout<D, RP>(P.NK, P.NV, P.a.B).total + 1024;
    auto kfn = attn_q8_kernel<D, RP>;
    cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int sms = P.a.num_ctas;
    P.a.num_ctas = sms * S::NT;
    e = launch_programmatic(kfn, dim3(sms), dim3(S::THREADS), smem, stream, P);
    return e != cudaSuccess ? e : launch_combine<UC>(P.a, stream);
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
    return attention_workspace_bytes(B, N, Hq, Hkv, D, num_ctas * Q8Shape<16>::NT);
}

cudaError_t launch_attention_q8(const AttnParams &p, const float *scales, cudaStream_t stream) {
    Q8Params P;
    memset(&P, 0, sizeof P);
    P.a = p;
    P.a.min_width = MIN_WIDTH;
    P.scales = reinterpret_cast<const float2 *>(scales);
    P.wait_ns = (uint32_t)p.wait_limit_ns;
    int RU, RC;
    row_chunks(p.N, p.G, &RU, &RC, &P.Nc);
    if (!encode_pool_q8(&P.tm_k, p.k_pool, p.num_blocks, p.Hkv, p.D) ||
        !encode_pool_q8(&P.tm_v, p.v_pool, p.num_blocks, p.Hkv, p.D))
        return cudaErrorInvalidValue;
    const int RP = RU > 64 ? 96 : (RU + 15) / 16 * 16;
    return p.D == 128 ? launch_q8_rp<128>(P, RP, stream) : launch_q8_rp<64>(P, RP, stream);
}

}  // namespace sv
