// sv_kv_append, sv_kv_append_q8: rotate the new rows' q and k by their
// positions and write K and V to the paged cache, for the rows of a verify step
// or for ragged prompts.
//
// The pair (x1, x2) of a row at position t turns by the angle whose cosine and
// sine the caller's table holds: (x1 c - x2 s, x2 c + x1 s). Products and sums
// are rounded one by one (no contraction), so the result is the formula's in
// fp32, bit for bit, whatever the compiler does.
//
// q, and K and V of the bf16 call: a CTA takes one row (or a few, where a row has
// few heads), a thread the same 16 entries of up to AP_BATCH heads at a time and
// their cosines and sines once. K and V of the 8-bit call: a page's scale is the
// maximum over its rows, so two warps take the page of one KV head, K or V.
// Little is computed; what bounds a call is memory when there are many rows, and
// the chain of loads (length, then block id and positions, then cosines and
// sines) when there are few, so the rows themselves are asked for first.
// Measured: 256 x 9 rows of 40 + 16 heads of 128 (67 MB) 13.3 us with L2 warm,
// 18.8 us cold (0.54 of the copy rate); 16 ragged prompts of up to 1500 rows into
// the 8-bit cache (259 MB) 67 us (0.59); 5 rows of one sequence 3.1 us.
#include "sv_page8.cuh"
#include "sv_q8.h"

namespace sv {
namespace {

constexpr int AP_THREADS = 256;
constexpr int AP_WARPS = AP_THREADS / 32;

// What a CTA needs to know of its sequence.
struct Seq {
    int C, n, start;  // context length, new rows, cache position of the first
    bool ok;
};

SV_DEV Seq read_seq(const AppendParams &p, int b) {
    Seq s;
    s.C = p.ctx_lens[b];
    s.n = p.new_lens ? p.new_lens[b] : p.N;
    s.start = s.C - s.n;
    s.ok = s.n >= 0 && s.n <= p.N && s.C >= s.n && s.C <= p.max_blocks * PAGE;
    return s;
}

SV_DEV int row_position(const AppendParams &p, const Seq &s, int b, int i) {
    return p.positions ? p.positions[(size_t)b * p.N + i] : s.start + i;
}

SV_DEV bool bad_position(const AppendParams &p, int t) { return p.R > 0 && (t < 0 || t >= p.max_position); }

// Status of sequence b, by a whole CTA.
SV_DEV void write_status(const AppendParams &p, const Seq &s, int b) {
    int bad_pos = 0, bad_blk = 0;
    if (s.ok && s.n > 0) {
        for (int i = threadIdx.x; i < s.n; i += AP_THREADS) bad_pos |= bad_position(p, row_position(p, s, b, i));
        for (int pg = s.start / PAGE + threadIdx.x; pg <= (s.C - 1) / PAGE; pg += AP_THREADS) {
            const int blk = p.block_table[(size_t)b * p.max_blocks + pg];
            bad_blk |= blk < 0 || blk >= p.num_blocks;
        }
    }
    bad_pos = __syncthreads_or(bad_pos);
    bad_blk = __syncthreads_or(bad_blk);
    if (threadIdx.x == 0)
        p.status[b] = (!s.ok || bad_pos ? SV_FLAG_BAD_CONTEXT : 0) | (bad_blk ? SV_FLAG_BAD_BLOCK : 0);
}

// A page of a sequence that gets new rows: its new rows [i0, i1), its block id
// and, in lanes 0..15 of every warp, its new rows' positions. Loads only; ok()
// looks at them, so that a caller can send its own loads in between.
struct PageRows {
    int page, i0, i1, blk, pos;

    SV_DEV PageRows(const AppendParams &p, const Seq &s, int b, int page_) : page(page_) {
        const int lane = threadIdx.x & 31;
        i0 = max(page * PAGE, s.start) - s.start;
        i1 = min(page * PAGE + PAGE, s.C) - s.start;
        blk = p.block_table[(size_t)b * p.max_blocks + page];
        pos = lane < PAGE && i0 + lane < i1 ? row_position(p, s, b, i0 + lane) : 0;
    }
    // Every lane of the warp takes part; false: the page is skipped.
    SV_DEV bool ok(const AppendParams &p) const {
        const int lane = threadIdx.x & 31;
        const bool bad = lane < PAGE && i0 + lane < i1 && bad_position(p, pos);
        return !__any_sync(0xffffffffu, bad) && blk >= 0 && blk < p.num_blocks;
    }
};

// A head is taken in slots of two chunks of 8 entries (16 bytes). Slot s < R/16
// holds entries that turn by the angles [8s, 8s + 8): chunks s and s + R/16 in
// the half layout, 2s and 2s + 1 in the interleaved one. The slots behind hold
// the entries that do not turn, two chunks each (the last one may have one).
struct Slot {
    int c1, c2;
    bool turns, two;
    SV_DEV Slot(const AppendParams &p, int s) {
        const int n = p.R / 16;
        turns = s < n;
        c1 = turns ? (p.interleaved ? 2 * s : s) : p.R / 8 + 2 * (s - n);
        c2 = turns && !p.interleaved ? s + n : c1 + 1;
        two = 8 * c2 < p.D;
    }
};

// Two fp32 products per instruction, each rounded by itself.
SV_DEV float2 mul2(float a0, float a1, uint64_t b) {
    float2 d;
    asm("{\n\t.reg .b64 a, d;\n\tmov.b64 a, {%2, %3};\n\tmul.rn.f32x2 d, a, %4;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a0), "f"(a1), "l"(b));
    return d;
}

// The cosines and sines of a slot at position t.
struct Turn {
    ulonglong2 cs[2], sn[2];
    SV_DEV void load(const AppendParams &p, int t, int s) {
        const float *row = p.cos_sin + (size_t)t * p.R + 8 * s;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            cs[k] = __ldg(reinterpret_cast<const ulonglong2 *>(row) + k);
            sn[k] = __ldg(reinterpret_cast<const ulonglong2 *>(row + p.R / 2) + k);
        }
    }
};

// A slot's 16 entries in memory order, in fp32.
SV_DEV void unpack_slot(const uint4 &u1, const uint4 &u2, float *y) {
    const uint32_t w[8] = {u1.x, u1.y, u1.z, u1.w, u2.x, u2.y, u2.z, u2.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[2 * j] = __uint_as_float(w[j] << 16);
        y[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}

// (x1 c - x2 s, x2 c + x1 s) for the slot's 8 pairs: entries j and 8 + j in the
// half layout, 2j and 2j + 1 in the interleaved one. The sums are scalar, so that
// no compiler contracts them with the products.
template <bool INTERLEAVED>
SV_DEV void turn_slot(const Turn &t, float *y) {
    const uint64_t cs[4] = {t.cs[0].x, t.cs[0].y, t.cs[1].x, t.cs[1].y};
    const uint64_t sn[4] = {t.sn[0].x, t.sn[0].y, t.sn[1].x, t.sn[1].y};
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float &a0 = y[INTERLEAVED ? 2 * j : j], &a1 = y[INTERLEAVED ? 2 * j + 2 : j + 1];
        float &b0 = y[INTERLEAVED ? 2 * j + 1 : 8 + j], &b1 = y[INTERLEAVED ? 2 * j + 3 : 9 + j];
        const float2 ac = mul2(a0, a1, cs[j / 2]), bs = mul2(b0, b1, sn[j / 2]);
        const float2 bc = mul2(b0, b1, cs[j / 2]), as = mul2(a0, a1, sn[j / 2]);
        a0 = __fsub_rn(ac.x, bs.x);
        a1 = __fsub_rn(ac.y, bs.y);
        b0 = __fadd_rn(bc.x, as.x);
        b1 = __fadd_rn(bc.y, as.y);
    }
}

// Turns a slot in bf16, rounding once.
template <bool INTERLEAVED>
SV_DEV void turn_bf16(const Turn &t, uint4 &u1, uint4 &u2) {
    float y[16];
    unpack_slot(u1, u2, y);
    turn_slot<INTERLEAVED>(t, y);
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
    u1 = make_uint4(w[0], w[1], w[2], w[3]);
    u2 = make_uint4(w[4], w[5], w[6], w[7]);
}

constexpr int AP_BATCH = 2;  // heads of a thread in flight

// Heads of row i of sequence b by `group` threads (whole warps): q to q_out, and
// (KV) k and v to their page of the bf16 cache.
template <bool KV>
SV_DEV void rotate_row(const AppendParams &p, int b, int i, int tid, int group) {
    const int lanes = group / p.slots;  // heads in flight
    const int h0 = tid / p.slots, sl = tid - h0 * p.slots;
    const Slot slot(p, sl);
    const size_t row = (size_t)b * p.N + i;
    const int hq = p.q ? p.Hq : 0;
    // the slots need not divide the group; rows past new_lens are not read
    const int n = p.new_lens ? p.new_lens[b] : p.N;
    const int heads = h0 < lanes && i < n && i < p.N ? hq + (KV ? 2 * p.Hkv : 0) : 0;
    uint4 u1[AP_BATCH], u2[AP_BATCH];
    auto fetch = [&](int h) {
#pragma unroll
        for (int k = 0; k < AP_BATCH; ++k, h += lanes)
            if (h < heads) {
                const uint16_t *src = h < hq ? p.q + row * p.q_stride + h * p.D
                                             : (h >= hq + p.Hkv ? p.v + row * p.kv_stride + (h - hq - p.Hkv) * p.D
                                                                : p.k + row * p.kv_stride + (h - hq) * p.D);
                u1[k] = __ldg(reinterpret_cast<const uint4 *>(src) + slot.c1);
                if (slot.two) u2[k] = __ldg(reinterpret_cast<const uint4 *>(src) + slot.c2);
            }
    };
    fetch(h0);
    const Seq s = read_seq(p, b);
    if (!s.ok || i >= s.n) return;
    const PageRows pr(p, s, b, (s.start + i) / PAGE);
    const int t = __shfl_sync(0xffffffffu, pr.pos, i - pr.i0);
    Turn turn;
    if (slot.turns) turn.load(p, max(0, min(t, p.max_position - 1)), sl);  // a position outside skips the page below
    if (!pr.ok(p)) return;
    const size_t page = (size_t)pr.blk * p.Hkv * PAGE + (s.start + i) % PAGE;  // row of the cache, of KV head 0
#pragma unroll 1
    for (int h = h0; h < heads; h += AP_BATCH * lanes) {
        if (h != h0) fetch(h);
#pragma unroll
        for (int k = 0; k < AP_BATCH; ++k) {
            const int hh = h + k * lanes;
            if (hh >= heads) break;
            const bool is_v = hh >= hq + p.Hkv;
            if (slot.turns && !is_v) {
                if (p.interleaved) turn_bf16<true>(turn, u1[k], u2[k]);
                else turn_bf16<false>(turn, u1[k], u2[k]);
            }
            uint16_t *dst = hh < hq ? p.q_out + (row * p.Hq + hh) * p.D
                                    : is_v ? static_cast<uint16_t *>(p.v_pool) + (page + (hh - hq - p.Hkv) * PAGE) * p.D
                                           : static_cast<uint16_t *>(p.k_pool) + (page + (hh - hq) * PAGE) * p.D;
            reinterpret_cast<uint4 *>(dst)[slot.c1] = u1[k];
            if (slot.two) reinterpret_cast<uint4 *>(dst)[slot.c2] = u2[k];
        }
    }
}

// Rows a CTA takes: as many as leave a thread no more than one batch of a row's
// heads, in whole warps.
int rows_per_cta(const AppendParams &p, bool kv) {
    const int items = ((p.q ? p.Hq : 0) + (kv ? 2 * p.Hkv : 0)) * p.slots;
    int rows = 1;
    while (rows < AP_WARPS && AP_THREADS / (2 * rows) * AP_BATCH >= items && AP_THREADS / (2 * rows) >= p.slots) rows *= 2;
    return rows;
}

// LOOP: `per` groups of rows to a CTA in place of one (the loop's registers cost the
// rows of a verify step 8 %).
template <bool LOOP>
__global__ void __launch_bounds__(AP_THREADS, 4) append_kernel(const __grid_constant__ AppendParams p, int rows, int per) {
    const int b = blockIdx.y, group = AP_THREADS / rows, sub = threadIdx.x / group;
    if (p.status && blockIdx.x == 0) write_status(p, read_seq(p, b), b);
    if constexpr (LOOP) {
#pragma unroll 1
        for (int g = 0; g < per; ++g)
            rotate_row<true>(p, b, (blockIdx.x * per + g) * rows + sub, threadIdx.x - sub * group, group);
    } else {
        rotate_row<true>(p, b, blockIdx.x * rows + sub, threadIdx.x - sub * group, group);
    }
}

// One page of one KV head, K or V, by two warps, each half of its rows; the
// whole CTA comes here for one page. tops: a float per warp. True where the CTA
// passed the barrier, false (for every thread alike) where the page is skipped.
template <int D>
SV_DEV bool append_page(const AppendParams &p, int b, int index, int job, bool has_job, int warp, int lane, float *tops) {
    // a lane holds one slot (two chunks) of NS of the page's rows
    constexpr int SLOTS = D / 16, ROWS = 32 / SLOTS, NS = PAGE / 2 / ROWS;
    const Seq s = read_seq(p, b);
    const int page = s.start / PAGE + index;
    if (!s.ok || s.n == 0 || page * PAGE >= s.C) return false;
    const int hk = job >> 1;
    const bool is_v = job & 1;
    const uint16_t *src = (is_v ? p.v : p.k) + (size_t)b * p.N * p.kv_stride + (size_t)hk * D;
    const int sl = lane % SLOTS, r0 = (warp & 1) * (PAGE / 2) + lane / SLOTS;  // rows r0, r0 + ROWS, ..
    const Slot slot(p, sl);
    const bool turns = slot.turns && !is_v;
    const int first = page * PAGE - s.start;  // the new row on the page's row 0, if there is one
    uint4 u1[NS], u2[NS];
#pragma unroll
    for (int st = 0; st < NS; ++st) {
        const int i = first + r0 + st * ROWS;
        u1[st] = u2[st] = make_uint4(0, 0, 0, 0);
        if (has_job && i >= 0 && i < s.n) {
            const uint4 *row = reinterpret_cast<const uint4 *>(src + i * p.kv_stride);
            u1[st] = __ldg(row + slot.c1);
            u2[st] = __ldg(row + slot.c2);
        }
    }
    const PageRows pr(p, s, b, page);
    if (!pr.ok(p)) return false;  // the same for every warp of the CTA
    uint8_t *dst = static_cast<uint8_t *>(is_v ? p.v_pool : p.k_pool) + ((size_t)pr.blk * p.Hkv + hk) * PAGE * D;
    float *scale = p.scales + ((size_t)pr.blk * p.Hkv + hk) * 2 + (is_v ? 1 : 0);
    const int kept = min(PAGE, s.C - page * PAGE);
    const float old_scale = has_job && first < 0 ? page8_scale(*scale) : 0.f;  // of rows that are there already
    float y[NS][16], top = 0.f, not_finite = 0.f;
#pragma unroll
    for (int st = 0; st < NS; ++st) {
        const int r = r0 + st * ROWS, i = first + r;
        const int t = __shfl_sync(0xffffffffu, pr.pos, (i - pr.i0) & 31);
        if (i < 0 && has_job) {
            const uint2 b1 = reinterpret_cast<const uint2 *>(dst + r * D)[slot.c1];
            const uint2 b2 = reinterpret_cast<const uint2 *>(dst + r * D)[slot.c2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                unpack_e4m3(b1, j, old_scale, y[st][2 * j], y[st][2 * j + 1]);
                unpack_e4m3(b2, j, old_scale, y[st][8 + 2 * j], y[st][9 + 2 * j]);
            }
        } else {
            unpack_slot(u1[st], u2[st], y[st]);
            if (turns && i < s.n) {
                Turn tn;
                tn.load(p, t, sl);
                if (p.interleaved) turn_slot<true>(tn, y[st]);
                else turn_slot<false>(tn, y[st]);
            }
        }
        // rows past the last one are zeros here; x * 0 is NaN where x is not finite
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            top = fmaxf(top, fabsf(y[st][j]));
            not_finite = fmaf(y[st][j], 0.f, not_finite);
        }
    }
    // entries that are not finite are rare: without any, nothing below looks for them
    const bool finite = __all_sync(0xffffffffu, not_finite == 0.f);
    if (!finite) {
        top = 0.f;
#pragma unroll
        for (int st = 0; st < NS; ++st)
#pragma unroll
            for (int j = 0; j < 16; ++j) top = fmaxf(top, page8_mag(y[st][j]));
    }
    top = warp_max(has_job ? top : 0.f);
    if (lane == 0) tops[warp] = top;
    __syncthreads();  // both halves have read the page and its scale before one writes
    if (!has_job) return true;
    const int e = page8_exponent(fmaxf(tops[warp], tops[warp ^ 1]));
    const float inv = exp2_int(-e);
    const uint64_t inv2 = (uint64_t)__float_as_uint(inv) << 32 | __float_as_uint(inv);
    if (lane == 0 && !(warp & 1)) *scale = exp2_int(e);
#pragma unroll
    for (int st = 0; st < NS; ++st) {
        const int r = r0 + st * ROWS;
        if (r >= kept) continue;
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 x = mul2(y[st][2 * j], y[st][2 * j + 1], inv2);
            w[j] = finite ? float2_to_e4m3x2(x.x, x.y) : page8_pair(y[st][2 * j], y[st][2 * j + 1], inv);
        }
        reinterpret_cast<uint2 *>(dst + r * D)[slot.c1] = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        reinterpret_cast<uint2 *>(dst + r * D)[slot.c2] = make_uint2(w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
    return true;
}

// Grid: (pages a sequence's rows can touch x kv_parts, then its rows; sequences),
// `per` pages or groups of rows to a CTA.
template <int D>
__global__ void __launch_bounds__(AP_THREADS, 3) append_q8_kernel(const __grid_constant__ AppendParams p, int kv_ctas,
                                                                  int kv_parts, int rows, int per) {
    __shared__ float tops[2][AP_WARPS];
    const int b = blockIdx.y, warp = threadIdx.x >> 5;
    if (p.status && blockIdx.x == 0) write_status(p, read_seq(p, b), b);
    const int x = blockIdx.x - kv_ctas;
    if (x < 0) {
        const int index = blockIdx.x / kv_parts, part = blockIdx.x - index * kv_parts;
        const int job = part * (AP_WARPS / 2) + (warp >> 1);
        // the maxima of two pages in turn: a warp may write the next page's while its
        // partner still reads this one's, and only the barrier of a page that is not
        // skipped keeps it from the one after that
        int turn = 0;
#pragma unroll 1
        for (int g = 0; g < per; ++g)
            turn ^= append_page<D>(p, b, index * per + g, job, job < 2 * p.Hkv, warp, threadIdx.x & 31, tops[turn]);
    } else {
        const int group = AP_THREADS / rows, sub = threadIdx.x / group;
#pragma unroll 1
        for (int g = 0; g < per; ++g)
            rotate_row<false>(p, b, (x * per + g) * rows + sub, threadIdx.x - sub * group, group);
    }
}

}  // namespace

cudaError_t launch_append(const AppendParams &params, bool q8, cudaStream_t stream) {
    AppendParams p = params;
    p.slots = p.R / 16 + ((p.D - p.R) / 8 + 1) / 2;
    const int rows = rows_per_cta(p, !q8);
    const long long groups = (p.N + rows - 1) / rows, pages = (p.N + PAGE - 2) / PAGE + 1;  // that N positions can touch
    const int kv_parts = q8 ? (2 * p.Hkv + AP_WARPS / 2 - 1) / (AP_WARPS / 2) : 0;
    const bool q_rows = !q8 || p.q;
    // Groups of rows, or pages, to a CTA. Many short CTAs, of which the shorter prompts of
    // a ragged batch leave some without rows, are worth taking four at a time once they
    // are seven to nine waves; with fewer, SMs run out of them. One group against four,
    // 32 + 16 heads of 128, rows of equal length (ragged) into the 8-bit cache: 16 x
    // 1500 123 against 113 us (76 against 68), 16 x 600 54 against 49 (35 against 31), 2 x
    // 2000 24.5 and 24.5 (22.2 and 22.4), 1 x 2000 12.9 against 14, 1 x 256 4.5 against
    // 9.6; bf16: 64 x 300 92 against 90 (63 against 56), 2 x 2000 23 against 24, 1 x
    // 256 3.5 against 6.9. Eight measured as four.
    int per = 1;
    if (p.N >= 256) {
        const int sms = attention_num_ctas();
        if (sms <= 0) return cudaErrorInvalidDevice;
        if (p.B * (pages * kv_parts + (q_rows ? groups : 0)) >= 28LL * sms) per = 4;
    }
    const long long row_ctas = (groups + per - 1) / per;
    if (!q8) {
        const dim3 grid((unsigned)row_ctas, (unsigned)p.B);
        if (per > 1)
            append_kernel<true><<<grid, AP_THREADS, 0, stream>>>(p, rows, per);
        else
            append_kernel<false><<<grid, AP_THREADS, 0, stream>>>(p, rows, per);
        return cudaGetLastError();
    }
    const long long kv_ctas = (pages + per - 1) / per * kv_parts;
    if (kv_ctas + row_ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)(kv_ctas + (q_rows ? row_ctas : 0)), (unsigned)p.B);
    if (p.D == 128)
        append_q8_kernel<128><<<grid, AP_THREADS, 0, stream>>>(p, (int)kv_ctas, kv_parts, rows, per);
    else
        append_q8_kernel<64><<<grid, AP_THREADS, 0, stream>>>(p, (int)kv_ctas, kv_parts, rows, per);
    return cudaGetLastError();
}

}  // namespace sv
