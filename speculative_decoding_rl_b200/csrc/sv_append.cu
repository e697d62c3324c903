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
// few heads), a thread 8 entries (16 bytes) of up to AP_BATCH heads at a time and
// their cosines and sines once. K and V of the 8-bit call: a page's scale is the
// maximum over its rows, so two warps take the page of one KV head, K or V.
// Little is computed; what bounds a call is memory when there are many rows, and
// the chain of loads (length, then block id and positions, then cosines and
// sines) when there are few, so the rows themselves are asked for first.
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

// The cosines and sines that 8 entries [8c, 8c + 8) of a head turn by.
struct Turn {
    float cs[8], sn[8];  // interleaved: the first four of each
    bool on;
    SV_DEV void load(const AppendParams &p, int t, int c) {
        on = 8 * c < p.R;
        if (!on) return;
        const float *row = p.cos_sin + (size_t)t * p.R;
        const int half = p.R / 2;
        if (p.interleaved) {
            *reinterpret_cast<float4 *>(cs) = __ldg(reinterpret_cast<const float4 *>(row + 4 * c));
            *reinterpret_cast<float4 *>(sn) = __ldg(reinterpret_cast<const float4 *>(row + half + 4 * c));
        } else {
            const int j = 8 * c < half ? 8 * c : 8 * c - half;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                reinterpret_cast<float4 *>(cs)[k] = __ldg(reinterpret_cast<const float4 *>(row + j) + k);
                reinterpret_cast<float4 *>(sn)[k] = __ldg(reinterpret_cast<const float4 *>(row + half + j) + k);
            }
        }
    }
};

SV_DEV void unpack8(uint4 u, float *x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}

SV_DEV uint4 pack8(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// x: entries [8c, 8c+8) of a head; other: in the half layout the entries they pair with.
SV_DEV void turn8(const AppendParams &p, const Turn &t, int c, float *x, const float *other) {
    if (!t.on) return;
    if (p.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = x[2 * j], b = x[2 * j + 1];
            x[2 * j] = __fsub_rn(__fmul_rn(a, t.cs[j]), __fmul_rn(b, t.sn[j]));
            x[2 * j + 1] = __fadd_rn(__fmul_rn(b, t.cs[j]), __fmul_rn(a, t.sn[j]));
        }
    } else if (16 * c < p.R) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fsub_rn(__fmul_rn(x[j], t.cs[j]), __fmul_rn(other[j], t.sn[j]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(__fmul_rn(x[j], t.cs[j]), __fmul_rn(other[j], t.sn[j]));
    }
}

// Chunk that chunk c pairs with in the half layout.
SV_DEV int pair_chunk(const AppendParams &p, int c) { return 16 * c < p.R ? c + p.R / 16 : c - p.R / 16; }

constexpr int AP_BATCH = 4;

// Heads of row i of sequence b by `group` threads (whole warps): q to q_out, and
// (KV) k and v to their page of the bf16 cache.
template <bool KV>
SV_DEV void rotate_row(const AppendParams &p, int b, int i, int tid, int group) {
    const int chunks = p.D / 8;
    const int lanes = group / chunks;  // heads in flight
    const int c = tid % chunks, h0 = tid / chunks;
    const size_t row = (size_t)b * p.N + i;
    const int hq = p.q ? p.Hq : 0;
    // D / 8 need not divide the group; rows past new_lens are not read
    const int n = p.new_lens ? p.new_lens[b] : p.N;
    const int heads = h0 < lanes && i < n && i < p.N ? hq + (KV ? 2 * p.Hkv : 0) : 0;
    auto source = [&](int h) {
        const int hk = h >= hq + p.Hkv ? h - hq - p.Hkv : h - hq;
        const uint16_t *src = h < hq ? p.q + row * p.q_stride + (size_t)h * p.D
                                     : (h >= hq + p.Hkv ? p.v : p.k) + row * p.kv_stride + (size_t)hk * p.D;
        return reinterpret_cast<const uint4 *>(src);
    };
    uint4 own[AP_BATCH];
    auto fetch = [&](int h) {
#pragma unroll
        for (int k = 0; k < AP_BATCH; ++k)
            if (h + k * lanes < heads) own[k] = __ldg(source(h + k * lanes) + c);
    };
    fetch(h0);
    const Seq s = read_seq(p, b);
    if (!s.ok || i >= s.n) return;
    const PageRows pr(p, s, b, (s.start + i) / PAGE);
    const int t = __shfl_sync(0xffffffffu, pr.pos, i - pr.i0);
    Turn turn;
    turn.on = false;
    if (p.R > 0) turn.load(p, max(0, min(t, p.max_position - 1)), c);  // a position outside skips the page below
    if (!pr.ok(p)) return;
    const bool pairs = !p.interleaved && p.R > 0;  // with the chunk pair_chunk, for the chunks that turn
    const bool near = 32 % chunks == 0;            // which a lane of the warp holds
    const int pc = turn.on ? pair_chunk(p, c) : c, mate = (int)(threadIdx.x & 31) - c + pc;
    const int at = (s.start + i) % PAGE;
    const int rounds = (hq + (KV ? 2 * p.Hkv : 0) + AP_BATCH * lanes - 1) / (AP_BATCH * lanes);
#pragma unroll 1
    for (int r = 0; r < rounds; ++r) {
        const int h = h0 + r * AP_BATCH * lanes;
        if (r) fetch(h);
#pragma unroll
        for (int k = 0; k < AP_BATCH; ++k) {
            const int hh = h + k * lanes;
            const bool is_q = hh < hq, is_v = hh >= hq + p.Hkv;
            uint4 m = own[k];
            if (pairs) {
                if (near) {
                    m.x = __shfl_sync(0xffffffffu, own[k].x, mate);
                    m.y = __shfl_sync(0xffffffffu, own[k].y, mate);
                    m.z = __shfl_sync(0xffffffffu, own[k].z, mate);
                    m.w = __shfl_sync(0xffffffffu, own[k].w, mate);
                } else if (hh < heads) {
                    m = __ldg(source(hh) + pc);
                }
            }
            if (hh >= heads) continue;
            const int hk = is_v ? hh - hq - p.Hkv : hh - hq;
            if (turn.on && !is_v) {
                float x[8], o[8];
                unpack8(own[k], x);
                unpack8(m, o);
                turn8(p, turn, c, x, o);
                own[k] = pack8(x);
            }
            uint16_t *dst;
            if (is_q) {
                dst = p.q_out + (row * p.Hq + hh) * p.D;
            } else {
                uint16_t *pool = static_cast<uint16_t *>(is_v ? p.v_pool : p.k_pool);
                dst = pool + (((size_t)pr.blk * p.Hkv + hk) * PAGE + at) * p.D;
            }
            reinterpret_cast<uint4 *>(dst)[c] = own[k];
        }
    }
}

// Rows a CTA takes: as many as leave a thread no more than one batch of a row's
// heads, in whole warps.
int rows_per_cta(const AppendParams &p, bool kv) {
    const int items = ((p.q ? p.Hq : 0) + (kv ? 2 * p.Hkv : 0)) * (p.D / 8);
    int rows = 1;
    while (rows < AP_WARPS && AP_THREADS / (2 * rows) * AP_BATCH >= items && AP_THREADS / (2 * rows) >= p.D / 8) rows *= 2;
    return rows;
}

__global__ void __launch_bounds__(AP_THREADS, 4) append_kernel(const __grid_constant__ AppendParams p, int rows) {
    const int b = blockIdx.y, group = AP_THREADS / rows, sub = threadIdx.x / group;
    if (p.status && blockIdx.x == 0) write_status(p, read_seq(p, b), b);
    rotate_row<true>(p, b, blockIdx.x * rows + sub, threadIdx.x - sub * group, group);
}

// One page of one KV head, K or V, by two warps, each half of its rows; the
// whole CTA comes here for one page. tops: a float per warp.
template <int D>
SV_DEV void append_page(const AppendParams &p, int b, int index, int job, bool has_job, int warp, int lane, float *tops) {
    using Pg = Page8<D>;
    constexpr int NS = Pg::STEPS / 2;
    const Seq s = read_seq(p, b);
    const int page = s.start / PAGE + index;
    if (!s.ok || s.n == 0 || page * PAGE >= s.C) return;
    const int hk = job >> 1, S0 = (warp & 1) * NS;
    const bool is_v = job & 1;
    const uint16_t *src = (is_v ? p.v : p.k) + (size_t)b * p.N * p.kv_stride + (size_t)hk * D;
    const int c = Pg::col(lane) / 8;
    const bool turns = !is_v && 8 * c < p.R, pairs = turns && !p.interleaved;
    // the lane of this lane's row that holds the paired chunk
    const int mate = lane - c + (pairs ? pair_chunk(p, c) : c);
    const int first = page * PAGE - s.start;  // the new row on the page's row 0, if there is one
    uint4 own[NS];
#pragma unroll
    for (int st = 0; st < NS; ++st) {
        const int i = first + Pg::row(S0 + st, lane);
        own[st] = make_uint4(0, 0, 0, 0);
        if (has_job && i >= 0 && i < s.n) own[st] = __ldg(reinterpret_cast<const uint4 *>(src + i * p.kv_stride) + c);
    }
    const PageRows pr(p, s, b, page);
    if (!pr.ok(p)) return;  // the same for every warp of the CTA
    uint8_t *dst = static_cast<uint8_t *>(is_v ? p.v_pool : p.k_pool) + ((size_t)pr.blk * p.Hkv + hk) * PAGE * D;
    float *scale = p.scales + ((size_t)pr.blk * p.Hkv + hk) * 2 + (is_v ? 1 : 0);
    float val[NS][8];
    if (has_job && first < 0) {  // rows that are there already
        const float old_scale = *scale;
#pragma unroll
        for (int st = 0; st < NS; ++st) {
            const int r = Pg::row(S0 + st, lane);
            if (first + r < 0) {
                const uint2 bytes = *reinterpret_cast<const uint2 *>(dst + r * D + 8 * c);
#pragma unroll
                for (int j = 0; j < 4; ++j) unpack_e4m3(bytes, j, old_scale, val[st][2 * j], val[st][2 * j + 1]);
            }
        }
    }
#pragma unroll
    for (int st = 0; st < NS; ++st) {
        const int i = first + Pg::row(S0 + st, lane);
        float o[8];
        if (!is_v && !p.interleaved) {
            uint4 m;
            m.x = __shfl_sync(0xffffffffu, own[st].x, mate);
            m.y = __shfl_sync(0xffffffffu, own[st].y, mate);
            m.z = __shfl_sync(0xffffffffu, own[st].z, mate);
            m.w = __shfl_sync(0xffffffffu, own[st].w, mate);
            unpack8(m, o);
        }
        const int t = __shfl_sync(0xffffffffu, pr.pos, (i - pr.i0) & 31);
        if (i >= 0) {
            unpack8(own[st], val[st]);
            if (turns && i < s.n) {
                Turn tn;
                tn.load(p, t, c);
                turn8(p, tn, c, val[st], o);
            }
        }
    }
    const int kept = min(PAGE, s.C - page * PAGE);
    auto get = [&](int st, int j, float &x, float &y) {
        x = val[st][2 * j];
        y = val[st][2 * j + 1];
    };
    const float top = warp_max(has_job ? Pg::template top<NS>(S0, kept, lane, get) : 0.f);
    if (lane == 0) tops[warp] = top;
    __syncthreads();  // both halves have read the page and its scale before one writes
    if (!has_job) return;
    const int e = page8_exponent(fmaxf(tops[warp], tops[warp ^ 1]));
    if (lane == 0 && !(warp & 1)) *scale = exp2_int(e);
    Pg::template write<NS>(dst, e, S0, kept, lane, get, [](int) { return false; });
}

// Grid: (pages a sequence's rows can touch x kv_parts, then its rows; sequences).
template <int D>
__global__ void __launch_bounds__(AP_THREADS, 3) append_q8_kernel(const __grid_constant__ AppendParams p, int pages,
                                                                  int kv_parts, int rows) {
    __shared__ float tops[AP_WARPS];
    const int b = blockIdx.y, warp = threadIdx.x >> 5;
    if (p.status && blockIdx.x == 0) write_status(p, read_seq(p, b), b);
    const int x = blockIdx.x - pages * kv_parts;
    if (x < 0) {
        const int index = blockIdx.x / kv_parts, part = blockIdx.x - index * kv_parts;
        const int job = part * (AP_WARPS / 2) + (warp >> 1);
        append_page<D>(p, b, index, job, job < 2 * p.Hkv, warp, threadIdx.x & 31, tops);
    } else {
        const int group = AP_THREADS / rows, sub = threadIdx.x / group;
        rotate_row<false>(p, b, x * rows + sub, threadIdx.x - sub * group, group);
    }
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, bool q8, cudaStream_t stream) {
    const int rows = rows_per_cta(p, !q8);
    const unsigned row_ctas = (unsigned)((p.N + rows - 1) / rows);
    if (!q8) {
        append_kernel<<<dim3(row_ctas, (unsigned)p.B), AP_THREADS, 0, stream>>>(p, rows);
        return cudaGetLastError();
    }
    const int pages = (p.N + PAGE - 2) / PAGE + 1;  // that N consecutive positions can touch
    const int kv_parts = (2 * p.Hkv + AP_WARPS / 2 - 1) / (AP_WARPS / 2);
    if ((long long)pages * kv_parts + row_ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)pages * kv_parts + (p.q ? row_ctas : 0u), (unsigned)p.B);
    if (p.D == 128)
        append_q8_kernel<128><<<grid, AP_THREADS, 0, stream>>>(p, pages, kv_parts, rows);
    else
        append_q8_kernel<64><<<grid, AP_THREADS, 0, stream>>>(p, pages, kv_parts, rows);
    return cudaGetLastError();
}

}  // namespace sv
