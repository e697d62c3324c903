// sv_kv_append, sv_kv_append_q8: rotate the new rows' q and k by their
// positions and write K and V to the paged cache, for the rows of a verify step
// or for ragged prompts.
//
// The pair (x1, x2) of a row at position t turns by the angle whose cosine and
// sine the caller's table holds: (x1 c - x2 s, x2 c + x1 s). Products and sums
// are rounded one by one (no contraction), so the result is the formula's in
// fp32, bit for bit, whatever the compiler does.
//
// The rows of a sequence are taken page by page of the cache: grid (pages a
// sequence's rows can touch, sequences, parts). In the bf16 call every part is
// one row of the page: all of its heads, 8 entries (16 bytes) per thread, a
// thread keeping its cosines and sines for the heads it takes. In the 8-bit
// call the first parts are the page's K and V, one warp to each (KV head, K or
// V), since a page's scale is the maximum over its rows; the others rotate q as
// the bf16 call does.
#include "sv_page8.cuh"
#include "sv_q8.h"

namespace sv {
namespace {

constexpr int AP_THREADS = 256;
constexpr int AP_WARPS = AP_THREADS / 32;

// What a CTA needs to know of its sequence and page.
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

// New rows [i0, i1) of sequence b on `page` and its block id (-1: the page is
// skipped, for a bad id or a bad position among those rows). Warp by warp, no
// barrier; every lane of the warp takes part.
SV_DEV int check_page(const AppendParams &p, const Seq &s, int b, int page, int *i0, int *i1) {
    const int lane = threadIdx.x & 31;
    *i0 = max(page * PAGE, s.start) - s.start;
    *i1 = min(page * PAGE + PAGE, s.C) - s.start;
    const int blk = p.block_table[(size_t)b * p.max_blocks + page];
    const int i = *i0 + lane;
    const bool bad = lane < PAGE && i < *i1 && bad_position(p, row_position(p, s, b, i));
    return __any_sync(0xffffffffu, bad) || blk < 0 || blk >= p.num_blocks ? -1 : blk;
}

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

// Heads [0, heads) of row i of sequence b, a thread per 8 entries: q to q_out,
// and (KV) k and v to their page of the bf16 cache.
template <bool KV>
SV_DEV void rotate_row(const AppendParams &p, const Seq &s, int b, int i, int blk) {
    const int chunks = p.D / 8;
    const int lanes = AP_THREADS / chunks;  // heads in flight
    const int c = threadIdx.x % chunks, h0 = threadIdx.x / chunks;
    if (h0 >= lanes) return;  // D / 8 does not divide the CTA
    Turn t;
    t.on = false;
    if (p.R > 0) t.load(p, row_position(p, s, b, i), c);
    const bool pairs = t.on && !p.interleaved;
    const size_t row = (size_t)b * p.N + i;
    const int hq = p.q ? p.Hq : 0;
    const int heads = hq + (KV ? 2 * p.Hkv : 0);
    const int at = (s.start + i) % PAGE;
#pragma unroll 4
    for (int h = h0; h < heads; h += lanes) {
        const bool is_q = h < hq, is_v = h >= hq + p.Hkv;
        const int hk = is_v ? h - hq - p.Hkv : h - hq;
        const uint16_t *src = is_q ? p.q + row * p.q_stride + (size_t)h * p.D
                                   : (is_v ? p.v : p.k) + row * p.kv_stride + (size_t)hk * p.D;
        uint4 own = __ldg(reinterpret_cast<const uint4 *>(src) + c);
        if (t.on && !is_v) {
            float x[8], o[8];
            unpack8(own, x);
            if (pairs) unpack8(__ldg(reinterpret_cast<const uint4 *>(src) + pair_chunk(p, c)), o);
            turn8(p, t, c, x, o);
            own = pack8(x);
        }
        uint16_t *dst;
        if (is_q) {
            dst = p.q_out + (row * p.Hq + h) * p.D;
        } else {
            uint16_t *pool = static_cast<uint16_t *>(is_v ? p.v_pool : p.k_pool);
            dst = pool + (((size_t)blk * p.Hkv + hk) * PAGE + at) * p.D;
        }
        reinterpret_cast<uint4 *>(dst)[c] = own;
    }
}

__global__ void __launch_bounds__(AP_THREADS) append_kernel(const __grid_constant__ AppendParams p) {
    const int b = blockIdx.y;
    const Seq s = read_seq(p, b);
    if (p.status && blockIdx.x == 0 && blockIdx.z == 0) write_status(p, s, b);
    const int page = s.start / PAGE + blockIdx.x;
    if (!s.ok || s.n == 0 || page * PAGE >= s.C) return;
    int i0, i1;
    const int blk = check_page(p, s, b, page, &i0, &i1);
    const int row = i0 + (int)blockIdx.z;  // part z is the z-th new row of the page
    if (blk >= 0 && row < i1) rotate_row<true>(p, s, b, row, blk);
}

// One page of one KV head, K or V, by a warp.
template <int D>
SV_DEV void append_page(const AppendParams &p, const Seq &s, int b, int page, int blk, int hk, bool is_v, int lane) {
    uint8_t *dst = static_cast<uint8_t *>(is_v ? p.v_pool : p.k_pool) + ((size_t)blk * p.Hkv + hk) * PAGE * D;
    float *scale = p.scales + ((size_t)blk * p.Hkv + hk) * 2 + (is_v ? 1 : 0);
    const float old_scale = page * PAGE < s.start ? *scale : 0.f;
    const uint16_t *src = is_v ? p.v : p.k;
    const int c = Page8<D>::col(lane) / 8;
    const bool pairs = !is_v && !p.interleaved && 8 * c < p.R;
    // the lane of this lane's row that holds the paired chunk
    const int mate = lane - c + (pairs ? pair_chunk(p, c) : c);
    Page8<D> pg;
#pragma unroll
    for (int st = 0; st < Page8<D>::STEPS; ++st) {
        const int r = Page8<D>::row(st, lane);
        const int t = page * PAGE + r, i = t - s.start;
        uint4 own = make_uint4(0, 0, 0, 0);
        const bool fresh = i >= 0 && i < s.n;
        if (fresh)
            own = __ldg(reinterpret_cast<const uint4 *>(src + ((size_t)b * p.N + i) * p.kv_stride + (size_t)hk * D) + c);
        else if (i < 0)
            *reinterpret_cast<uint2 *>(&own) = *reinterpret_cast<const uint2 *>(dst + r * D + 8 * c);
        float o[8];
        {
            uint4 m;
            m.x = __shfl_sync(0xffffffffu, own.x, mate);
            m.y = __shfl_sync(0xffffffffu, own.y, mate);
            m.z = __shfl_sync(0xffffffffu, own.z, mate);
            m.w = __shfl_sync(0xffffffffu, own.w, mate);
            unpack8(m, o);
        }
        if (i < 0) {
            pg.set(st, make_uint2(own.x, own.y), old_scale);
        } else {
            unpack8(own, pg.val[st]);
            if (fresh && !is_v && 8 * c < p.R) {
                Turn tn;
                tn.load(p, row_position(p, s, b, i), c);
                turn8(p, tn, c, pg.val[st], o);
            }
        }
    }
    pg.store(dst, scale, min(PAGE, s.C - page * PAGE), lane);
}

template <int D>
__global__ void __launch_bounds__(AP_THREADS) append_q8_kernel(const __grid_constant__ AppendParams p, int kv_parts) {
    const int b = blockIdx.y;
    const Seq s = read_seq(p, b);
    if (p.status && blockIdx.x == 0 && blockIdx.z == 0) write_status(p, s, b);
    const int page = s.start / PAGE + blockIdx.x;
    if (!s.ok || s.n == 0 || page * PAGE >= s.C) return;
    int i0, i1;
    const int blk = check_page(p, s, b, page, &i0, &i1);
    if (blk < 0) return;
    if ((int)blockIdx.z < kv_parts) {
        const int job = blockIdx.z * AP_WARPS + (threadIdx.x >> 5);
        if (job < 2 * p.Hkv) append_page<D>(p, s, b, page, blk, job >> 1, job & 1, threadIdx.x & 31);
        return;
    }
    const int row = i0 + (int)blockIdx.z - kv_parts;
    if (row < i1) rotate_row<false>(p, s, b, row, 0);
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, bool q8, cudaStream_t stream) {
    // pages that N consecutive positions can touch, and new rows on one of them
    const unsigned pages = (unsigned)((p.N + PAGE - 2) / PAGE + 1), rows = (unsigned)(p.N < PAGE ? p.N : PAGE);
    if (!q8) {
        append_kernel<<<dim3(pages, (unsigned)p.B, rows), AP_THREADS, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const int kv_parts = (2 * p.Hkv + AP_WARPS - 1) / AP_WARPS;
    const dim3 grid(pages, (unsigned)p.B, (unsigned)kv_parts + (p.q ? rows : 0u));
    if (p.D == 128)
        append_q8_kernel<128><<<grid, AP_THREADS, 0, stream>>>(p, kv_parts);
    else
        append_q8_kernel<64><<<grid, AP_THREADS, 0, stream>>>(p, kv_parts);
    return cudaGetLastError();
}

}  // namespace sv
