// sv_kv_commit_q8: keep the root and the accepted draft nodes of every
// sequence, compacted behind the root in path order, in every layer and KV head
// of the 8-bit cache.
//
// A row that moves to another page comes under another scale, so a page that
// receives a row is rebuilt: its kept rows, each from where it was, under the
// smallest power of two that holds them. A job is K or V of one (sequence,
// layer, KV head); a warp holds one page of it in registers and goes over the
// pages in ascending order. Rows only move down (path[k] >= k + 1), so what a
// page still has to give goes to itself or to a page before it, and no warp
// waits for another.
//
// The call moves little; what bounds it is the chain of loads (lengths and
// path, then block ids, then rows and scales) and the number of warps that run
// through it. A warp therefore does all jobs it is given after one walk of the
// first two steps, as many as make the grid fill the SMs about once. Rows that
// stay under a scale that stays are read for the scale, but not written.
// Measured: 64 paths of a draft tree in 48 layers of 4 heads (25.7 MB of rows that
// the rebuilt pages keep, 4.2 MB of them moved) 28.3 us, 26 in short runs; one path
// in 28 layers 4.0 us.
#include "sv_page8.cuh"
#include "sv_q8.h"

namespace sv {
namespace {

constexpr int CQ_WARPS = 8;

template <int D>
__global__ void __launch_bounds__(32 * CQ_WARPS, 3) kv_commit_q8_kernel(const __grid_constant__ CommitQ8Launch P,
                                                                     int stride) {
    const int b = blockIdx.x, lane = threadIdx.x & 31;
    const int first = blockIdx.y * CQ_WARPS + (threadIdx.x >> 5);
    const int N = P.N, C = P.ctx_lens[b], a = P.accept_len[b];
    // path[k] in lane k % 32
    const int *path = P.accept_path + (size_t)b * (N > 1 ? N - 1 : 1);
    const int n0 = lane < N - 1 ? path[lane] : 0, n1 = lane + 32 < N - 1 ? path[lane + 32] : 0;
    auto node = [&](int k) {  // any k in [0, 64); all lanes take part
        const int x = __shfl_sync(0xffffffffu, n0, k & 31), y = __shfl_sync(0xffffffffu, n1, k & 31);
        return k < 32 ? x : y;
    };
    const int root = C - N;
    int f = C < N || C > P.max_blocks * PAGE ? SV_FLAG_BAD_CONTEXT : 0;
    // block ids of the pages that hold the new rows, lane by lane (N <= 64: at most 5)
    const int page0 = f ? 0 : root / PAGE;
    int blk = 0;
    bool bad_blk = false;
    if (!f && page0 + lane <= (C - 1) / PAGE) {
        blk = P.block_table[(size_t)b * P.max_blocks + page0 + lane];
        bad_blk = blk < 0 || blk >= P.num_blocks;
    }
    if (__any_sync(0xffffffffu, bad_blk)) f |= SV_FLAG_BAD_BLOCK;
    const bool len_ok = a >= 0 && a <= N - 1;
    const int m0 = __shfl_up_sync(0xffffffffu, n0, 1), m1 = __shfl_up_sync(0xffffffffu, n1, 1);
    const int top0 = __shfl_sync(0xffffffffu, n0, 31);
    const int prev0 = lane ? m0 : 0, prev1 = lane ? m1 : top0;
    const bool bad0 = lane < a && (n0 <= prev0 || n0 > N - 1), bad1 = lane + 32 < a && (n1 <= prev1 || n1 > N - 1);
    if (!len_ok || __any_sync(0xffffffffu, bad0 || bad1)) f |= SV_FLAG_BAD_PATH;
    if (first == 0 && lane == 0) {
        P.new_ctx[b] = f ? C : C - N + 1 + a;
        if (P.status) P.status[b] = f;
    }
    if (f) return;
    // first accepted node that moves; all later ones move too
    const unsigned mv0 = __ballot_sync(0xffffffffu, lane < a && n0 != lane + 1);
    const unsigned mv1 = __ballot_sync(0xffffffffu, lane + 32 < a && n1 != lane + 33);
    if (!(mv0 | mv1)) return;
    const int k0 = mv0 ? __ffs(mv0) - 1 : 31 + __ffs(mv1);
    const int last = root + a;  // the last position kept
    const int jobs = 2 * P.Hkv * P.L;
    for (int page = (root + 1 + k0) / PAGE; page <= last / PAGE; ++page) {
        // where the rows of this lane come from: page's index among the loaded ids and row
        int from[Page8<D>::STEPS];
        uint32_t stays = 0;  // steps whose row does not move
#pragma unroll
        for (int st = 0; st < Page8<D>::STEPS; ++st) {
            const int t = page * PAGE + Page8<D>::row(st, lane);
            const int moved = root + node((t - root - 1) & 63);
            const int src = t > root + k0 && t <= last ? moved : t;
            // rows past the last one kept are not read: any place of the page will do
            const int at = t <= last ? src : page * PAGE;
            const int id = __shfl_sync(0xffffffffu, blk, at / PAGE - page0);
            stays |= (uint32_t)(at == t) << st;
            from[st] = id * PAGE + at % PAGE;  // below 2^31: num_blocks * 16 entries are within the pools
        }
        const int dst = __shfl_sync(0xffffffffu, blk, page - page0);
        const int kept = min(PAGE, last + 1 - page * PAGE);
#pragma unroll 1
        for (int j = first; j < jobs; j += stride) {
            const int is_v = j & 1, h = (j >> 1) % P.Hkv;
            const sv_kv_q8 &layer = P.layer[(j >> 1) / P.Hkv];
            uint8_t *pool = static_cast<uint8_t *>(is_v ? layer.v_pool : layer.k_pool);
            uint2 raw[Page8<D>::STEPS];
            float scale[Page8<D>::STEPS];
#pragma unroll
            for (int st = 0; st < Page8<D>::STEPS; ++st) {
                const size_t at = (size_t)(from[st] / PAGE) * P.Hkv + h;
                raw[st] = *reinterpret_cast<const uint2 *>(pool + (at * PAGE + from[st] % PAGE) * D + Page8<D>::col(lane));
                scale[st] = page8_scale(layer.scales[2 * at + is_v]);
            }
            const size_t at = (size_t)dst * P.Hkv + h;
            __syncwarp();  // every lane has read the page before one writes it
            auto get = [&](int st, int i, float &x, float &y) { unpack_e4m3(raw[st], i, scale[st], x, y); };
            const int e = page8_exponent(warp_max(Page8<D>::top(kept, lane, get)));
            if (lane == 0) layer.scales[2 * at + is_v] = exp2_int(e);
            Page8<D>::write(pool + at * PAGE * D, e, kept, lane, get,
                            [&](int st) { return stays >> st & 1 && scale[st] == exp2_int(e); });
        }
        __syncwarp();
    }
}

}  // namespace

cudaError_t launch_kv_commit_q8(const CommitQ8Launch &c, cudaStream_t stream) {
    // A warp takes every stride-th job of its sequence: one each while the warps
    // fit the SMs (24 a piece at this kernel's 80 registers), more beyond (64 paths
    // in 48 layers: 35 us in place of 72 with a CTA of its own for each job).
    const int sms = attention_num_ctas();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const long long jobs = 2LL * c.Hkv * c.L, fit = 24LL * sms;
    const long long per = (jobs * c.B + fit - 1) / fit;
    const long long warps = (jobs + per - 1) / per;
    const unsigned ctas = (unsigned)((warps + CQ_WARPS - 1) / CQ_WARPS);
    const dim3 grid((unsigned)c.B, ctas);
    const int stride = (int)ctas * CQ_WARPS;
    if (c.D == 128)
        kv_commit_q8_kernel<128><<<grid, 32 * CQ_WARPS, 0, stream>>>(c, stride);
    else
        kv_commit_q8_kernel<64><<<grid, 32 * CQ_WARPS, 0, stream>>>(c, stride);
    return cudaGetLastError();
}

}  // namespace sv
