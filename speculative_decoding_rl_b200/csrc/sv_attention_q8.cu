// sv_verify_attention_q8: GQA attention of every active sequence's N draft
// query rows over its paged 8-bit KV cache (e4m3 pages under one scale each for
// K and V of a KV head).
//
// First form: one warp per output row, 32 keys at a time, a key to a lane for
// the scores and D/32 entries to a lane for the output, online softmax in fp32.
#include "sv_page8.cuh"
#include "sv_q8.h"

namespace sv {
namespace {

constexpr int AQ_WARPS = 8;

template <int D>
__global__ void __launch_bounds__(32 * AQ_WARPS) attention_q8_kernel(const AttnParams p, const float *scales) {
    __shared__ float qs[AQ_WARPS][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const int row = blockIdx.x * AQ_WARPS + warp;  // (i, hq)
    const int C = p.ctx_lens[b];
    const bool ok = C >= p.N && C <= p.max_blocks * PAGE;
    const int *tbl = p.block_table + (size_t)b * p.max_blocks;
    if (blockIdx.x == 0 && warp == 0 && p.status) {
        int bad = 0;
        if (ok)
            for (int j = lane; j < (C + PAGE - 1) / PAGE; j += 32) bad |= tbl[j] < 0 || tbl[j] >= p.num_blocks;
        bad = warp_or(bad);
        if (lane == 0) p.status[b] = ok ? (bad ? SV_FLAG_BAD_BLOCK : 0) : SV_FLAG_BAD_CONTEXT;
    }
    if (row >= p.N * p.Hq) return;
    const int i = row / p.Hq, hq = row % p.Hq, h = hq / p.G;
    uint16_t *out = p.out + (((size_t)b * p.N + i) * p.Hq + hq) * D;
    constexpr int E = D / 32;
    if (!ok) {
        for (int e = lane; e < D; e += 32) out[e] = 0;
        return;
    }
    const uint16_t *q = p.q + (((size_t)b * p.N + i) * p.Hq + hq) * D;
    for (int e = lane; e < D; e += 32) qs[warp][e] = bf16_bits_to_float(q[e]);
    __syncwarp();
    const uint8_t *kp = reinterpret_cast<const uint8_t *>(p.k_pool), *vp = reinterpret_cast<const uint8_t *>(p.v_pool);
    const uint64_t mask = p.mask ? p.mask[(size_t)b * p.N + i] : 0;
    float m = -3.402823466e38f, l = 0.f, o[E] = {};
    for (int t0 = 0; t0 < C; t0 += 32) {
        const int t = t0 + lane;
        int blk = t < C ? tbl[t / PAGE] : -1;
        if (blk >= p.num_blocks) blk = -1;
        float s = 0.f, vs = 0.f;
        if (blk >= 0) {
            const float2 sc = reinterpret_cast<const float2 *>(scales)[(size_t)blk * p.Hkv + h];
            vs = fmaxf(sc.y, PAGE8_SCALE_MIN);
            const uint8_t *kr = kp + (((size_t)blk * p.Hkv + h) * PAGE + t % PAGE) * D;
            for (int e = 0; e < D; e += 8) {
                const uint2 w = *reinterpret_cast<const uint2 *>(kr + e);
                const uint32_t u[4] = {w.x, w.x >> 16, w.y, w.y >> 16};
                for (int k = 0; k < 4; ++k) {
                    const float2 f = e4m3x2_to_float2(u[k]);
                    s = fmaf(f.x, qs[warp][e + 2 * k], s);
                    s = fmaf(f.y, qs[warp][e + 2 * k + 1], s);
                }
            }
            s *= fmaxf(sc.x, PAGE8_SCALE_MIN) * p.scale_log2;
        }
        const int nk = t - (C - p.N);
        const bool sees = t < C && (nk < 0 || (p.mask ? (mask >> nk) & 1 : nk <= i));
        if (!sees) s = -INFINITY;
        const float mx = fmaxf(m, warp_max(s));
        const float w = sees ? exp2f(s - mx) : 0.f, al = exp2f(m - mx);
        m = mx;
        l = l * al + warp_sum(w);
        for (int e = 0; e < E; ++e) o[e] *= al;
        for (int k = 0; k < 32; ++k) {
            const int kb = __shfl_sync(0xffffffffu, blk, k);
            const float wk = __shfl_sync(0xffffffffu, w, k) * __shfl_sync(0xffffffffu, vs, k);
            if (kb < 0 || !__shfl_sync(0xffffffffu, sees, k)) continue;
            const uint8_t *vr = vp + (((size_t)kb * p.Hkv + h) * PAGE + (t0 + k) % PAGE) * D + lane * E;
            for (int e = 0; e < E; e += 2) {
                const float2 f = e4m3x2_to_float2(*reinterpret_cast<const uint16_t *>(vr + e));
                o[e] = fmaf(wk, f.x, o[e]);
                o[e + 1] = fmaf(wk, f.y, o[e + 1]);
            }
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int e = 0; e < E; ++e) {
        const __nv_bfloat16 v = __float2bfloat16_rn(o[e] * inv);
        out[lane * E + e] = *reinterpret_cast<const uint16_t *>(&v);
    }
}

}  // namespace

size_t attention_q8_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int num_ctas) {
    return attention_workspace_bytes(B, N, Hq, Hkv, D, num_ctas);
}

cudaError_t launch_attention_q8(const AttnParams &p, const float *scales, cudaStream_t stream) {
    const dim3 grid((unsigned)((p.N * p.Hq + AQ_WARPS - 1) / AQ_WARPS), (unsigned)p.B);
    if (p.D == 128)
        attention_q8_kernel<128><<<grid, 32 * AQ_WARPS, 0, stream>>>(p, scales);
    else
        attention_q8_kernel<64><<<grid, 32 * AQ_WARPS, 0, stream>>>(p, scales);
    return cudaGetLastError();
}

}  // namespace sv
