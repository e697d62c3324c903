// One page (16 tokens) of one KV head of the 8-bit cache, held by a warp.
//
// A page's entries stand for e4m3 * 2^e. e is the smallest integer in
// [PAGE8_E_MIN, PAGE8_E_MAX] with max|x| <= 448 * 2^e over the rows kept, so a
// page's bytes depend on its rows alone, not on what was there before. e4m3 is
// a floating-point type: multiplying by a power of two moves no value that
// stays in its normal range, so a page can change its scale with every row that
// comes or goes at no loss.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {

constexpr int PAGE8_E_MIN = -100, PAGE8_E_MAX = 119;  // bf16's largest value is below 448 * 2^120
constexpr float PAGE8_SCALE_MIN = 7.8886090522101181e-31f;  // 2^-100

SV_DEV float exp2_int(int e) { return __int_as_float((e + 127) << 23); }  // 2^e for normal results

// Smallest e with amax <= 448 * 2^e, clamped. 448 = 1.75 * 2^8.
SV_DEV int page8_exponent(float amax) {
    const int bits = __float_as_int(amax);  // amax >= 0 and finite
    const int x = (bits >> 23) - 127;
    const int e = (bits & 0x7FFFFF) <= 0x600000 ? x - 8 : x - 7;
    return max(PAGE8_E_MIN, min(PAGE8_E_MAX, e));
}

SV_DEV float2 e4m3x2_to_float2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3);
    return __half22float2(__half2(h));
}
SV_DEV uint32_t float2_to_e4m3x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// A warp's view of a page: 8 consecutive entries of a row per lane and step,
// D/8 lanes to a row, so a step covers 256 consecutive bytes of the page.
template <int D>
struct Page8 {
    static constexpr int LANES_ROW = D / 8;
    static constexpr int ROWS_STEP = 32 / LANES_ROW;
    static constexpr int STEPS = PAGE / ROWS_STEP;
    float val[STEPS][8];

    SV_DEV static int row(int step, int lane) { return step * ROWS_STEP + lane / LANES_ROW; }
    SV_DEV static int col(int lane) { return lane % LANES_ROW * 8; }

    SV_DEV void set(int step, uint2 bytes, float scale) {
        const uint32_t w[4] = {bytes.x, bytes.x >> 16, bytes.y, bytes.y >> 16};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = e4m3x2_to_float2(w[j]);
            val[step][2 * j] = f.x * scale;
            val[step][2 * j + 1] = f.y * scale;
        }
    }

    // Scale of the rows [0, kept) and those rows written to `page` (16 x D bytes). Rows
    // past `kept` are left as they were.
    SV_DEV void store(uint8_t *page, float *scale, int kept, int lane) const {
        float amax = 0.f;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            if (row(s, lane) < kept)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float a = fabsf(val[s][j]);
                    amax = fmaxf(amax, a < INFINITY ? a : 0.f);  // NaN and infinities do not enter the scale
                }
        amax = warp_max(amax);
        const int e = page8_exponent(amax);
        const float inv = exp2_int(-e);
        if (lane == 0) *scale = exp2_int(e);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int r = row(s, lane);
            if (r >= kept) continue;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a = val[s][2 * j], b = val[s][2 * j + 1];
                a = fabsf(a) < INFINITY ? a * inv : NAN;
                b = fabsf(b) < INFINITY ? b * inv : NAN;
                w[j] = float2_to_e4m3x2(a, b);
            }
            *reinterpret_cast<uint2 *>(page + r * D + col(lane)) =
                make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        }
    }
};

}  // namespace sv
