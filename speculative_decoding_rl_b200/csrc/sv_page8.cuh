// One page (16 tokens) of one KV head of the 8-bit cache, held by a warp.
//
// A page's entries stand for e4m3 * 2^e. e is the smallest integer in
// [PAGE8_E_MIN, PAGE8_E_MAX] with max|x| <= 448 * 2^e over the rows kept whenever
// a call writes rows to the page. e4m3 is a floating-point type: multiplying by a
// power of two moves no value that stays in its normal range, from 2^-6 to 448, so
// a page can change its scale with every row that comes or goes and only entries
// below 2^-13 of the largest one lose bits.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {

constexpr int PAGE8_E_MIN = -100, PAGE8_E_MAX = 119;  // bf16's largest value is below 448 * 2^120
constexpr float PAGE8_SCALE_MIN = 7.8886090522101181e-31f;  // 2^-100

// What a page's scale counts as, to every call that reads it.
SV_DEV float page8_scale(float s) { return fmaxf(s, PAGE8_SCALE_MIN); }

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

// The e4m3 byte of x * inv, NaN for entries that are not finite.
SV_DEV uint32_t page8_pair(float a, float b, float inv) {
    a = fabsf(a) < INFINITY ? a * inv : NAN;
    b = fabsf(b) < INFINITY ? b * inv : NAN;
    return float2_to_e4m3x2(a, b);
}

// |x| where it is finite, else 0: NaN and infinities do not enter a scale.
SV_DEV float page8_mag(float x) {
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.f;
}

// A warp's view of a page: 8 consecutive entries of a row per lane and step,
// D/8 lanes to a row, so a step covers 256 consecutive bytes of the page.
template <int D>
struct Page8 {
    static constexpr int LANES_ROW = D / 8;
    static constexpr int ROWS_STEP = 32 / LANES_ROW;
    static constexpr int STEPS = PAGE / ROWS_STEP;

    SV_DEV static int row(int step, int lane) { return step * ROWS_STEP + lane / LANES_ROW; }
    SV_DEV static int col(int lane) { return lane % LANES_ROW * 8; }

    // A page's rows [0, kept). get(step, i, a, b) gives
    // entries 2i and 2i + 1 of the lane's 8 of a step in fp32.
    // Largest magnitude of the lane's entries:
    template <typename Get>
    SV_DEV static float top(int kept, int lane, Get get) {
        float amax = 0.f;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            if (row(s, lane) < kept)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a, b;
                    get(s, i, a, b);
                    amax = fmaxf(amax, fmaxf(page8_mag(a), page8_mag(b)));
                }
        return amax;
    }
    // The rows under 2^e, to `page` (16 x D bytes), but for those that are(step)
    // says are there already; rows past `kept` stay as they were.
    template <typename Get, typename Are>
    SV_DEV static void write(uint8_t *page, int e, int kept, int lane, Get get, Are are) {
        const float inv = exp2_int(-e);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int r = row(s, lane);
            if (r >= kept || are(s)) continue;
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float a, b;
                get(s, i, a, b);
                w[i] = page8_pair(a, b, inv);
            }
            *reinterpret_cast<uint2 *>(page + r * D + col(lane)) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        }
    }
};

// Entries 2i and 2i + 1 of 8 e4m3 bytes under a scale.
SV_DEV void unpack_e4m3(uint2 bytes, int i, float scale, float &a, float &b) {
    const uint32_t w = i < 2 ? bytes.x : bytes.y;
    const float2 f = e4m3x2_to_float2(i & 1 ? w >> 16 : w);
    a = f.x * scale;
    b = f.y * scale;
}

}  // namespace sv
