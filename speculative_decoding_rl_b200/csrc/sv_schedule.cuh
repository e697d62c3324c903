// The split-context schedule of the verify-attention kernels (bf16 and 8-bit
// cache) and their launch.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "sv_internal.h"
#include "sv_tc.cuh"

namespace sv {

// Running column maximum of a column that has seen no visible key: finite, so
// that s*scale - M_NONE is +huge for a visible score (it votes for a raise) and
// -inf for a masked one (p = 0), with no special case in the exponentials.
constexpr float M_NONE = -3.402823466e38f;
// Drain limit: after an abort, a role still waits this long for its own copies
// and products in flight. The limit of every other wait is AttnParams::wait_limit_ns
// (2 s; test hooks shorten it).
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;

// ---------------------------------------------------------------------------
// Schedule helpers (attention and combine kernels agree on these).
// ---------------------------------------------------------------------------
SV_DEV int seq_tiles(const AttnParams &p, int b) {
    const int C = p.ctx_lens[b];
    const bool ok = C >= p.N && C <= p.max_blocks * PAGE;
    return ok ? (C + TILE_KEYS - 1) / TILE_KEYS : 0;
}

// Schedule positions of one unit of sequence b: its tiles plus the unit's cost
// UC (here and below; the same in every kernel of a call).
template <int UC = UNIT_COST>
SV_DEV int seq_slots(const AttnParams &p, int b) {
    const int t = seq_tiles(p, b);
    return t > 0 ? t + UC : 0;
}

// Tiles of a sequence from its schedule positions.
template <int UC = UNIT_COST>
SV_DEV int real_tiles(int positions) { return positions > 0 ? positions - UC : 0; }

// Exclusive prefix of per-sequence schedule positions (seq_slots) into
// TP[0..B] (and, when CL is given, the context lengths into CL[0..B)); the
// whole block participates.
template <int UC = UNIT_COST>
SV_DEV void tile_prefix(const AttnParams &p, int *TP, int *scratch, int *CL = nullptr) {
    const int nt = blockDim.x, tid = threadIdx.x;
    const int per = (p.B + nt - 1) / nt;
    const int s0 = min(tid * per, p.B), s1 = min(s0 + per, p.B);
    int local = 0;
#pragma unroll 1
    for (int b = s0; b < s1; ++b) {
        local += seq_slots<UC>(p, b);
        if (CL) CL[b] = p.ctx_lens[b];
    }
    const int lane = tid & 31, warp = tid >> 5;
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int wpre = 0;
#pragma unroll 1
    for (int w = 0; w < warp; ++w) wpre += scratch[w];
    int run = wpre + incl - local;
#pragma unroll 1
    for (int b = s0; b < s1; ++b) {
        TP[b] = run;
        run += seq_slots<UC>(p, b);
    }
    if (tid == nt - 1) TP[p.B] = run;
    __syncthreads();
}

// Positions of a work range.
SV_DEV int schedule_width(const AttnParams &p, int total) {
    return max(max(1, p.min_width), (total + p.num_ctas - 1) / p.num_ctas);
}

// Schedule position t -> sequence b (largest b with ups*TP[b] <= t).
SV_DEV int tile_seq(const int *TP, int B, int ups, int t) {
    int lo = 0, hi = B;
#pragma unroll 1
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ups * TP[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// A tile: sequence b, head/row-chunk hr, tile j of the unit's Tb tiles.
struct TileInfo {
    int b, hr, j, Tb;
};

// The tile after ti in the end-to-end order (j, then head/row chunk, then
// sequence; sequences without tiles are skipped). Callers stop at their range's
// end, so running past the last sequence only has to be harmless.
template <int UC = UNIT_COST>
SV_DEV void next_tile(TileInfo &ti, const int *TP, int B, int ups) {
    if (++ti.j < ti.Tb) return;
    ti.j = 0;
    if (++ti.hr < ups) return;
    ti.hr = 0;
#pragma unroll 1
    do {
        ++ti.b;
        ti.Tb = ti.b < B ? real_tiles<UC>(TP[ti.b + 1] - TP[ti.b]) : 1;
    } while (ti.b < B && ti.Tb == 0);
}

// The first tile a CTA owns and how many it owns: the tiles whose schedule
// positions fall in [v0, v1) (positions past a unit's tiles hold no work).
template <int UC = UNIT_COST>
SV_DEV TileInfo cta_tiles(const int *TP, int B, int ups, int v0, int v1, int *ntiles) {
    TileInfo ti{0, 0, 0, 1};
    *ntiles = 0;
    if (v0 >= v1) return ti;
    ti.b = tile_seq(TP, B, ups, v0);
    const int T1 = TP[ti.b + 1] - TP[ti.b];  // positions per unit of b (> 0)
    const int off = v0 - ups * TP[ti.b];
    ti.hr = off / T1;
    ti.j = off - ti.hr * T1;
    ti.Tb = real_tiles<UC>(T1);
    if (ti.j >= ti.Tb) {  // a position past the unit's tiles: start at the next unit
        ti.j = ti.Tb - 1;
        next_tile<UC>(ti, TP, B, ups);
    }
    TileInfo w = ti;
    int n = 0;
#pragma unroll 1
    while (w.b < B) {
        const int pos = ups * TP[w.b] + w.hr * (w.Tb + UC) + w.j;
        if (pos >= v1) break;
        const int here = min(w.Tb - w.j, v1 - pos);
        n += here;
        w.j = w.Tb - 1;
        next_tile<UC>(w, TP, B, ups);
    }
    *ntiles = n;
    return ti;
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
constexpr int SMEM_LIMIT = 227 * 1024;

// The driver's tensor-map encoder, or null.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// Merges the partials of the units that were split over several ranges into p.out.
template <int UC = UNIT_COST>
cudaError_t launch_combine(const AttnParams &p, cudaStream_t stream);

// Launch with programmatic stream serialization: the kernel may start while the
// previous kernel in the stream finishes; it waits (griddep_wait) before it
// reads any input or writes anything.
template <typename... Args>
static cudaError_t launch_programmatic(void (*kfn)(Args...), dim3 grid, dim3 block, size_t smem,
                                       cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kfn, args...);
}

}  // namespace sv
