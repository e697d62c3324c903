// sv_kv_commit_q8: keep the root and the accepted draft nodes of every
// sequence, compacted behind the root in path order, in every layer and KV head
// of the 8-bit cache.
//
// A row that moves to another page comes under another scale, so a page that
// receives a row is rebuilt: its kept rows, each from where it was, under the
// smallest power of two that holds them. One CTA per (sequence, KV head,
// layer); a warp for each page that can receive a row and K or V holds that
// page's 16 rows in registers, and the CTA writes after every warp has read (a
// destination can be another move's source).
#include "sv_page8.cuh"
#include "sv_q8.h"

namespace sv {
namespace {

template <int D>
__global__ void __launch_bounds__(320) kv_commit_q8_kernel(const __grid_constant__ CommitQ8Launch P) {
    const int b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int N = P.N, C = P.ctx_lens[b], a = P.accept_len[b];
    const int *tbl = P.block_table + (size_t)b * P.max_blocks;
    const int *path = P.accept_path + (size_t)b * (N > 1 ? N - 1 : 1);
    int f = 0;
    if (C < N || C > P.max_blocks * PAGE) f |= SV_FLAG_BAD_CONTEXT;
    if (!f)
        for (int pg = (C - N) / PAGE; pg <= (C - 1) / PAGE; ++pg)
            if (tbl[pg] < 0 || tbl[pg] >= P.num_blocks) { f |= SV_FLAG_BAD_BLOCK; break; }
    int k0 = a;  // first accepted node that moves; all later ones move too
    if (a < 0 || a > N - 1) {
        f |= SV_FLAG_BAD_PATH;
    } else {
        for (int k = 0, prev = 0; k < a; ++k) {
            const int node = path[k];
            if (node < 1 || node > N - 1 || node <= prev) { f |= SV_FLAG_BAD_PATH; break; }
            if (node != k + 1 && k0 == a) k0 = k;
            prev = node;
        }
    }
    if (h == 0 && blockIdx.z == 0 && tid == 0) {
        P.new_ctx[b] = f ? C : C - N + 1 + a;
        if (P.status) P.status[b] = f;
    }
    if (f || k0 == a) return;

    const sv_kv_q8 &layer = P.layer[blockIdx.z];
    const int root = C - N, last = root + a;  // the last position kept
    const int page = (root + 1 + k0) / PAGE + (warp >> 1);
    const bool is_v = warp & 1, mine = page <= last / PAGE;
    uint8_t *pool = static_cast<uint8_t *>(is_v ? layer.v_pool : layer.k_pool);
    Page8<D> pg;
    if (mine) {
#pragma unroll
        for (int st = 0; st < Page8<D>::STEPS; ++st) {
            const int t = page * PAGE + Page8<D>::row(st, lane);
            if (t > last) continue;
            const int src = t > root + k0 ? root + path[t - root - 1] : t;
            const size_t at = (size_t)tbl[src / PAGE] * P.Hkv + h;
            pg.set(st,
                   *reinterpret_cast<const uint2 *>(pool + (at * PAGE + src % PAGE) * D + Page8<D>::col(lane)),
                   layer.scales[2 * at + is_v]);
        }
    }
    __syncthreads();
    if (mine) {
        const size_t at = (size_t)tbl[page] * P.Hkv + h;
        pg.store(pool + at * PAGE * D, layer.scales + 2 * at + is_v, min(PAGE, last + 1 - page * PAGE), lane);
    }
}

}  // namespace

cudaError_t launch_kv_commit_q8(const CommitQ8Launch &c, cudaStream_t stream) {
    // pages that N - 1 consecutive positions can touch, two warps each (at most 10 for N = 64)
    const unsigned pages = (unsigned)((c.N - 1 + PAGE - 2) / PAGE + 1);
    const dim3 grid((unsigned)c.B, (unsigned)c.Hkv, (unsigned)c.L);
    if (c.D == 128)
        kv_commit_q8_kernel<128><<<grid, 64 * pages, 0, stream>>>(c);
    else
        kv_commit_q8_kernel<64><<<grid, 64 * pages, 0, stream>>>(c);
    return cudaGetLastError();
}

}  // namespace sv
