// Division of a step's paged attention among the CTAs, on the GPU, from the lengths.
//
// A tile (a group of new tokens of one sequence and one KV head) costs the keys it
// walks plus a constant for its start and end.  The tiles, in the order (sequence, KV
// head, tile), form one line of cost; CTA c of `ranges` takes [c, c + 1) / ranges of
// it, so all CTAs end together however ragged the lengths are, and neighbouring CTAs
// share a sequence and head in L2.  A range may start and end inside a tile; cuts fall
// on key blocks and leave at least `snap` blocks on both sides, and a range is long
// enough that no two cuts meet.
//
// Costs are arithmetic series (paged_walk.cuh), so nothing per tile is stored: one CTA
// scans the sequences, then one thread per CTA of the attention bisects for its cut.
#include <cuda_runtime.h>

#include <cstdint>

#include "paged.h"
#include "paged_walk.cuh"

namespace xs {
namespace {

constexpr int PLAN_THREADS = 512;

__global__ void __launch_bounds__(PLAN_THREADS) paged_plan_kernel(const __grid_constant__ PagedPlanArgs a) {
    extern __shared__ long long prefix[];   // [n + 1] cost before each kept sequence (all KV heads)
    PagedPos* cut = reinterpret_cast<PagedPos*>(prefix + a.n + 1);   // [grid + 1]
    __shared__ long long warp_cost[PLAN_THREADS / 32];
    __shared__ int warp_count[PLAN_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    long long cost_before = 0;
    int kept_before = 0;
    for (int i0 = 0; i0 < a.n; i0 += PLAN_THREADS) {
        const int i = i0 + tid;
        PagedSeq s{0, 0, 0, i};
        if (i < a.n) {
            const int q0 = a.cu_q[i], q1 = a.cu_q[i + 1], kv = a.kv_lens[i];
            s.q_start = q0 > 0 ? q0 : 0;
            s.q_len = q1 > s.q_start ? q1 - s.q_start : 0;
            s.kv_len = kv > 0 ? kv : 0;
        }
        const int keep = s.q_len > 0;
        const long long cost =
            keep ? a.Hkv * paged_cost(s, paged_tiles(s, a.tile.tokens), a.tile, a.causal, a.window) : 0;
        long long x = cost;
        int k = keep;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, d);
            const int z = __shfl_up_sync(0xffffffffu, k, d);
            if (lane >= d) {
                x += y;
                k += z;
            }
        }
        if (lane == 31) {
            warp_cost[warp] = x;
            warp_count[warp] = k;
        }
        __syncthreads();
        long long cb = 0, call = 0;
        int kb = 0, kall = 0;
#pragma unroll
        for (int w = 0; w < PLAN_THREADS / 32; ++w) {
            if (w == warp) {
                cb = call;
                kb = kall;
            }
            call += warp_cost[w];
            kall += warp_count[w];
        }
        if (keep) {
            const int at = kept_before + kb + k - 1;
            prefix[at] = cost_before + cb + x - cost;
            a.work.seqs[at] = s;
        }
        cost_before += call;
        kept_before += kall;
        __syncthreads();
    }
    const int kept = kept_before;
    const long long total = cost_before;
    if (tid == 0) prefix[kept] = total;
    // every range at least twice the snap plus a start, so that cuts in one tile differ
    const long long least = static_cast<long long>(2 * a.tile.snap + 1) * a.tile.block + a.tile.start_cost;
    long long ranges = total / least;
    if (ranges > a.tile.grid) ranges = a.tile.grid;
    if (ranges < 1) ranges = kept > 0 ? 1 : 0;
    __syncthreads();   // prefix, and the seqs written by other threads of this CTA
    for (int c = tid; c <= ranges && ranges > 0; c += PLAN_THREADS) {
        PagedPos p{kept, 0, 0, 0};
        if (c == 0) p.seq = 0;
        if (c > 0 && c < ranges) {
            const long long x = total / ranges * c + total % ranges * c / ranges;
            int lo = 0, hi = kept;   // prefix[lo] <= x < prefix[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (prefix[mid] <= x)
                    lo = mid;
                else
                    hi = mid;
            }
            p = paged_locate(a.work.seqs[lo], lo, x - prefix[lo], (prefix[lo + 1] - prefix[lo]) / a.Hkv, a.tile, a.Hkv,
                             a.causal, a.window);
        }
        cut[c] = p;
    }
    __syncthreads();
    // first cut at or past p
    auto first_at = [&](const PagedPos& p) {
        int lo = 0, hi = static_cast<int>(ranges);
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (paged_before(cut[mid], p))
                lo = mid + 1;
            else
                hi = mid;
        }
        return lo;
    };
    for (int c = tid; c < a.tile.grid; c += PLAN_THREADS) {
        PagedRange r{};
        if (c < ranges) {
            r.start = cut[c];
            r.end = cut[c + 1];
            r.first = a.work.seqs[r.start.seq < kept ? r.start.seq : 0];
            PagedPos p = r.start;
            if (p.k > 0) {
                p.k = 1;
                r.c0 = first_at(p) - 1;              // the CTA before the tile's first inner cut starts the tile
                p.k = 0x7fffffff;
                r.c1 = first_at(p) - 1;              // the CTA of its last inner cut ends it
            }
            p = r.end;
            p.k = 0x7fffffff;
            r.c1_last = r.end.k > 0 ? first_at(p) - 1 : c;
        } else {
            r.start = r.end = PagedPos{kept, 0, 0, 0};
        }
        a.work.ranges[c] = r;
        a.work.counters[c] = 0;
    }
    if (tid == 0) {
        PagedHeader h{};
        h.n_seqs = kept;
        h.ranges = static_cast<int>(ranges);
        h.n = a.n;
        h.H = a.H;
        h.Hkv = a.Hkv;
        h.D = a.D;
        h.tokens = a.tile.tokens;
        h.block = a.tile.block;
        h.grid = a.tile.grid;
        h.causal = a.causal;
        h.window = a.window;
        *a.work.header = h;
    }
}

}  // namespace

cudaError_t launch_paged_plan(const PagedPlanArgs& a, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(a.n + 2) / 2 * 16 + static_cast<size_t>(a.tile.grid + 1) * sizeof(PagedPos);
    if (smem > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    paged_plan_kernel<<<1, PLAN_THREADS, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace xs
