// One step of a paged cache, laid out on the GPU from the requests' lengths: the
// pages that the new tokens need are taken from a free list, the block tables get
// them, and every new token gets its position and its slot.
//
//   held_i = ceil(c_i / page), need_i = ceil((c_i + a_i) / page) - held_i
//
// with c_i cached and a_i new tokens; a_i < 0 gives the request's pages back.
// Exclusive prefix sums over the requests (tokens, pages needed, pages given back)
// say which rows and which pages a request gets; page k of the step is entry
// avail - 1 - k of the free list followed by the pages given back.
//
// What bounds it: the launch and a chain of dependent steps (load the lengths,
// scan, look up, store); the bytes are a few MB at most.  So it is one launch with
// no exchange between CTAs: every CTA scans all requests itself (at most 8192: one to
// eight per thread, in registers up to 4096 requests, partly spilled above; all three sums
// in one scan), then the CTAs share the outputs out between them, one thread per token, per
// page taken and per page given back, each finding its request by bisection.  A page that this step hands out is never read from the table or the
// list cell that another CTA writes: it is computed again from the prefix sums and
// cells that stay as they are.  256 requests with one token each: 3.2 us; 4096 requests
// with 125,000 tokens: 8 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "paged.h"
#include "ptx.cuh"

namespace xs {
namespace {

enum { GRANTED = 0, NO_PAGES = 1, TOO_LONG = 2, NO_ROWS = 3 };

// Three sums over the requests before a thread's own, and over all of them.
struct Sums {
    long long rows, need, give;
};

__device__ __forceinline__ Sums warp_scan(Sums x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long r = __shfl_up_sync(0xffffffffu, x.rows, d), n = __shfl_up_sync(0xffffffffu, x.need, d),
                        g = __shfl_up_sync(0xffffffffu, x.give, d);
        if (lane >= d) {
            x.rows += r;
            x.need += n;
            x.give += g;
        }
    }
    return x;
}

// sums: [2 THREADS / 32 + 1].  One warp scans the warps' sums for all (32 warps each doing it for
// itself spent 2 us in shuffles).
template <int THREADS>
__device__ __forceinline__ Sums block_scan(Sums v, Sums* sums, Sums& total) {
    constexpr int WARPS = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Sums x = warp_scan(v);
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const Sums s = lane < WARPS ? sums[lane] : Sums{0, 0, 0};
        const Sums y = warp_scan(s);
        if (lane < WARPS) sums[WARPS + lane] = Sums{y.rows - s.rows, y.need - s.need, y.give - s.give};
        if (lane == 31) sums[2 * WARPS] = y;
    }
    __syncthreads();
    const Sums before = sums[WARPS + warp];
    total = sums[2 * WARPS];
    return Sums{before.rows + x.rows - v.rows, before.need + x.need - v.need, before.give + x.give - v.give};
}

// The request whose part [p[i], p[i+1]) of a prefix sum holds x (0 <= x < p[n]).
__device__ __forceinline__ int find(const int* p, int n, int x) {
    int lo = 0, hi = n;   // p[lo] <= x < p[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int clamp_int(long long x) { return x > 0x7fffffffll ? 0x7fffffff : static_cast<int>(x); }

// Thread tid owns requests [tid K, tid K + K).
template <int THREADS, int K>
__global__ void __launch_bounds__(THREADS) paged_step_kernel(const __grid_constant__ StepArgs a) {
    extern __shared__ int smem[];
    __shared__ Sums warp_sums[THREADS / 16 + 1];
    __shared__ int taken_max;
    const int n = a.n, tid = threadIdx.x;
    int* len = smem;           // [n] cached tokens (not negative)
    int* tok = len + n;        // [n + 1] first row
    int* need = tok + n + 1;   // [n + 1] pages needed before
    int* give = need + n + 1;  // [n + 1] pages given back before
    const int shift = a.page_shift;
    auto pages_of = [&](long long tokens) -> long long { return (tokens + (1ll << shift) - 1) >> shift; };

    pdl_launch();
    pdl_wait();
    const int list = min(max(*a.free_count, 0), a.n_pages);   // entries of the free list
    int c[K], stat[K], rows_of[K], need_of[K];
    Sums sum{0, 0, 0};
    bool ended[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const int i = tid * K + j;
        const int cached = i < n ? a.cache_lens[i] : 0, x = i < n ? a.new_lens[i] : 0;
        c[j] = max(cached, 0);
        const long long after = pages_of(static_cast<long long>(c[j]) + max(x, 0)), held = pages_of(c[j]);
        const bool bad = cached < 0 || after > a.width;
        stat[j] = bad ? TOO_LONG : GRANTED;
        ended[j] = x < 0 && !bad;
        rows_of[j] = bad ? 0 : max(x, 0);
        need_of[j] = bad ? 0 : static_cast<int>(after - held);
        sum.rows += rows_of[j];
        sum.need += need_of[j];
        sum.give += ended[j] ? held : 0;
    }
    if (tid == 0) taken_max = 0;
    Sums total;
    Sums before = block_scan<THREADS>(sum, warp_sums, total);
    const int avail = static_cast<int>(min(static_cast<long long>(a.n_pages), list + total.give));
    int taken = static_cast<int>(min(total.need, static_cast<long long>(a.n_pages)));
    if (total.rows > a.rows || total.need > avail) {   // some are refused: their rows and pages go to nobody
        Sums at = before;
        sum = Sums{0, 0, 0};
#pragma unroll
        for (int j = 0; j < K; ++j) {
            at.rows += rows_of[j];
            if (rows_of[j] > 0 && at.rows > a.rows) {
                stat[j] = NO_ROWS;
                rows_of[j] = need_of[j] = 0;
            }
            sum.need += need_of[j];
        }
        Sums all;
        at = block_scan<THREADS>(sum, warp_sums, all);
        before.need = at.need;
        total.need = all.need;
        int mine = 0;
        sum = Sums{0, 0, 0};
#pragma unroll
        for (int j = 0; j < K; ++j) {
            at.need += need_of[j];
            if (need_of[j] > 0) {
                if (at.need > avail) {
                    stat[j] = NO_PAGES;   // its pages stay counted: requests behind it that need some are refused too
                    rows_of[j] = 0;
                } else {
                    mine = static_cast<int>(at.need);
                }
            }
            sum.rows += rows_of[j];
        }
        if (mine > 0) atomicMax(&taken_max, mine);   // a maximum: the order does not matter
        before.rows = block_scan<THREADS>(sum, warp_sums, all).rows;
        total.rows = all.rows;
        taken = taken_max;   // (the scan synchronises)
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const int i = tid * K + j;
        if (i < n) {
            len[i] = c[j];
            tok[i] = clamp_int(before.rows);
            need[i] = clamp_int(before.need);
            give[i] = clamp_int(before.give);
            if (blockIdx.x == 0) {
                a.kv_lens[i] = ended[j] ? 0 : c[j] + rows_of[j];
                a.cu_q[i] = tok[i];
                a.status[i] = stat[j];
            }
        }
        before.rows += rows_of[j];
        before.need += need_of[j];
        before.give += ended[j] ? pages_of(c[j]) : 0;
    }
    const int rows = static_cast<int>(total.rows);
    if (tid == 0) {
        tok[n] = rows;
        need[n] = clamp_int(total.need);
        give[n] = clamp_int(total.give);
        if (blockIdx.x == 0) {
            a.cu_q[n] = rows;
            *a.free_count_out = avail - taken;
        }
    }
    __syncthreads();

    // page k of the step
    auto page_at = [&](int k) -> int {
        const int e = avail - 1 - k;
        if (e < list) return a.free_pages[e];
        const int q = find(give, n, e - list);
        return a.table[static_cast<long long>(q) * a.width + (e - list - give[q])];
    };
    const int gtid = blockIdx.x * THREADS + tid, gsize = gridDim.x * THREADS;
    // Pages given back, behind the list's own, then pages taken, behind the request's own: from the last
    // thread on, which has no row (a thread that had all three took the steps one after the other)
    const int given = avail - list;
    for (int z = gsize - 1 - gtid; z < given + taken; z += gsize) {
        if (z < given) {
            const int q = find(give, n, z);
            a.free_pages[list + z] = a.table[static_cast<long long>(q) * a.width + (z - give[q])];
        } else {
            const int k = z - given, q = find(need, n, k);
            a.table[static_cast<long long>(q) * a.width + pages_of(len[q]) + (k - need[q])] = page_at(k);
        }
    }
    // positions and slots
    for (long long r = gtid; r < a.rows; r += gsize) {
        int pos = 0;
        long long slot = -1;
        if (r < rows) {
            const int q = find(tok, n, static_cast<int>(r));
            pos = len[q] + static_cast<int>(r) - tok[q];
            const int col = pos >> shift;
            const int held = static_cast<int>(pages_of(len[q]));
            const int page = col < held ? a.table[static_cast<long long>(q) * a.width + col]
                                        : page_at(need[q] + col - held);
            if (page >= 0 && page < a.n_pages)
                slot = (static_cast<long long>(page) << shift) + (pos & ((1 << shift) - 1));
        }
        a.positions[r] = pos;
        a.slots[r] = slot;
    }
}

}  // namespace

template <int THREADS, int K>
static cudaError_t launch(const StepArgs& a, int num_sms, cudaStream_t stream) {
    const size_t smem = (static_cast<size_t>(a.n) * 4 + 3) * sizeof(int);
    constexpr int most = (THREADS * K * 4 + 3) * static_cast<int>(sizeof(int));
    if (most > 40 * 1024 && smem > 40 * 1024) {
        // The limit is the function's, not the launch's: one constant for all, so that no thread's call takes it
        // below what another's launch needs
        const cudaError_t e =
            cudaFuncSetAttribute(paged_step_kernel<THREADS, K>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
    }
    long long work = a.rows > a.n ? a.rows : a.n;
    if (work < a.n_pages / 8) work = a.n_pages / 8;   // ended requests may give that many pages back
    long long grid = (work + THREADS - 1) / THREADS;
    if (grid > num_sms) grid = num_sms;
    return launch_overlapped(paged_step_kernel<THREADS, K>, dim3(static_cast<unsigned>(grid)), THREADS, smem, stream, a);
}

// One CTA per 512 or 1024 rows, or pages that may come back, at most one per SM.
cudaError_t launch_paged_step(const StepArgs& a, int num_sms, cudaStream_t stream) {
    if (a.n <= 512) return launch<512, 1>(a, num_sms, stream);
    if (a.n <= 2048) return launch<1024, 2>(a, num_sms, stream);
    if (a.n <= 4096) return launch<1024, 4>(a, num_sms, stream);
    static_assert(MAX_PAGED_SEQS <= 8 * 1024, "eight requests per thread at most");
    return launch<1024, 8>(a, num_sms, stream);
}

}  // namespace xs
