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
// no exchange between CTAs: every CTA scans all requests itself (at most 8192, in
// shared memory), then the CTAs share the outputs out between them, one thread per
// token, per page taken and per page given back, each finding its request by
// bisection.  A page that this step hands out is never read from the table or the
// list cell that another CTA writes: it is computed again from the prefix sums and
// cells that stay as they are.
#include <cuda_runtime.h>

#include <cstdint>

#include "paged.h"

namespace xs {
namespace {

constexpr int STEP_THREADS = 512;

enum { GRANTED = 0, NO_PAGES = 1, TOO_LONG = 2, NO_ROWS = 3 };

// Exclusive prefix sum over the block's threads (64 bits), and the total.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sums, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    long long before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < STEP_THREADS / 32; ++w) {
        const long long s = warp_sums[w];
        if (w < warp) before += s;
        sum += s;
    }
    __syncthreads();   // warp_sums may be written again
    total = sum;
    return before + x - v;
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

__global__ void __launch_bounds__(STEP_THREADS) paged_step_kernel(const __grid_constant__ StepArgs a) {
    extern __shared__ int smem[];
    __shared__ long long warp_sums[STEP_THREADS / 32];
    __shared__ int taken_max;
    const int n = a.n, tid = threadIdx.x;
    int* len = smem;           // [n] cached tokens (not negative)
    int* add = len + n;        // [n] new tokens; -1: ended
    int* tok = add + n;        // [n + 1] first row
    int* need = tok + n + 1;   // [n + 1] pages needed before
    int* give = need + n + 1;  // [n + 1] pages given back before
    unsigned char* stat = reinterpret_cast<unsigned char*>(give + n + 1);   // [n]
    const int shift = a.page_shift;
    auto pages_of = [&](long long tokens) -> long long { return (tokens + (1ll << shift) - 1) >> shift; };

    for (int i = tid; i < n; i += STEP_THREADS) {
        const int c = a.cache_lens[i], x = a.new_lens[i];
        const bool bad = c < 0 || pages_of(static_cast<long long>(c > 0 ? c : 0) + (x > 0 ? x : 0)) > a.width;
        len[i] = c > 0 ? c : 0;
        add[i] = x < 0 ? (bad ? 0 : -1) : x;
        stat[i] = bad ? TOO_LONG : GRANTED;
    }
    const int list = min(max(*a.free_count, 0), a.n_pages);   // entries of the free list
    if (tid == 0) taken_max = 0;
    __syncthreads();

    // thread tid scans requests [i0, i1)
    const int per = (n + STEP_THREADS - 1) / STEP_THREADS;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    long long total;
    // pages given back
    long long v = 0;
    for (int i = i0; i < i1; ++i) v += add[i] < 0 ? pages_of(len[i]) : 0;
    long long x = block_scan(v, warp_sums, total);
    for (int i = i0; i < i1; ++i) {
        give[i] = clamp_int(x);
        x += add[i] < 0 ? pages_of(len[i]) : 0;
    }
    if (tid == 0) give[n] = clamp_int(total);
    const long long given_all = total;
    const int avail = static_cast<int>(min(static_cast<long long>(a.n_pages), list + given_all));
    // rows
    auto tokens = [&](int i) -> long long { return stat[i] == GRANTED && add[i] > 0 ? add[i] : 0; };
    v = 0;
    for (int i = i0; i < i1; ++i) v += tokens(i);
    x = block_scan(v, warp_sums, total);
    const bool all_rows = total <= a.rows;
    for (int i = i0; i < i1; ++i) {
        tok[i] = clamp_int(x);
        const long long t = tokens(i);
        x += t;
        if (t > 0 && x > a.rows) stat[i] = NO_ROWS;
    }
    if (tid == 0) tok[n] = clamp_int(total);
    // pages needed
    auto needed = [&](int i) -> long long {
        return stat[i] == GRANTED && add[i] > 0 ? pages_of(static_cast<long long>(len[i]) + add[i]) - pages_of(len[i])
                                                : 0;
    };
    v = 0;
    for (int i = i0; i < i1; ++i) v += needed(i);
    x = block_scan(v, warp_sums, total);
    int mine = 0;
    for (int i = i0; i < i1; ++i) {
        need[i] = clamp_int(x);
        const long long p = needed(i);
        x += p;
        if (p > 0) {
            if (x > avail)
                stat[i] = NO_PAGES;
            else
                mine = static_cast<int>(x);
        }
    }
    if (tid == 0) need[n] = clamp_int(total);
    const bool all_pages = total <= avail;
    if (mine > 0) atomicMax(&taken_max, mine);   // a maximum: the order does not matter
    if (!all_rows || !all_pages) {               // refused requests give their rows up: scan once more
        v = 0;
        for (int i = i0; i < i1; ++i) v += tokens(i);
        x = block_scan(v, warp_sums, total);
        for (int i = i0; i < i1; ++i) {
            tok[i] = clamp_int(x);
            x += tokens(i);
        }
        if (tid == 0) tok[n] = clamp_int(total);
    }
    __syncthreads();
    const int taken = taken_max, rows = tok[n];

    // page k of the step
    auto page_at = [&](int k) -> int {
        const int e = avail - 1 - k;
        if (e < list) return a.free_pages[e];
        const int q = find(give, n, e - list);
        return a.table[static_cast<long long>(q) * a.width + (e - list - give[q])];
    };
    const int gtid = blockIdx.x * STEP_THREADS + tid, gsize = gridDim.x * STEP_THREADS;
    for (int i = gtid; i < n; i += gsize) {
        const int t = static_cast<int>(tokens(i));
        a.kv_lens[i] = add[i] < 0 ? 0 : len[i] + t;
        a.cu_q[i] = tok[i];
        a.status[i] = stat[i];
    }
    if (gtid == 0) {
        a.cu_q[n] = rows;
        *a.free_count_out = avail - taken;
    }
    // pages given back, behind the list's own
    for (int e = list + gtid; e < avail; e += gsize) {
        const int q = find(give, n, e - list);
        a.free_pages[e] = a.table[static_cast<long long>(q) * a.width + (e - list - give[q])];
    }
    // pages taken, behind the request's own
    for (int k = gtid; k < taken; k += gsize) {
        const int q = find(need, n, k);
        a.table[static_cast<long long>(q) * a.width + pages_of(len[q]) + (k - need[q])] = page_at(k);
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

// One CTA per 512 rows (at most one per SM): a single CTA for a decoding batch.
cudaError_t launch_paged_step(const StepArgs& a, int num_sms, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(a.n) * 21 + 12 + 4;
    if (smem > 48 * 1024 - 256) {   // 256: the static part
        const cudaError_t e = cudaFuncSetAttribute(paged_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   MAX_PAGED_SEQS * 21 + 16);
        if (e != cudaSuccess) return e;
    }
    long long work = a.rows > a.n ? a.rows : a.n;
    long long grid = (work + STEP_THREADS - 1) / STEP_THREADS;
    if (grid > num_sms) grid = num_sms;
    paged_step_kernel<<<static_cast<unsigned>(grid), STEP_THREADS, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace xs
