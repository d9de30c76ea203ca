// Geometry of a paged-attention tile, shared by the plan and the attention kernels.
#pragma once

#include <cuda_runtime.h>

#include "paged.h"

namespace xs {

// a / b for a >= 0, b > 0, in 32 bits where both fit (a 64-bit division takes several times as long).
__host__ __device__ __forceinline__ long long paged_div(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return a / b;
}

__host__ __device__ __forceinline__ int paged_tiles(const PagedSeq& s, int tokens) {
    return (s.q_len + tokens - 1) / tokens;
}

// Keys [lo, hi) that some row of tile t sees, hi > lo (a tile whose rows see nothing
// gets one key, which the rows' own bounds mask).
__host__ __device__ __forceinline__ void paged_tile_keys(const PagedSeq& s, int t, int tokens, int causal, int window,
                                                         int& lo, int& hi) {
    const long long base = static_cast<long long>(s.kv_len) - s.q_len;   // position of the first new token
    const long long first = base + static_cast<long long>(t) * tokens;
    long long last = static_cast<long long>(t + 1) * tokens;
    if (last > s.q_len) last = s.q_len;
    last += base;                                                        // one past the last token's position
    long long h = causal ? last : s.kv_len;
    if (h < 1) h = 1;
    long long l = 0;
    if (window > 0 && first - window + 1 > 0) l = first - window + 1;
    hi = static_cast<int>(h);
    lo = static_cast<int>(l);
}

// Keys below it are before the window of the sequence's first new token: no row sees them.  (The first block of any
// tile may begin below it.)
__host__ __device__ __forceinline__ int paged_unseen(const PagedSeq& s, int window) {
    const long long l = static_cast<long long>(s.kv_len) - s.q_len - window + 1;
    return window > 0 && l > 0 ? static_cast<int>(l) : 0;
}

// Key blocks of tile t: blocks [first, first + count).
__host__ __device__ __forceinline__ void paged_tile_blocks(const PagedSeq& s, int t, const PagedTiling& g, int causal,
                                                           int window, int& first, int& count) {
    int lo, hi;
    paged_tile_keys(s, t, g.tokens, causal, window, lo, hi);
    first = lo / g.block;
    count = (hi + g.block - 1) / g.block - first;
}

// Sum over tiles t < m of (hi_t - lo_t + start_cost): the arithmetic series of
// paged_tile_keys with its clamps.  m <= paged_tiles.
__host__ __device__ __forceinline__ long long paged_cost(const PagedSeq& s, long long m, const PagedTiling& g,
                                                         int causal, int window) {
    const long long R = g.tokens, q = s.q_len, kv = s.kv_len > 0 ? s.kv_len : 1;
    const long long base = static_cast<long long>(s.kv_len) - q;
    long long hi = m * kv;
    if (causal) {
        long long full = m;   // tiles that end at base + (t + 1) R
        hi = 0;
        if (m > 0 && m * R > q) {
            full = m - 1;
            hi = kv;          // the last, short one ends at the sequence's end
        }
        long long z = base < 0 ? paged_div(-base, R) : 0;   // tiles whose end is not past 0: one key each
        if (z > full) z = full;
        hi += z + (full - z) * base + R * (full * (full + 1) / 2 - z * (z + 1) / 2);
    }
    long long lo = 0;
    if (window > 0) {
        const long long b = base - window + 1;    // start of tile 0, before the clamp at 0
        long long z = b <= 0 ? paged_div(-b, R) + 1 : 0;    // tiles that start at key 0
        if (z > m) z = m;
        lo = (m - z) * b + R * (m * (m - 1) / 2 - z * (z - 1) / 2);
    }
    return hi - lo + m * g.start_cost;
}

// The tile after `p`: the next tile of the KV head, the next KV head, the next sequence.
// Returns whether the sequence changed.
__host__ __device__ __forceinline__ bool paged_next(PagedPos& p, const PagedSeq& s, int tokens, int Hkv) {
    p.k = 0;
    if (++p.tile < paged_tiles(s, tokens)) return false;
    p.tile = 0;
    if (++p.head < Hkv) return false;
    p.head = 0;
    ++p.seq;
    return true;
}

__host__ __device__ __forceinline__ bool paged_same_tile(const PagedPos& a, const PagedPos& b) {
    return a.seq == b.seq && a.head == b.head && a.tile == b.tile;
}

// Whether `p` names a tile of the step (lengths whose costs overflow 64 bits can plan others).
__host__ __device__ __forceinline__ bool paged_valid(const PagedPos& p, const PagedSeq& s, int n_seqs, int tokens,
                                                     int Hkv) {
    return p.seq >= 0 && p.seq < n_seqs && p.head >= 0 && p.head < Hkv && p.tile >= 0 && p.tile < paged_tiles(s, tokens) &&
           p.k >= 0;
}

// a < b in the order of the work
__host__ __device__ __forceinline__ bool paged_before(const PagedPos& a, const PagedPos& b) {
    if (a.seq != b.seq) return a.seq < b.seq;
    if (a.head != b.head) return a.head < b.head;
    if (a.tile != b.tile) return a.tile < b.tile;
    return a.k < b.k;
}

// Where cost x of a sequence's cost * Hkv falls: a block of a tile.  Cuts closer than
// `snap` blocks to a tile's end move to that end, cuts in a tile of fewer than `whole`
// blocks to the nearer one.
__host__ __device__ __forceinline__ PagedPos paged_locate(const PagedSeq& s, int seq, long long x, long long seq_cost,
                                                          const PagedTiling& g, int Hkv, int causal, int window) {
    PagedPos p;
    p.seq = seq;
    p.head = p.tile = p.k = 0;
    if (seq_cost < 1) return p;   // lengths whose costs overflow 64 bits
    const long long head = x < 0 ? 0 : paged_div(x, seq_cost);
    p.head = head < 0 ? 0 : head < Hkv ? static_cast<int>(head) : Hkv - 1;
    long long y = x - p.head * seq_cost;
    int lo = 0, hi = paged_tiles(s, g.tokens);   // cost(lo) <= y < cost(hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (paged_cost(s, mid, g, causal, window) <= y)
            lo = mid;
        else
            hi = mid;
    }
    p.tile = lo;
    y -= paged_cost(s, lo, g, causal, window) + g.start_cost;
    int first, count;
    paged_tile_blocks(s, lo, g, causal, window, first, count);
    const long long k = y > 0 ? (y + g.block / 2) / g.block : 0;
    p.k = k > count ? count : static_cast<int>(k);
    const bool whole = count < g.whole;
    if (p.k < g.snap || (whole && 2 * p.k < count)) {
        p.k = 0;
    } else if (count - p.k < g.snap || whole) {
        paged_next(p, s, g.tokens, Hkv);
    }
    return p;
}

}  // namespace xs
