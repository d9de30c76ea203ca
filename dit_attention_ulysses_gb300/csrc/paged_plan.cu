// Division of a step's paged attention among the CTAs, on the GPU, from the lengths.
//
// A tile (a group of new tokens of one sequence and one KV head) costs the keys it
// walks plus a constant for its start and end.  The tiles, in the order (sequence, KV
// head, tile), form one line of cost.
//
// Cut part: CTA c takes a contiguous range of the line such that all CTAs end together
// however ragged the lengths are.  A range may start and end inside a tile; cuts fall on
// key blocks and leave at least `snap` blocks on both sides.
//
// Waves (tiles of 128 rows): before that, whole tiles are dealt out wave by wave, tile
// w * grid + c (or the w * grid + c-th group of `slot` tiles) to CTA c, for as many waves
// as leave every CTA below its share of the whole; the ranges make up the difference, or
// the last tiles run whole too where that costs less than cutting them.
// The CTAs then walk the keys of the same one or few KV heads at the same time, from the
// same end, and share them in L2.  One range each over the whole line had every CTA at
// another place of all heads' keys: 226 MB of them at 24 heads of 18432 keys, read at 9
// TB/s (895 us against 787 with waves, everything else alike).
//
// Costs are arithmetic series (paged_walk.cuh), so nothing per tile is stored but the
// waves' slots: one CTA scans the sequences, then its threads bisect for slots and cuts.
// What bounds it is that chain, once per step: 8.5 us for a decoding batch, 10 for 24 short
// chunks, 14 .. 16 for long ones, 23 for 8192 sequences.
#include <cuda_runtime.h>

#include <cstdint>

#include "paged.h"
#include "paged_walk.cuh"
#include "ptx.cuh"

namespace xs {
namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int MAX_RANGES = 511;
constexpr int SORTED = 4 * PLAN_THREADS;      // tiles that a plan sorts, four per thread
constexpr int SORT_ROWS = SORTED / 32;        // one per warp and turn
constexpr int SMEM_MOST = 200 * 1024;         // dynamic shared memory: 8192 sequences on 152 SMs take 172,448 bytes

// Sums over the threads before this one, and over all.
struct Sums {
    long long cost, tiles, kept;
};

__device__ __forceinline__ Sums warp_scan(Sums x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long c = __shfl_up_sync(0xffffffffu, x.cost, d), t = __shfl_up_sync(0xffffffffu, x.tiles, d);
        const int k = __shfl_up_sync(0xffffffffu, static_cast<int>(x.kept), d);
        if (lane >= d) {
            x.cost += c;
            x.tiles += t;
            x.kept += k;
        }
    }
    return x;
}

// sums: [2 PLAN_THREADS / 32 + 1]
__device__ __forceinline__ Sums block_scan(Sums v, Sums* sums, Sums& total) {
    constexpr int WARPS = PLAN_THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Sums x = warp_scan(v);
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const Sums s = lane < WARPS ? sums[lane] : Sums{0, 0, 0};
        const Sums y = warp_scan(s);
        if (lane < WARPS) sums[WARPS + lane] = Sums{y.cost - s.cost, y.tiles - s.tiles, y.kept - s.kept};
        if (lane == 31) sums[2 * WARPS] = y;
    }
    __syncthreads();
    const Sums before = sums[WARPS + warp];
    total = sums[2 * WARPS];
    return Sums{before.cost + x.cost - v.cost, before.tiles + x.tiles - v.tiles, before.kept + x.kept - v.kept};
}

// Last i in [0, n) with p[i] <= x.
template <typename T>
__device__ __forceinline__ int find(const T* p, int n, long long x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(PLAN_THREADS) paged_plan_kernel(const __grid_constant__ PagedPlanArgs a) {
    extern __shared__ __align__(16) long long prefix[];   // [n + 1] cost before each kept sequence (all KV heads)
    long long* tiles = prefix + a.n + 1;                  // [n + 1] tiles before it
    PagedPos* cut = reinterpret_cast<PagedPos*>(tiles + a.n + 1);      // [grid + 1]
    unsigned* slot_cost = reinterpret_cast<unsigned*>(cut + a.tile.grid + 1);   // [grid][waves]
    __shared__ long long cut_key[MAX_RANGES + 1];         // order of a cut: twice its tile, plus one inside the tile
    __shared__ Sums warp_sums[PLAN_THREADS / 16 + 1];
    __shared__ int waves_min, longest, most_keys, most_new;
    __shared__ __align__(16) unsigned short sorter[32 * SORT_ROWS];   // [step of cost][row]: tiles before a row's
    __shared__ int step_tiles[32];
    const int tid = threadIdx.x;

    pdl_launch();
    pdl_wait();
    PagedTiling keys_only = a.tile;
    keys_only.start_cost = 0;
    long long total = 0, all_tiles = 0;
    int kept = 0;
    int my_keys = 0, my_new = 0;
    if (tid == 0) longest = most_keys = most_new = 0;
    for (int i0 = 0; i0 < a.n; i0 += PLAN_THREADS) {
        const int i = i0 + tid;
        PagedSeq s{0, 0, 0, i};
        if (i < a.n) {
            const int q0 = a.cu_q[i], q1 = a.cu_q[i + 1], kv = a.kv_lens[i];
            s.q_start = q0 > 0 ? q0 : 0;
            s.q_len = q1 > s.q_start ? q1 - s.q_start : 0;
            s.kv_len = kv > 0 ? kv : 0;
        }
        const int mine = s.q_len > 0 ? paged_tiles(s, a.tile.tokens) : 0;
        const long long cost = mine > 0 ? a.Hkv * paged_cost(s, mine, keys_only, a.causal, a.window) : 0;
        Sums all;
        const Sums before = block_scan(Sums{cost, static_cast<long long>(mine) * a.Hkv, mine > 0 ? 1 : 0}, warp_sums, all);
        if (mine > 0) {
            const int at = kept + static_cast<int>(before.kept);
            prefix[at] = total + before.cost;
            tiles[at] = all_tiles + before.tiles;
            a.work.seqs[at] = s;
            my_keys = max(my_keys, s.kv_len);
            my_new = max(my_new, s.q_len);
        }
        total += all.cost;
        all_tiles += all.tiles;
        kept += static_cast<int>(all.kept);
    }
    my_keys = __reduce_max_sync(0xffffffffu, my_keys);
    my_new = __reduce_max_sync(0xffffffffu, my_new);
    if ((tid & 31) == 0) {   // (the scans have synchronised; the threads meet again before these are read)
        atomicMax(&most_keys, my_keys);
        atomicMax(&most_new, my_new);
    }
    // Few keys per CTA: the time is latency, and short pieces of many CTAs beat long ones of some,
    // though their parts take longer to join
    PagedTiling tile = a.tile;
    const bool few = a.tile.waves == 0 && total < static_cast<long long>(a.tile.grid) * a.tile.few_keys;
    if (few) {
        tile.start_cost = a.tile.few_start_cost;
        tile.least = a.tile.few_least;
    }
    if (tid == 0) {
        prefix[kept] = total;
        tiles[kept] = all_tiles;
        waves_min = a.tile.waves;
    }
    const long long keys = total, heads = static_cast<long long>(kept) * a.Hkv;
    total += all_tiles * tile.start_cost;
    __syncthreads();   // the prefix sums, and the sequences written by other threads of this CTA
    for (int i = tid; i <= kept; i += PLAN_THREADS) prefix[i] += tiles[i] * tile.start_cost;
    __syncthreads();

    // As many CTAs as there is work for, but one per tile while there are CTAs.  At two blocks per range no two
    // cuts fall on one block inside a tile (on a tile's start they may: a range is then empty).
    const int grid = a.tile.grid;
    const long long least = tile.least;
    // A CTA's part of the longest tile takes time as its keys do, the join of that tile as the parts do: the sum
    // is least at sqrt(join * keys) keys to a part
    const int rows = min(most_new, a.tile.tokens) * (a.H / a.Hkv);
    const int join = a.tile.join * ((rows + a.tile.join_rows - 1) / a.tile.join_rows);
    const float span = static_cast<float>(a.window > 0 ? min(most_keys, a.window) : most_keys);
    const long long part = static_cast<long long>(sqrtf(static_cast<float>(join) * span));
    long long ranges = total > 0 ? paged_div(total, max(least, part)) : 0;
    if (ranges < all_tiles) ranges = all_tiles;
    if (ranges > grid) ranges = grid;
    // Tiles of about one length: parts that do not straddle tiles, if that leaves few enough CTAs out.  Few tokens and
    // few keys: always, in the whole batches that a join reads when there are many (1 x 6000 keys, 32 / 8 heads: 11.5
    // us with 304 parts, 10.4 with 256; 8 x 2048: 14.5 and 13.2; ragged batches lose 3 .. 10 % by it).  Chunks: if no
    // CTA gets more work than half a cut costs (64 tokens over 16384 keys, 32 / 8 heads: 36 .. 38 us with 152 parts,
    // 33 .. 37.4 with 144; 100 over 30100, 16 / 2, two sequences: 59 and 57; but 1000 over 21000, 4 / 4: 48 and,
    // with 128, 51)
    if (all_tiles > 0 && ranges >= 2 * all_tiles && 16.0f * span * all_tiles <= 17.0f * keys) {
        const long long even = ranges / all_tiles * all_tiles;
        if (a.tile.waves > 0) {
            if (paged_div(total, even) - paged_div(total, ranges) <= tile.one_each / 2) ranges = even;
        } else if (few && ranges >= 16 * all_tiles) {
            ranges = (ranges + 8 * all_tiles) / (16 * all_tiles) * (16 * all_tiles);
            while (ranges > grid) ranges -= 16 * all_tiles;
        } else if (few && ranges >= 3 * all_tiles) {
            ranges = even;
        }
    }
    if (ranges * 2 * tile.block > total) ranges = total > 0 ? paged_div(total, 2 * tile.block) : 0;
    if (ranges < 1) ranges = kept > 0 ? 1 : 0;

    // ---- waves
    // They pay where several tiles share a head's keys: four and more, or two if all keys together do not stay
    // in L2 anyway (with few tiles and few keys a range runs a head's tiles one after the other).  The rest is
    // cut, or runs whole as a last, partial wave, if that takes a CTA little longer than its share: a cut tile
    // costs 8 us, and CTAs at other places of more keys than L2 holds wait for DRAM (8 x 64 new tokens over 8192
    // keys, 32 / 8 heads, two tiles to a head: 87 us cut, 74 whole; 8 x 96: 142 and 101; 8 x 128, whose last
    // wave is nearly empty: 131 and 135).  Up to SORTED tiles are tried whole whatever they share.
    int waves = 0, slot_ctas = grid;
    long long per_slot = 1;
    const long long share = ranges > 0 && total > 0 ? paged_div(total, ranges) : 0;   // of every CTA
    const int key_bytes = a.D * (a.tile.cache8 ? 2 : 4);   // of K and V
    const bool spilling = all_tiles > 0 && paged_div(keys, all_tiles) * heads * key_bytes > a.tile.l2_bytes;
    const bool shared = all_tiles >= 4 * heads || (spilling && all_tiles >= 2 * heads);
    if (a.tile.waves > 0 && kept > 0 && (shared || all_tiles <= SORTED)) {
        // one tile per slot, more (up to 64) where there are more tiles than slots; what is left is cut
        const long long slots = static_cast<long long>(grid) * a.tile.waves;
        per_slot = min(paged_div(all_tiles + slots - 1, slots), 64ll);
        const int most = static_cast<int>(min(paged_div(all_tiles, grid * per_slot), static_cast<long long>(a.tile.waves)));
        // per_slot == 1: all tiles, those of the partial wave too (all_tiles <= slots then)
        const int extra = per_slot == 1 ? static_cast<int>(all_tiles - static_cast<long long>(most) * grid) : 0;
        const int last = most - (extra > 0 ? 0 : 1);   // the last wave of all tiles
        // slot of `per_slot` tiles from tile `first` on, and its cost
        auto describe = [&](long long first, long long& cost) {
            PagedSlot slot;
            cost = 0;
            long long left = per_slot, t = first;
            while (left > 0) {   // one turn per KV head that the slot touches
                const int q = find(tiles, kept, t);
                const PagedSeq s = a.work.seqs[q];
                const int of_head = paged_tiles(s, a.tile.tokens);
                const long long x = t - tiles[q];
                PagedPos p;
                p.seq = q;
                p.head = static_cast<int>(paged_div(x, of_head));
                p.tile = static_cast<int>(x - static_cast<long long>(p.head) * of_head);
                p.k = 0;
                const long long n = left < of_head - p.tile ? left : of_head - p.tile;
                if (t == first) {
                    slot.pos = p;
                    slot.seq = s;
                }
                if (per_slot == 1) {
                    int lo, hi;
                    paged_tile_keys(s, p.tile, tile.tokens, a.causal, a.window, lo, hi);
                    cost = static_cast<long long>(hi) - lo + tile.start_cost;
                } else {
                    cost += paged_cost(s, p.tile + n, tile, a.causal, a.window) -
                            paged_cost(s, p.tile, tile, a.causal, a.window);
                }
                t += n;
                left -= n;
            }
            return slot;
        };
        auto sum_up = [&]() {   // the longest CTA, and the waves that leave every CTA below its share
            __syncthreads();
            if (tid < grid) {
                long long sum = 0;
                int fit = most;
                for (int w = 0; w < most; ++w) {
                    sum += slot_cost[w * grid + tid];
                    if (sum > share - least && fit == most) fit = w;
                }
                if (tid < extra) sum += slot_cost[most * grid + tid];
                atomicMin(&waves_min, fit);   // a minimum and a maximum: the order does not matter
                atomicMax(&longest, static_cast<int>(min(sum, 0x7fffffffll)));
            }
            __syncthreads();
        };
        const long long rest = paged_div(share * extra, all_tiles);
        const long long spare = max(static_cast<long long>(tile.one_each), shared && spilling ? 3 * rest / 8 : 0ll);
        bool whole = per_slot == 1 && last < a.tile.waves;
        if (whole && all_tiles <= SORTED) {
            // Few tiles: by falling cost (in 32 steps of the greatest, stable), the waves in turn from the first and
            // from the last CTA on, so that a CTA's long and short tiles even out.  24 ragged chunks of up to 9
            // blocks a tile, two tiles to a CTA: 17 us, 23 as cut ranges; causal prompts of 1024 / 2048 / 4608
            // tokens: 17.5 / 40 / 112 us, in the line's order with cuts 21 / 49 / 124; four of 2048: 141 and 152.
            const int warp = tid >> 5, lane = tid & 31, count = static_cast<int>(all_tiles);
            int most_cost = 0;
#pragma unroll 1
            for (int i = tid; i < count; i += PLAN_THREADS) {
                long long cost;
                describe(i, cost);
                slot_cost[i] = static_cast<unsigned>(min(cost, 0x7fffffffll));
                most_cost = max(most_cost, static_cast<int>(slot_cost[i]));
            }
            most_cost = __reduce_max_sync(0xffffffffu, most_cost);
            if (lane == 0) atomicMax(&longest, most_cost);
            for (int i = tid; i < 32 * SORT_ROWS / 2; i += PLAN_THREADS) reinterpret_cast<unsigned*>(sorter)[i] = 0;
            __syncthreads();
            constexpr int EACH = SORTED / PLAN_THREADS;
            unsigned cost[EACH];
            int place[EACH];   // first step and tiles before this one in its warp, then the slot
#pragma unroll
            for (int j = 0; j < EACH; ++j) {
                const int i = tid + j * PLAN_THREADS;
                cost[j] = i < count ? slot_cost[i] : 0;
                const int key = i < count ? 31 - static_cast<int>(paged_div(31ll * cost[j], longest)) : 32;
                const unsigned peers = __match_any_sync(0xffffffffu, key);
                const int before = __popc(peers & ((1u << lane) - 1));
                if (key < 32 && before == 0)
                    sorter[key * SORT_ROWS + j * 32 + warp] = static_cast<unsigned short>(__popc(peers));
                place[j] = key << 8 | before;
            }
            __syncthreads();
            {   // warp b: step b, from row to row
                unsigned short* const row = sorter + warp * SORT_ROWS + lane * EACH;
                int n[EACH], sum = 0;
#pragma unroll
                for (int j = 0; j < EACH; ++j) sum += n[j] = row[j];
                int at = sum;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, at, d);
                    if (lane >= d) at += y;
                }
                if (lane == 31) step_tiles[warp] = at;
                at -= sum;
#pragma unroll
                for (int j = 0; j < EACH; ++j) {
                    row[j] = static_cast<unsigned short>(at);
                    at += n[j];
                }
            }
            __syncthreads();
            if (warp == 0) {
                const int n = step_tiles[lane];
                int at = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, at, d);
                    if (lane >= d) at += y;
                }
                step_tiles[lane] = at - n;
                if (lane == 0) longest = 0;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < EACH; ++j) {
                if (tid + j * PLAN_THREADS >= count) continue;
                const int key = place[j] >> 8;
                const int rank = step_tiles[key] + sorter[key * SORT_ROWS + j * 32 + warp] + (place[j] & 255);
                const int w = rank / grid, i = rank - w * grid;
                place[j] = w * grid + (((last - w) & 1) ? grid - 1 - i : i);
                slot_cost[place[j]] = cost[j];
            }
            sum_up();
            whole = longest <= share + spare;
            if (!whole && shared) {   // back to the line
                __syncthreads();
                if (tid == 0) {
                    longest = 0;
                    waves_min = a.tile.waves;
                }
#pragma unroll
                for (int j = 0; j < EACH; ++j) {
                    const int i = tid + j * PLAN_THREADS;
                    if (i < count) slot_cost[i] = cost[j];
                }
                sum_up();
            }
            if (whole) {   // the costs have done their work
                __syncthreads();
#pragma unroll
                for (int j = 0; j < EACH; ++j) {
                    const int i = tid + j * PLAN_THREADS;
                    if (i < count) slot_cost[i] = static_cast<unsigned>(place[j]);
                }
            }
            if (whole || shared) {
#pragma unroll 1
                for (int i = tid; i < count; i += PLAN_THREADS) {
                    const int at = whole ? static_cast<int>(slot_cost[i]) : i, w = at / grid;
                    long long unused;
                    a.work.slots[static_cast<size_t>(at - w * grid) * MAX_PAGED_WAVES + w] = describe(i, unused);
                }
            }
        } else {
            for (int i = tid; i < grid * most + extra; i += PLAN_THREADS) {
                const int w = i / grid, c = i - w * grid;
                long long cost;
                a.work.slots[static_cast<size_t>(c) * MAX_PAGED_WAVES + w] = describe(i * per_slot, cost);
                slot_cost[i] = static_cast<unsigned>(min(cost, 0xffffffffll));
            }
            sum_up();
            whole = whole && longest <= share + spare;
        }
        if (whole) {
            waves = last + 1;
            if (extra > 0) slot_ctas = extra;
            ranges = 0;   // nothing is left to cut
        } else if (shared && ranges == grid && all_tiles >= grid) {
            waves = waves_min;
        }
    }
    // ---- cuts: CTA c gets its share less what its waves cost, along the rest of the line
    long long x0 = 0;   // cost of the waves' tiles
    if (waves > 0 && ranges > 0) {
        const long long t = static_cast<long long>(waves) * grid * per_slot;
        if (t >= all_tiles) {
            x0 = total;
        } else {
            const int q = find(tiles, kept, t);
            const PagedSeq s = a.work.seqs[q];
            const int of_head = paged_tiles(s, a.tile.tokens);
            const long long x = t - tiles[q], head = paged_div(x, of_head);
            x0 = prefix[q] + head * paged_cost(s, of_head, tile, a.causal, a.window) +
                 paged_cost(s, x - head * of_head, tile, a.causal, a.window);
        }
    }
    // grid <= PLAN_THREADS: one thread per CTA
    long long spent = 0;
    if (tid < ranges)
        for (int w = 0; w < waves; ++w) spent += slot_cost[w * grid + tid];
    const long long mine = tid < ranges ? share - spent : 0;
    Sums all;
    const long long before = block_scan(Sums{mine > 0 ? mine : 0, 0, 0}, warp_sums, all).cost, shares = all.cost;
    if (tid <= ranges && ranges > 0) {
        PagedPos p{kept, 0, 0, 0};
        if (tid < ranges && shares > 0) {
            // what the shares leave over (fewer than `ranges`, the remainder of the division) spread evenly
            const long long over = total - x0 - shares;
            const long long x = x0 + before + (over > 0 ? paged_div(over * tid, ranges) : 0);
            if (x < total) {
                const int q = find(prefix, kept, x);
                p = paged_locate(a.work.seqs[q], q, x - prefix[q], paged_div(prefix[q + 1] - prefix[q], a.Hkv), tile, a.Hkv, a.causal,
                                 a.window);
            }
        }
        cut[tid] = p;
        long long id = tiles[p.seq];   // (a cut at a sequence's start may name the sequence after the last)
        if (p.seq < kept) id += static_cast<long long>(p.head) * paged_tiles(a.work.seqs[p.seq], tile.tokens) + p.tile;
        cut_key[tid] = 2 * id + (p.k > 0 ? 1 : 0);
    }
    __syncthreads();
    // first cut of at least this key
    auto first_at = [&](long long key) {
        int lo = 0, hi = static_cast<int>(ranges);
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cut_key[mid] < key)
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
            if (r.start.k > 0) {
                r.c0 = first_at(cut_key[c]) - 1;       // the CTA before the tile's first inner cut starts the tile
                r.c1 = first_at(cut_key[c] + 1) - 1;   // the CTA of its last inner cut ends it
            }
            r.c1_last = r.end.k > 0 ? first_at(cut_key[c + 1] + 1) - 1 : c;
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
        h.waves = waves;
        h.slot = static_cast<int>(per_slot);
        h.slot_ctas = slot_ctas;
        h.cache8 = a.tile.cache8;
        *a.work.header = h;
    }
}

}  // namespace

cudaError_t launch_paged_plan(const PagedPlanArgs& a, cudaStream_t stream) {
    if (a.tile.grid > MAX_RANGES || a.tile.waves > MAX_PAGED_WAVES) return cudaErrorInvalidConfiguration;
    const size_t smem = static_cast<size_t>(a.n + 1) * 16 + static_cast<size_t>(a.tile.grid + 1) * sizeof(PagedPos) +
                        static_cast<size_t>(a.tile.grid) * a.tile.waves * sizeof(float);
    if (smem > SMEM_MOST) return cudaErrorInvalidConfiguration;
    if (smem > 32 * 1024) {   // (the kernel has 14 KB of its own beside these)
        // The limit is the function's, not the launch's: one constant for all, so that no thread's call takes it
        // below what another's launch needs
        const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MOST);
        if (e != cudaSuccess) return e;
    }
    return launch_overlapped(paged_plan_kernel, dim3(1), PLAN_THREADS, smem, stream, a);
}

}  // namespace xs
