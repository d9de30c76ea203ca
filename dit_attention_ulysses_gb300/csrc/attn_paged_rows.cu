// Attention of a few new tokens over a paged cache: up to 16 packed query rows per KV
// head (single tokens and short drafts of grouped-query models).
//
//   O = sum_t 2^(c s_t - m) V_t / sum_t 2^(c s_t - m),  s_t = <Q, K_t>,
//   c = scale log2(e),  m = the running maximum of c s_t,  lse = (m + log2 l) ln 2,
//
// t over the keys that the row sees.  One pass over K and V.
//
// What bounds it: the bytes of K and V.  Each is used by the 16 packed rows of
// its KV head only (2 to 16 flops per byte), so the matrix instructions are mma.sync on
// one m16 tile: a tcgen05 tile of 128 rows would leave 7 of 8 rows of its softmax unused,
// and this work has no other use for tensor memory.  What counts is bytes in flight
// and short tails:
//   * 2 CTAs of 4 warps per SM.  A warp walks every fourth group of 32 keys of its CTA's
//     piece on its own, with its own ring of 32-key slots that TMA fills (8 KB each at
//     D = 128, three per warp: 190 KB in flight or in use per SM), its own running
//     maximum, sum and accumulators, so nothing in the key loop waits for another warp;
//     the four partial results meet in shared memory once per piece.
//   * The work is cut by cost, not by tile (paged_plan.cu): all CTAs end together for any
//     mix of lengths.  Pieces of a cut tile go to the workspace; the last CTA to finish
//     one reads them back in CTA order (the sum does not depend on who is last) and
//     stores the tile.  No CTA waits for another.
//   * Page numbers are read 16 groups ahead, 32 at a time, into the lanes' registers.
//
// Measured: 64 x 8192 keys, 8 KV heads of 128: 320 us, 6.7 TB/s, as fast as the card copies;
// 64 ragged sequences of 1 .. 16384 keys: 101 us (90 at that rate); heads of 64 side by side
// in a token: 5.4 TB/s, in pages of their own 6.1; one sequence of 64 / 1024 / 4097 keys: 4.4 /
// 7.3 / 10.3 us, of which range, page numbers and first copy take 2.9, a group of keys per
// warp 0.9, the join of the warps 0.4, and for a cut tile its count 1.0 and its parts 2.5.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "device_wait.cuh"
#include "error_words.cuh"
#include "kernels.h"
#include "paged.h"
#include "paged_rows.cuh"
#include "paged_walk.cuh"
#include "ptx.cuh"

namespace xs {
namespace {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int GROUP = 32;                  // keys of a ring slot

template <int D>
struct RowsCfg {
    static constexpr int SLOT = GROUP * D * 2;
    static constexpr int SLOTS = 3 * 128 / D;          // per warp
    static constexpr int OCTET = D / 64 * 1024;        // 8 keys of a slot: [64-channel panel][key][channel]
    static constexpr int ROWS = 16;
    static constexpr int RING = WARPS * SLOTS * SLOT;  // 96 KB; reused to join the warps' results
    static constexpr int O_STRIDE = D + 8;             // floats; keeps the joining stores off each other's banks
    static constexpr int Q_OFF = RING;
    static constexpr int ML_OFF = Q_OFF + ROWS * D * 2;
    static constexpr int BAR_OFF = ML_OFF + WARPS * ROWS * 8;
    static constexpr int MISC_OFF = BAR_OFF + WARPS * SLOTS * 8;
    static constexpr int SMEM = MISC_OFF + 16;
    static constexpr int ALLOC = SMEM + 1024;          // alignment of the swizzled slots
    static_assert(WARPS * ROWS * O_STRIDE * 4 <= RING, "the joined results fit the ring");
    static_assert(ALLOC <= 113 * 1024, "two CTAs per SM");
};

template <int D, bool F16>
__global__ void __launch_bounds__(THREADS, 2)
    attn_paged_rows_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                           const __grid_constant__ PagedAttnArgs a) {
    using C = RowsCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF);
    volatile int* last_flag = abort_flag + 1;
    const uint32_t ring = smem_addr(smem) + warp * C::SLOTS * C::SLOT;
    const uint32_t bars = smem_addr(smem + C::BAR_OFF) + warp * C::SLOTS * 8;
    const uint32_t q_smem = smem_addr(smem + C::Q_OFF);
    float* join_o = reinterpret_cast<float*>(smem);                      // [WARPS][ROWS][O_STRIDE]
    float2* join_ml = reinterpret_cast<float2*>(smem + C::ML_OFF);       // [WARPS][ROWS]

    if (tid == 0) {
        *abort_flag = 0;
        for (int i = 0; i < WARPS * C::SLOTS; ++i) mbar_init(smem_addr(smem + C::BAR_OFF) + i * 8, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    pdl_wait();
    const PagedRange range = a.work.ranges[blockIdx.x];
    const int n_seqs = a.work.header->n_seqs;
    {
        const PagedHeader& h = *a.work.header;
        if (h.n != a.n || h.H != a.H || h.Hkv != a.Hkv || h.D != D || h.tokens != a.tile.tokens ||
            h.block != a.tile.block || h.grid != a.tile.grid || h.causal != a.causal || h.window != a.window || h.cache8 != 0) {
            if (tid == 0) report_error(XS_DEVICE_BOUNDS_CODE, PAGED_MAGIC_SITE, h.n, h.tokens, h.grid);
            return;
        }
    }
    __syncthreads();

    const int page_size = 1 << a.page_shift;
    const int box = page_size < GROUP ? page_size : GROUP;   // rows of one TMA copy: 16 or 32
    const int halves = GROUP / box;
    uint32_t item = 0;      // ring items (K and V alternately) waited for since the launch
    bool ok = true;
    PagedPos pos = range.start;
    PagedSeq seq = range.first;
    while (paged_before(pos, range.end)) {
        if (!paged_valid(pos, seq, n_seqs, a.tile.tokens, a.Hkv)) {
            if (tid == 0) report_error(XS_DEVICE_BOUNDS_CODE, PAGED_MAGIC_SITE, pos.seq, pos.head, pos.tile);
            return;
        }
        // the piece: blocks [k0, k1) of the tile
        int blk0, count, lo_tile, hi_tile;
        paged_tile_blocks(seq, pos.tile, a.tile, a.causal, a.window, blk0, count);
        paged_tile_keys(seq, pos.tile, a.tile.tokens, a.causal, a.window, lo_tile, hi_tile);
        const bool cut_end = paged_same_tile(pos, range.end);
        const int k1 = cut_end ? min(range.end.k, count) : count;
        const bool whole = pos.k == 0 && !cut_end;
        const int key0 = (blk0 + pos.k) * a.tile.block;
        const int key1 = min((blk0 + k1) * a.tile.block, hi_tile);
        const int groups_all = key1 > key0 ? (key1 - key0 + GROUP - 1) / GROUP : 0;
        const int groups = groups_all > warp ? (groups_all - warp + WARPS - 1) / WARPS : 0;   // of this warp
        const int tok0 = pos.tile * a.tile.tokens;                       // first token of the tile
        const int n_tok = min(a.tile.tokens, seq.q_len - tok0);
        const int n_rows = n_tok * a.G;
        const long long base = static_cast<long long>(seq.kv_len) - seq.q_len;
        // keys [loaded, unseen) come in with the first copy although no row of the sequence sees them
        const int unseen = paged_unseen(seq, a.window), loaded = lo_tile & ~(box - 1);
        const int* table = a.table + static_cast<long long>(seq.index) * a.table_stride;

        // group g of this warp starts at key0 + (warp + WARPS g) * GROUP
        auto key_of = [&](int g) { return key0 + (warp + WARPS * g) * GROUP; };
        // page number of half `lane & 1` of group `first + lane / 2`; -1 (read as zeros) past the keys,
        // before the window and past the table
        auto load_pages = [&](int first) -> int {
            const int g = first + (lane >> 1);
            const int key = key_of(g) + (lane & 1) * box;
            if (g >= groups || (lane & 1) >= halves || key >= seq.kv_len || key + box <= lo_tile) return -1;
            const int col = key >> a.page_shift;
            return static_cast<unsigned>(col) < static_cast<unsigned>(a.width) ? table[col] : -1;
        };
        int pages = load_pages(0), pages_next = load_pages(16);
        int page_base = 0;   // group of `pages`' first lane pair
        auto issue = [&](int i) {   // item i of the piece: K (even) or V (odd) of group i / 2
            const int g = i >> 1;
            const int from = ((g - page_base) & 15) * 2;
            const int src = g - page_base < 16 ? pages : pages_next;
            const int p0 = __shfl_sync(0xffffffffu, src, from), p1 = __shfl_sync(0xffffffffu, src, from + 1);
            const uint32_t slot = (item + i) % C::SLOTS;
            if (lane == 0) {
                const uint32_t bar = bars + slot * 8;
                mbar_arrive_expect_tx(bar, C::SLOT);
                const int row = key_of(g) & (page_size - 1);
                const uint32_t dst = ring + slot * C::SLOT;
                const CUtensorMap* m = (i & 1) ? &tv : &tk;
                const int x = pos.head * ((i & 1) ? a.v_head : a.k_head);
                tma_load_5d(dst, m, bar, x, 0, 0, row >> 3, p0);
                if (halves == 2) tma_load_5d(dst + C::SLOT / 2, m, bar, x, 0, 0, row >> 3, p1);
            }
        };
        const int items = 2 * groups;
        int issued = 0;
        for (; issued < C::SLOTS && issued < items; ++issued) issue(issued);

        // Q rows into shared memory, swizzled as TMA does; rows past the tile are zero
        for (int i = tid; i < C::ROWS * (D / 8); i += THREADS) {
            const int r = i / (D / 8), c8 = i % (D / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < n_rows) {
                int t, gh;
                fdivmod(r, a.fd_G, t, gh);
                const long long token = static_cast<long long>(seq.q_start) + tok0 + t;
                if (token < a.T)
                    v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + token * a.q_stride +
                                                        (static_cast<long long>(pos.head) * a.G + gh) * D + c8 * 8);
            }
            const int panel = c8 >> 3, cc = c8 & 7;
            *reinterpret_cast<uint4*>(smem + C::Q_OFF + panel * (C::ROWS * 128) + r * 128 + ((cc ^ (r & 7)) << 4)) = v;
        }
        __syncthreads();

        // bounds of this thread's rows (two per m16 tile), and of all rows of the tile
        int lo_row[2], hi_row[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = e * 8 + (lane >> 2);
            int t, gh;
            fdivmod(r, a.fd_G, t, gh);
            const long long p = base + tok0 + t;
            long long h = a.causal ? p + 1 : seq.kv_len, l = a.window > 0 ? p - a.window + 1 : 0;
            if (r >= n_rows || h < 0) h = 0;
            hi_row[e] = static_cast<int>(h);
            lo_row[e] = static_cast<int>(l > 0 ? l : 0);
        }
        // keys that every row sees: [all_lo, all_hi)
        const long long all_hi = a.causal ? base + tok0 + 1 : seq.kv_len;
        const long long all_lo = a.window > 0 ? base + tok0 + n_tok - a.window : 0;

        uint32_t qf[D / 16][4];
        const int q_row = (lane & 7) + ((lane >> 3) & 1) * 8;
        auto load_q = [&](int ks, uint32_t (&f)[4]) {
            const int r = q_row, cc = ks * 2 + (lane >> 4);
            ldmatrix4(q_smem + (cc >> 3) * (C::ROWS * 128) + r * 128 + (((cc & 7) ^ (r & 7)) << 4), f[0], f[1], f[2],
                      f[3]);
        };
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) load_q(ks, qf[ks]);
        float o[D / 8][4], m_run[2], l_run[2];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
        m_run[0] = m_run[1] = NO_MAX;
        l_run[0] = l_run[1] = 0.0f;

        int waited = 0;
        for (int g = 0; g < groups && ok; ++g) {
            if (g == page_base + 16) {
                pages = pages_next;
                page_base = g;
                pages_next = load_pages(g + 16);
            }
            const int key = key_of(g);
            // ---- S = Q K^T
            uint32_t slot = (item + 2 * g) % C::SLOTS, round = (item + 2 * g) / C::SLOTS;
            ok = ring_wait(bars + slot * 8, round & 1, abort_flag, a.timeout_ns, pos.seq, g);
            if (!ok) break;
            ++waited;
            float s[GROUP / 8][4];
#pragma unroll
            for (int i = 0; i < GROUP / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][e] = 0.0f;
            {
                const uint32_t kbase = ring + slot * C::SLOT;
                const int krow = ((lane >> 4) << 3) + (lane & 7);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const int cc = ks * 2 + ((lane >> 3) & 1);
                    uint32_t b[GROUP / 16][4];
#pragma unroll
                    for (int kb = 0; kb < GROUP / 16; ++kb) {
                        const int r = kb * 16 + krow;
                        ldmatrix4(kbase + (r >> 3) * C::OCTET + (cc >> 3) * 1024 + (r & 7) * 128 + (((cc & 7) ^ (r & 7)) << 4), b[kb][0],
                                  b[kb][1], b[kb][2], b[kb][3]);
                    }
#pragma unroll
                    for (int kb = 0; kb < GROUP / 16; ++kb) {
                        mma16816<F16>(s[2 * kb], qf[ks], b[kb][0], b[kb][1]);
                        mma16816<F16>(s[2 * kb + 1], qf[ks], b[kb][2], b[kb][3]);
                    }
                }
            }
            __syncwarp();   // every lane has read the slot
            if (issued < items) issue(issued++);
            // ---- softmax of the group
            const bool masked = key + GROUP > all_hi || key < all_lo;
            bool moved = false;
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = __int_as_float(0xff800000);
#pragma unroll
                for (int i = 0; i < GROUP / 8; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float x = s[i][2 * e + j] * a.c;
                        if (masked) {
                            const int t = key + i * 8 + (lane & 3) * 2 + j;
                            if (t >= hi_row[e] || t < lo_row[e]) x = __int_as_float(0xff800000);
                        }
                        s[i][2 * e + j] = x;
                        mx = fmaxf(mx, x);
                    }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                alpha[e] = 1.0f;
                if (mx - m_run[e] > RESCALE_THRESHOLD) {   // (the sum would be rounded: far from 0, up to a P of 2^16)
                    alpha[e] = ex2_approx(m_run[e] - mx);
                    m_run[e] = mx;
                    moved = true;
                }
            }
            if (__any_sync(0xffffffffu, moved)) {
                l_run[0] *= alpha[0];
                l_run[1] *= alpha[1];
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][0] *= alpha[0];
                    o[i][1] *= alpha[0];
                    o[i][2] *= alpha[1];
                    o[i][3] *= alpha[1];
                }
            }
            // P in 16 bits is the A operand of the second product (its relative rounding, half a step of
            // the type, is of the size of the output's own); the sum takes the fp32 values
            uint32_t pf[GROUP / 16][4];
#pragma unroll
            for (int kb = 0; kb < GROUP / 16; ++kb)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const float* x = s[2 * kb + hf];
                    const float p0 = ex2_approx(x[0] - m_run[0]), p1 = ex2_approx(x[1] - m_run[0]);
                    const float p2 = ex2_approx(x[2] - m_run[1]), p3 = ex2_approx(x[3] - m_run[1]);
                    l_run[0] += p0 + p1;
                    l_run[1] += p2 + p3;
                    pf[kb][2 * hf] = pack2<F16>(p0, p1);
                    pf[kb][2 * hf + 1] = pack2<F16>(p2, p3);
                }
            // ---- O += P V
            slot = (item + 2 * g + 1) % C::SLOTS;
            round = (item + 2 * g + 1) / C::SLOTS;
            ok = ring_wait(bars + slot * 8, round & 1, abort_flag, a.timeout_ns, pos.seq, g);
            if (!ok) break;
            ++waited;
            if (key + GROUP > seq.kv_len || (key < unseen && loaded < unseen)) {
                // what no row of the sequence sees holds whatever was there (rows of a page past its end, keys of a page
                // before its first row's window): 0 * NaN must not reach the sum
                const int bad = seq.kv_len > key ? min(seq.kv_len - key, GROUP) : 0;
                const int from = max(loaded - key, 0), low = max(min(unseen - key, GROUP) - from, 0);   // rows
                for (int i = lane; i < (low + GROUP - bad) * (D / 8); i += 32) {
                    const int r = i / (D / 8) + (i < low * (D / 8) ? from : bad - low), cc = i % (D / 8);
                    *reinterpret_cast<uint4*>(smem + (ring - smem_addr(smem)) + slot * C::SLOT +
                                              (r >> 3) * C::OCTET + (cc >> 3) * 1024 + (r & 7) * 128 + (cc & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();   // before the next TMA copy into the slot
                __syncwarp();
            }
            {
                const uint32_t vbase = ring + slot * C::SLOT;
                const int vrow = ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
                for (int kb = 0; kb < GROUP / 16; ++kb) {
                    const int r = kb * 16 + vrow;
#pragma unroll
                    for (int nb = 0; nb < D / 16; ++nb) {
                        const int cc = nb * 2 + (lane >> 4);
                        uint32_t b0, b1, b2, b3;
                        ldmatrix4_trans(vbase + (r >> 3) * C::OCTET + (cc >> 3) * 1024 + (r & 7) * 128 +
                                            (((cc & 7) ^ (r & 7)) << 4), b0, b1,
                                        b2, b3);
                        mma16816<F16>(o[2 * nb], pf[kb], b0, b1);
                        mma16816<F16>(o[2 * nb + 1], pf[kb], b2, b3);
                    }
                }
            }
            __syncwarp();
            if (issued < items) issue(issued++);
        }
        if (!ok)   // copies in flight land before the ring is written or the CTA ends
            for (int i = waited; i < issued; ++i)
                drain_wait(bars + ((item + i) % C::SLOTS) * 8, ((item + i) / C::SLOTS) & 1, 20000000ull);
        item += items;

        if (cut_end) pdl_launch();   // the end is near

        // ---- join the warps
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 1);
            l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 2);
        }
        __syncthreads();   // every warp is done with its ring
        if (*abort_flag) return;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = e * 8 + (lane >> 2);
            if (r >= n_rows) continue;
            if ((lane & 3) == 0) join_ml[warp * C::ROWS + r] = make_float2(m_run[e], l_run[e]);
            float* d = join_o + (warp * C::ROWS + r) * C::O_STRIDE + (lane & 3) * 2;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<float2*>(d + i * 8) = make_float2(o[i][2 * e], o[i][2 * e + 1]);
        }
        __syncthreads();
        // this piece's CTA slot: 2c + 1 for a piece that starts its tile, 2c for one that continues it
        const size_t part = 2 * static_cast<size_t>(blockIdx.x) + (pos.k == 0 ? 1 : 0);
        for (int i = tid; i < n_rows * (D / 4); i += THREADS) {
            const int r = i / (D / 4), c4 = i % (D / 4);
            float m = NO_MAX;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) m = fmaxf(m, join_ml[w * C::ROWS + r].x);
            float l = 0.0f;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float2 ml = join_ml[w * C::ROWS + r];
                const float f = ex2_approx(ml.x - m);
                const float4 v = *reinterpret_cast<const float4*>(join_o + (w * C::ROWS + r) * C::O_STRIDE + c4 * 4);
                l += ml.y * f;
                acc.x += v.x * f;
                acc.y += v.y * f;
                acc.z += v.z * f;
                acc.w += v.w * f;
            }
            if (whole) {
                int t, gh;
                fdivmod(r, a.fd_G, t, gh);
                const int token = seq.q_start + tok0 + t;
                if (token < a.T) store_out<F16>(a, token, pos.head * a.G + gh, c4, acc, m, l);
            } else {
                *reinterpret_cast<float4*>(a.work.part_o + (part * C::ROWS + r) * D + c4 * 4) = acc;
                if (c4 == 0) a.work.part_ml[part * C::ROWS + r] = make_float2(m, l);
            }
        }
        if (!whole) {
            const int c0 = pos.k == 0 ? static_cast<int>(blockIdx.x) : range.c0;
            const int c1 = pos.k == 0 ? range.c1_last : range.c1;
            if (c0 < 0 || c1 < c0 || c1 >= a.tile.grid) {
                if (tid == 0) report_error(XS_DEVICE_BOUNDS_CODE, PAGED_MAGIC_SITE, c0, c1, pos.tile);
                return;
            }
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const unsigned n_parts = static_cast<unsigned>(c1 - c0 + 1);
                const bool last = atomicAdd(a.work.counters + c0, 1u) + 1u == n_parts;
                if (last) a.work.counters[c0] = 0;   // for the next launch on this plan
                *last_flag = last ? 1 : 0;
            }
            __syncthreads();
            if (*last_flag) {
                __threadfence();   // the other CTAs' parts, published before their counts
                join_parts<D, C::ROWS, THREADS, 1, F16>(a, seq.q_start + tok0, pos.head, n_rows, c0, c1);
            }
        }
        fence_proxy_async_smem();   // the joined results before the next copies into the ring
        __syncthreads();
        if (cut_end) break;
        if (paged_next(pos, seq, a.tile.tokens, a.Hkv) && paged_before(pos, range.end) && pos.seq < n_seqs)
            seq = a.work.seqs[pos.seq];
    }
}

template <int D, bool F16>
cudaError_t launch_rows(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, cudaStream_t stream) {
    auto kern = attn_paged_rows_kernel<D, F16>;
    const int smem = RowsCfg<D>::ALLOC;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kern, dim3(static_cast<unsigned>(a.tile.grid)), THREADS, smem, stream, tk, tv, a);
}

}  // namespace

cudaError_t launch_attn_paged_rows(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, int dtype,
                                   cudaStream_t stream) {
    if (a.D == 128) return dtype == 0 ? launch_rows<128, false>(tk, tv, a, stream) : launch_rows<128, true>(tk, tv, a, stream);
    return dtype == 0 ? launch_rows<64, false>(tk, tv, a, stream) : launch_rows<64, true>(tk, tv, a, stream);
}

cudaError_t paged_rows_error_words(ErrorWords* w) { return error_words_here(w); }

cudaError_t read_and_clear_paged_rows_error(int* value, DeviceErrorInfo* info, int* drain_failed, unsigned long long* when) {
    return read_and_clear_error_words(value, info, drain_failed, when);
}

}  // namespace xs
