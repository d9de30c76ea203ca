// Attention of chunks of new tokens over a paged cache on the tcgen05 tensor cores.
//
//   O = sum_t 2^(c s_t - m) V_t / sum_t 2^(c s_t - m),  s_t = <Q, K_t>,
//   c = scale log2(e),  m = a running maximum of c s_t,  lse = (m + log2 l) ln 2,
//
// t over the keys that the row sees.  One pass over K and V in blocks of 128 keys.
//
// What bounds it: for chunks the two products (4 D flops per seen row, head and key) and
// the exponentials between them, which run at about the same time per block; for tiles
// with few rows the bytes of K and V.
//
// A tile is 128 packed query rows of one KV head: `tokens` new tokens, the G query heads
// of a token side by side, so a K/V block is loaded once for all heads that share it and
// the diagonal of a causal chunk wastes 128 / G keys per tile instead of 128.  Q comes in
// by one 4-D TMA box (64 channels x G heads x tokens) per 64 channels.
//
// Organisation (one persistent CTA per SM, 12 warps, as in attn_fwd.cu):
//   warps 0-7  softmax + epilogue, two threads per row
//   warp  8    producer of V: lanes hold the page numbers of four blocks at a time, and each
//              issues one page's copy
//   warp  9    issuer of the S = Q K^T MMAs (one lane) and TMEM owner
//   warp 10    issuer of the O += P V MMAs (one lane; all lanes clear the V rows past a
//              sequence's end and before its first row's window, whose contents 0 * NaN
//              would carry into O)
//   warp 11    producer of Q and K: walks the CTA's part of the plan and describes every
//              piece of work in shared memory for the other roles
// TMEM: S buffers 0-2 (P over their first halves) and the O accumulator, as in attn_fwd.cu.
//
// Work: paged_plan.cu deals out whole tiles in waves and then gives every CTA a range of
// the rest, so that all end together.  A tile cut
// among CTAs goes to the workspace in parts; the last CTA to finish one joins the parts in
// CTA order.  No CTA waits for another, so the launch is an ordinary one.
//
// Measured: 4608 tokens over 18432 keys, 24 heads: 700 us in short runs (1490 TFLOP/s, 77 %
// of cuBLAS's burst; the dense kernel reaches 1600 on 18432^2), 740 at the power limit; two
// chunks of 2048 over 16384, 32 / 8 heads: 700 and 750; any page size within 3 %.  A tile
// costs some 3 us beside its blocks (first copies 2.6, last PV and epilogue 2.9, overlapped
// in part), a cut tile 6 more (part 1.1, fence and count 1.8, join 1.2 per part, some 0.3 with up
// to 32 rows, whose join all warps share: 8 tokens over 32768 keys, 32 / 8 heads, 49 -> 37 us).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_tile.cuh"
#include "device_wait.cuh"
#include "error_words.cuh"
#include "kernels.h"
#include "paged.h"
#include "paged_chunk.cuh"
#include "paged_walk.cuh"
#include "ptx.cuh"

namespace xs {
namespace {

constexpr int NUM_THREADS = 384;
constexpr int WARP_V = 8;
constexpr int WARP_MMA_S = 9;
constexpr int WARP_MMA_PV = 10;
constexpr int WARP_K = 11;

template <int D>
struct Cfg {
    static constexpr int TILE_BYTES = BLOCK_M * D * 2;
    static constexpr int PANELS = D / 64;
    static constexpr int GROUP = PANELS * 1024;        // 8 keys of a K/V tile: [panel][key][64 channels]
    static constexpr int Q_BUFS = (D == 128) ? 1 : 2;
    static constexpr int KV_STAGES = (D == 128) ? 4 : 10;
    static constexpr int Q_OFF = 0;
    static constexpr int KV_OFF = Q_BUFS * TILE_BYTES;
    static constexpr int STAGE_OFF = KV_OFF + KV_STAGES * TILE_BYTES;  // epilogue staging, 2 KB per softmax warp
    static constexpr int BAR_OFF = STAGE_OFF + NUM_SOFTMAX_WARPS * 2048;
    static constexpr int B_Q_FULL = 0;                 // [2]  TMA -> MMA, per Q buffer
    static constexpr int B_Q_FREE = 2;                 // [2]  MMA -> TMA
    static constexpr int B_S_FULL = 4;                 // [3]  S MMA -> softmax, per S buffer
    static constexpr int B_P_FULL = 7;                 // [3]  softmax -> PV MMA
    static constexpr int B_P_FREE = 10;                // [3]  PV MMA -> S MMA / rescale
    static constexpr int B_O_FINAL = 13;               // [1]  MMA -> epilogue
    static constexpr int B_O_FREE = 14;                // [1]  epilogue -> MMA
    static constexpr int B_DRAIN = 15;                 // [1]  both issuers
    static constexpr int B_PIECE = 16;                 // [4]  producer -> all: descriptor written
    static constexpr int B_PART = 20;                  // [1]  softmax warps -> warp 0: part written
    static constexpr int B_JOIN = 21;                  // [1]  warp 0 -> softmax warps: who joins
    static constexpr int B_KV_FULL = 22;               // [NS] TMA -> MMA
    static constexpr int B_KV_FREE = 22 + KV_STAGES;   // [NS] MMA -> TMA
    static constexpr int NUM_BARS = 22 + 2 * KV_STAGES;
    static constexpr int PIECE_OFF = (BAR_OFF + NUM_BARS * 8 + 63) / 64 * 64;
    static constexpr int MISC_OFF = PIECE_OFF + PIECES * 64;
    static constexpr int LOADED_OFF = MISC_OFF + 16;
    static constexpr int SMEM_BYTES = LOADED_OFF + KV_STAGES * 4;
    static constexpr int SMEM_ALLOC = SMEM_BYTES + 1024;
};
static_assert(Cfg<128>::SMEM_ALLOC <= 232448 && Cfg<64>::SMEM_ALLOC <= 232448, "shared memory budget");

// kind::f16 with both operands fp16 or both bf16, fp32 accumulation.
template <bool F16>
__host__ __device__ constexpr uint32_t idesc(uint32_t M, uint32_t N, uint32_t b_mn_major) {
    const uint32_t bf16 = idesc_bf16_f32(M, N, b_mn_major);
    return F16 ? bf16 & ~((1u << 7) | (1u << 10)) : bf16;
}

// --------------------------------------------------------------- producers
// Two warps share the K/V ring: one loads K blocks (and walks the plan, describes the
// pieces and loads Q), one V blocks; each item goes to the ring position of the
// consumption order K0, K1, V0, K2, V1, ...  A copy costs its warp some 30 ns to issue
// (lanes with different pages issue one after the other), so with 16-token pages one warp
// for both held every block back to 16 of them: 1060 us at 4608 x 18432, 24 heads.
//
// loaded[stage] (shared memory) is one more than the round of the stage's newest copy, for
// an aborting CTA to let the copies in flight land.

// One ring item, by the whole warp: waits for its stage, then one copy per page.
template <int D>
__device__ __forceinline__ bool load_item(const CUtensorMap* map, const PagedAttnArgs& a, uint32_t kv_base, uint32_t bar0,
                                          uint32_t item, int pages, int blk, int key0, int x, int boxes, int box,
                                          volatile int* abort_flag, int u, volatile uint32_t* loaded) {
    using C = Cfg<D>;
    const int lane = static_cast<int>(lane_id());
    const uint32_t stage = item % C::KV_STAGES, round = item / C::KV_STAGES;
    const uint32_t full = bar0 + (C::B_KV_FULL + stage) * 8u;
    bool ok = true;
    if (lane == 0) {
        if (round > 0)
            ok = thread_wait(bar0 + (C::B_KV_FREE + stage) * 8u, (round - 1) & 1, abort_flag, a.timeout_ns, u, blk);
        if (ok) {
            mbar_arrive_expect_tx(full, C::TILE_BYTES);
            loaded[stage] = round + 1;
        }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    const int page = __shfl_sync(0xffffffffu, pages, (blk & 3) * 8 + (lane & 7));
    __syncwarp();
    if (!ok) return false;
    if (lane < boxes)
        tma_load_5d(kv_base + stage * C::TILE_BYTES + lane * box * (D * 2), map, full, x, 0, 0,
                    ((key0 + blk * BLOCK_N) & ((1 << a.page_shift) - 1)) >> 3, page);
    return true;
}

// A descriptor slot is reused four pieces later: the producer is then past the wait for
// the Q buffer of piece u - 1 or u - 2, whose scores are issued only after the last PV of
// the piece before, so every role has left piece u - 4.
template <int D>
__device__ void producer_k_role(const CUtensorMap* tq, const CUtensorMap* tk, const PagedAttnArgs& a, uint8_t* smem,
                                uint32_t bar0, volatile int* abort_flag) {
    using C = Cfg<D>;
    const int lane = static_cast<int>(lane_id());
    const uint32_t sbase = smem_addr(smem);
    auto bar = [&](int i) { return bar0 + static_cast<uint32_t>(i) * 8u; };
    const int box = 1 << (a.page_shift < 7 ? a.page_shift : 7);   // keys of one copy
    const int boxes = BLOCK_N / box;                              // 1 .. 8
    const int tokens = a.tile.tokens;

    PieceWalk walk(a, 0);
    uint32_t item0 = 0;       // first ring item of the piece
    int u = 0;
    int q_last = -1;          // piece of the last Q load issued
    volatile uint32_t* const loaded = reinterpret_cast<volatile uint32_t*>(smem + C::LOADED_OFF);
    bool ok = true;
    for (;; ++u) {
        const int qb = u % C::Q_BUFS;
        if (u >= C::Q_BUFS) {
            if (lane == 0)
                ok = thread_wait(bar(C::B_Q_FREE + qb), ((u / C::Q_BUFS) - 1) & 1, abort_flag, a.timeout_ns, u);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            __syncwarp();
        }
        if (!ok) break;
        Piece d{};
        const bool more = walk.describe(a, box, d);
        if (lane == 0) {
            *reinterpret_cast<Piece*>(smem + C::PIECE_OFF + (u % PIECES) * 64) = d;
            mbar_arrive(bar(C::B_PIECE + u % PIECES));   // release: the descriptor is visible to whoever waits
        }
        if (!more) break;
        if (walk.cut_end) pdl_launch();   // the CTA's last piece (a CTA that ends without one counts when it exits)
        if (lane == 0) {
            mbar_arrive_expect_tx(bar(C::B_Q_FULL + qb), static_cast<uint32_t>(tokens * a.G) * D * 2);
            for (int pnl = 0; pnl < C::PANELS; ++pnl)
                tma_load_4d(sbase + C::Q_OFF + qb * C::TILE_BYTES + pnl * PANEL_BYTES, tq, bar(C::B_Q_FULL + qb),
                            pnl * 64, 0, d.head, d.row0);
        }
        q_last = u;
        const int* table = a.table + static_cast<long long>(d.index) * a.table_stride;
        int cur = -1, next = load_pages(a, table, 0, d.key0, d.nb, d.kv_len, d.lo_key, boxes, box);
        for (int j = 0; j < d.nb && ok; ++j) {
            if ((j & 3) == 0) {
                cur = next;
                next = load_pages(a, table, (j >> 2) + 1, d.key0, d.nb, d.kv_len, d.lo_key, boxes, box);
            }
            ok = load_item<D>(tk, a, sbase + C::KV_OFF, bar0, item0 + ring_pos_k(j), cur, j, d.key0, d.head * a.k_head,
                              boxes, box, abort_flag, u, loaded);
        }
        if (!ok) break;
        item0 += 2u * d.nb;
        walk.advance(a);
    }
    // the newest Q copy lands before the CTA exits
    if (!ok && lane == 0 && q_last >= 0)
        drain_wait(bar(C::B_Q_FULL + q_last % C::Q_BUFS), (q_last / C::Q_BUFS) & 1, 20000000ull);
    __syncwarp();
}

template <int D>
__device__ void producer_v_role(const CUtensorMap* tv, const PagedAttnArgs& a, uint8_t* smem, uint32_t bar0,
                                volatile int* abort_flag) {
    using C = Cfg<D>;
    const uint32_t sbase = smem_addr(smem);
    const int box = 1 << (a.page_shift < 7 ? a.page_shift : 7);
    const int boxes = BLOCK_N / box;
    uint32_t item0 = 0;
    volatile uint32_t* const loaded = reinterpret_cast<volatile uint32_t*>(smem + C::LOADED_OFF);
    bool ok = true;
    for (int u = 0; ok; ++u) {
        ok = warp_wait(bar0 + (C::B_PIECE + u % PIECES) * 8u, (u / PIECES) & 1, abort_flag, a.timeout_ns, u);
        if (!ok) break;
        const Piece d = piece_of(smem, C::PIECE_OFF, u);
        if (d.nb == 0) break;
        const int* table = a.table + static_cast<long long>(d.index) * a.table_stride;
        int cur = -1, next = load_pages(a, table, 0, d.key0, d.nb, d.kv_len, d.lo_key, boxes, box);
        for (int j = 0; j < d.nb && ok; ++j) {
            if ((j & 3) == 0) {
                cur = next;
                next = load_pages(a, table, (j >> 2) + 1, d.key0, d.nb, d.kv_len, d.lo_key, boxes, box);
            }
            ok = load_item<D>(tv, a, sbase + C::KV_OFF, bar0, item0 + ring_pos_v(j, d.nb), cur, j, d.key0,
                              d.head * a.v_head, boxes, box, abort_flag, u, loaded);
        }
        item0 += 2u * d.nb;
    }
    __syncwarp();
}

// --------------------------------------------------------------------- MMA
// A K/V tile is [8-key group][panel][key][64 channels] (paged.h): the 8-key groups are C::GROUP apart
// (SBO of both operands), the panels 1024 B.  As K (K-major), k-step kk covers 16 channels, 32 B within
// the rows of panel kk / 4; as V (MN-major, panels by LBO), 16 keys, two groups.
__device__ __forceinline__ constexpr uint32_t kv_k_step16(int kk) {
    return static_cast<uint32_t>((kk >> 2) * (1024 >> 4) + (kk & 3) * 2);
}
template <int D>
__device__ __forceinline__ constexpr uint32_t kv_v_step16(int kk) {
    return static_cast<uint32_t>(kk * (2 * Cfg<D>::GROUP >> 4));
}

// Issuer of S(j) = Q K_j^T (SS) into S buffer (block index) % 3.  One thread.
template <int D, bool F16>
__device__ void mma_s_role(const PagedAttnArgs& a, uint8_t* smem, uint32_t bar0, uint32_t tmem_base,
                           volatile int* abort_flag) {
    using C = Cfg<D>;
    const uint32_t sbase = smem_addr(smem);
    auto bar = [&](int i) { return bar0 + static_cast<uint32_t>(i) * 8u; };
    constexpr uint32_t IDESC_QK = idesc<F16>(BLOCK_M, BLOCK_N, 0);
    const uint64_t qdesc0 = smem_desc_sw128(sbase + C::Q_OFF, 16, 1024);   // Q buffer 0
    const uint64_t kdesc0 = smem_desc_sw128(sbase + C::KV_OFF, 16, C::GROUP);  // ring stage 0, as K
    uint32_t g = 0;      // key blocks over the CTA's lifetime
    uint32_t sb = 0, sph = 0;   // S buffer of block g (g % 3) and its phase parity ((g / 3) & 1)
    uint32_t item0 = 0;  // first ring item of the current piece of work
    int u = 0;
    bool ok = true;
    for (; ok; ++u) {
        ok = thread_wait(bar(C::B_PIECE + u % PIECES), (u / PIECES) & 1, abort_flag, a.timeout_ns, u);
        if (!ok) break;
        const int n = piece_of(smem, C::PIECE_OFF, u).nb;
        if (n == 0) break;
        const int qb = u % C::Q_BUFS;
        const uint64_t qdesc = desc_add(qdesc0, qb * (C::TILE_BYTES >> 4));
        ok = thread_wait(bar(C::B_Q_FULL + qb), (u / C::Q_BUFS) & 1, abort_flag, a.timeout_ns, u);
        // the previous piece's last PV first: its epilogue waits for it
        if (ok && u > 0) ok = thread_wait(bar(C::B_O_FINAL), (u - 1) & 1, abort_flag, a.timeout_ns, u);
        for (int j = 0; j < n && ok; ++j) {
            const uint32_t gs = g + j;
            if (gs >= S_BUFS) ok = thread_wait(bar(C::B_P_FREE + sb), sph ^ 1u, abort_flag, a.timeout_ns, u, j);
            const uint32_t item = item0 + ring_pos_k(j);
            const uint32_t stage = item % C::KV_STAGES;
            if (ok)
                ok = thread_wait(bar(C::B_KV_FULL + stage), (item / C::KV_STAGES) & 1, abort_flag, a.timeout_ns, u, j);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kdesc = desc_add(kdesc0, stage * (C::TILE_BYTES >> 4));
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(tmem_base + S_COL + sb * 128u, desc_add(qdesc, k_step16(kk)), desc_add(kdesc, kv_k_step16(kk)),
                       IDESC_QK, kk > 0);
            mma_commit(bar(C::B_S_FULL + sb));
            mma_commit(bar(C::B_KV_FREE + stage));
            if (j == n - 1) mma_commit(bar(C::B_Q_FREE + qb));
            if (++sb == S_BUFS) {
                sb = 0;
                sph ^= 1u;
            }
        }
        g += n;
        item0 += 2u * n;
    }
    // B_DRAIN completes when both issuers' MMAs have all completed (TMEM is freed after it)
    mma_commit(bar(C::B_DRAIN));
    drain_wait(bar(C::B_DRAIN), 0, a.timeout_ns > 20000000ull ? a.timeout_ns : 20000000ull);
}

// Issuer of PV(j): O += P(j) V_j.  Lane 0 waits and issues; the warp clears V rows.
template <int D, bool F16>
__device__ void mma_pv_role(const PagedAttnArgs& a, uint8_t* smem, uint32_t bar0, uint32_t tmem_base,
                            volatile int* abort_flag) {
    using C = Cfg<D>;
    const int lane = static_cast<int>(lane_id());
    const uint32_t sbase = smem_addr(smem);
    auto bar = [&](int i) { return bar0 + static_cast<uint32_t>(i) * 8u; };
    constexpr uint32_t IDESC_PV = idesc<F16>(BLOCK_M, D, 1);
    const uint64_t vdesc0 = smem_desc_sw128(sbase + C::KV_OFF, 1024, C::GROUP);  // ring stage 0, as V
    uint32_t pb = 0, pph = 0;   // buffer of block g (g % 3) and its phase parity ((g / 3) & 1)
    uint32_t item0 = 0;
    int u = 0;
    bool ok = true;
    for (; ok; ++u) {
        ok = warp_wait(bar(C::B_PIECE + u % PIECES), (u / PIECES) & 1, abort_flag, a.timeout_ns, u);
        if (!ok) break;
        const Piece& d = piece_of(smem, C::PIECE_OFF, u);
        const int n = d.nb;
        if (n == 0) break;
        // blocks [tail, n) reach past the sequence: their V rows from `left` on are cleared; so are the first block's
        // `low` rows below `unseen`
        const int left = d.kv_len - d.key0, low = d.unseen_rows;
        const int tail = left > 0 ? left / BLOCK_N : 0;
        // every block below `stop` is lane 0's alone; then the warp clears one and goes on
        for (int j0 = 0; j0 < n && ok;) {
            const bool clear = j0 >= tail || (j0 == 0 && low > 0);
            const int stop = clear ? j0 + 1 : (tail < n ? tail : n);
            if (clear) {
                const uint32_t item = item0 + ring_pos_v(j0, n);
                const uint32_t stage = item % C::KV_STAGES;
                ok = warp_wait(bar(C::B_KV_FULL + stage), (item / C::KV_STAGES) & 1, abort_flag, a.timeout_ns, u, j0);
                if (!ok) break;
                const int first = min(max(left - j0 * BLOCK_N, 0), BLOCK_N), below = j0 == 0 ? low : 0;
                const int from = d.unseen - d.key0 - below;
                uint8_t* v = smem + C::KV_OFF + stage * C::TILE_BYTES;
                for (int i = lane; i < (below + BLOCK_N - first) * (D / 8); i += 32) {
                    const int r = i / (D / 8) + (i < below * (D / 8) ? from : first - below), c8 = i % (D / 8);
                    *reinterpret_cast<uint4*>(v + (r >> 3) * C::GROUP + (c8 >> 3) * 1024 + (r & 7) * 128 + (c8 & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();   // before the MMA reads it, and the next copy writes it
                __syncwarp();
            }
            if (lane == 0) {
                for (int j = j0; j < stop && ok; ++j) {
                    ok = thread_wait(bar(C::B_P_FULL + pb), pph, abort_flag, a.timeout_ns, u, j);
                    // the epilogue has read the previous piece's O (PV(0) overwrites it)
                    if (ok && j == 0 && u > 0) ok = thread_wait(bar(C::B_O_FREE), (u - 1) & 1, abort_flag, a.timeout_ns, u, j);
                    const uint32_t item = item0 + ring_pos_v(j, n);
                    const uint32_t stage = item % C::KV_STAGES;
                    if (ok)
                        ok = thread_wait(bar(C::B_KV_FULL + stage), (item / C::KV_STAGES) & 1, abort_flag, a.timeout_ns, u, j);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vdesc = desc_add(vdesc0, stage * (C::TILE_BYTES >> 4));
#pragma unroll
                    for (int kk = 0; kk < BLOCK_N / 16; ++kk)
                        mma_ts(tmem_base + O_COL, tmem_base + S_COL + pb * 128u + kk * 8, desc_add(vdesc, kv_v_step16<D>(kk)),
                               IDESC_PV, (j > 0) || (kk > 0));
                    mma_commit(bar(C::B_P_FREE + pb));
                    mma_commit(bar(C::B_KV_FREE + stage));
                    if (j == n - 1) mma_commit(bar(C::B_O_FINAL));
                    if (++pb == S_BUFS) {
                        pb = 0;
                        pph ^= 1u;
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            j0 = stop;
        }
        item0 += 2u * n;
    }
    if (lane == 0) {
        mma_commit(bar(C::B_DRAIN));
        drain_wait(bar(C::B_DRAIN), 0, a.timeout_ns > 20000000ull ? a.timeout_ns : 20000000ull);
    }
    __syncwarp();
}

// ------------------------------------------------------- softmax + epilogue
template <int D, bool F16>
__device__ void softmax_role(const PagedAttnArgs& a, uint8_t* smem, uint32_t bar0, uint32_t tmem_base,
                             volatile int* abort_flag) {
    using C = Cfg<D>;
    constexpr int DH = D / 2;  // O columns owned by each of a row's two threads
    const int warp = threadIdx.x >> 5;
    const int lane = static_cast<int>(lane_id());
    const int quarter = warp & 3;             // TMEM lane quarter this warp may access
    const int half = lane >> 4;               // key columns [64*half, 64*half + 64), O columns [DH*half, +DH)
    const int warp_row = quarter * 32 + (warp >> 2) * 16;   // the warp's first row
    const int row = warp_row + (lane & 15);
    const uint32_t t_base = tmem_base + (static_cast<uint32_t>(warp_row) << 16);
    auto bar = [&](int i) { return bar0 + static_cast<uint32_t>(i) * 8u; };
    const float c = a.c;

    uint32_t sb = 0, sph = 0;    // S buffer of block g (g % 3) and its phase parity ((g / 3) & 1)
    uint32_t pb = 2, pph = 1;    // the same for block g - 1 (the O rescale waits for PV(g-1))
    int u = 0, n_parts = 0;
    bool ok = true;
    for (; ok; ++u) {
        ok = warp_wait(bar(C::B_PIECE + u % PIECES), (u / PIECES) & 1, abort_flag, a.timeout_ns, u);
        if (!ok) break;
        const Piece& d = piece_of(smem, C::PIECE_OFF, u);
        const int n = d.nb;
        if (n == 0) break;
        const bool idle = warp_row >= d.n_rows;   // no query row in this warp
        // columns [lo, hi) of the piece that this row sees; rows past the tile take the last one's
        int lo = 0, hi;
        {
            const int r = row < d.n_rows ? row : d.n_rows - 1;
            const int p = d.pos0 + fdiv(r, a.fd_G);
            hi = (a.causal ? (p < 0 ? 0 : p + 1) : d.kv_len) - d.key0;
            if (a.window > 0 && p - a.window >= 0) lo = p - a.window + 1 - d.key0;
        }
        float m_run = NO_MAX, l_run = 0.0f;
        for (int j = 0; j < n; ++j) {
            ok = warp_wait(bar(C::B_S_FULL + sb), sph, abort_flag, a.timeout_ns, u, j);
            if (!ok) break;
            if (!idle) {
                tc_fence_after();
                uint32_t sr[2][32];
                tmem_ld16x2_32<64>(t_base + S_COL + sb * 128u, sr[0]);
                tmem_ld16x2_32<64>(t_base + S_COL + sb * 128u + 32, sr[1]);
                tmem_wait_ld();
                const int from = lo - j * BLOCK_N, to = hi - j * BLOCK_N;
                if (__any_sync(0xffffffffu, from > 0 || to < BLOCK_N)) {   // warp-uniform path
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int col = half * 64 + q * 32 + i;
                            if (col < from || col >= to) sr[q][i] = 0xff800000u;  // -inf
                        }
                }
                // row max: the two halves of the row are lanes i and i ^ 16
                const float m_half = max64(sr);
                const float m_blk = fmaxf(fmaxf(m_half, __shfl_xor_sync(0xffffffffu, m_half, 16)) * c, NO_MAX);
                float m_use = m_run, alpha = 1.0f;
                bool rescale = false;
                if (m_blk - m_run > RESCALE_THRESHOLD) {
                    m_use = m_blk;
                    alpha = ex2_approx(m_run - m_blk);
                    rescale = j > 0;
                }
                uint32_t pk[32];
                const float sum = exp64<false, F16>(sr, c, m_use, 0, 0, pk);
                // Rescale of this thread's half of the O row (rare); PV(g-1) must have completed
                // first.  Warp-uniform: TMEM access is collective.
                if (__any_sync(0xffffffffu, rescale)) {
                    ok = warp_wait(bar(C::B_P_FREE + pb), pph, abort_flag, a.timeout_ns, u, j);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int q = 0; q < DH / 32; ++q) {
                        uint32_t orr[32];
                        tmem_ld16x2_32<DH>(t_base + O_COL + q * 32, orr);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) orr[i] = __float_as_uint(__uint_as_float(orr[i]) * alpha);
                        tmem_st16x2_32<DH>(t_base + O_COL + q * 32, orr);
                    }
                }
                // P over the first 64 columns of the scores just read
                tmem_st16x2_32<32>(t_base + S_COL + sb * 128u, pk);
                tmem_wait_st();
                tc_fence_before();
                l_run = l_run * alpha + sum;
                m_run = m_use;
            }
            warp_arrive(bar(C::B_P_FULL + sb));
            pb = sb;
            pph = sph;
            if (++sb == S_BUFS) {
                sb = 0;
                sph ^= 1u;
            }
        }
        if (!ok) break;
        // ---- epilogue: the owner of this tile stores it to the destination shard
        const float l_row = l_run + __shfl_xor_sync(0xffffffffu, l_run, 16);
        ok = warp_wait(bar(C::B_O_FINAL), u & 1, abort_flag, a.timeout_ns, u);
        if (!ok) break;
        tc_fence_after();
        if (d.part >= 0) {
            ok = part_epilogue<C, D, F16>(a, d, smem, bar0, t_base + O_COL, row, half, warp, m_run, l_row, n_parts & 1,
                                       abort_flag);
            ++n_parts;
            continue;
        }
        if (!idle) store_tile<D, F16>(a, d, smem + C::STAGE_OFF + warp * 2048, t_base + O_COL, row, half, m_run, l_row);
        tc_fence_before();
        warp_arrive(bar(C::B_O_FREE));
    }
}

template <int D, bool F16>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ PagedAttnArgs args) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t bar0 = smem_addr(smem + C::BAR_OFF);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);   // [1]: who joins a cut tile
    const int warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar0 + 8 * (C::B_Q_FULL + i), 1);   // (index 1 unused when Q_BUFS == 1)
            mbar_init(bar0 + 8 * (C::B_Q_FREE + i), 1);
        }
        for (int i = 0; i < S_BUFS; ++i) {
            mbar_init(bar0 + 8 * (C::B_S_FULL + i), 1);
            mbar_init(bar0 + 8 * (C::B_P_FULL + i), NUM_SOFTMAX_WARPS);
            mbar_init(bar0 + 8 * (C::B_P_FREE + i), 1);
        }
        mbar_init(bar0 + 8 * C::B_O_FINAL, 1);
        mbar_init(bar0 + 8 * C::B_O_FREE, NUM_SOFTMAX_WARPS);
        mbar_init(bar0 + 8 * C::B_DRAIN, 2);
        for (int i = 0; i < PIECES; ++i) mbar_init(bar0 + 8 * (C::B_PIECE + i), 1);
        mbar_init(bar0 + 8 * C::B_PART, NUM_SOFTMAX_WARPS);
        mbar_init(bar0 + 8 * C::B_JOIN, 1);
        for (int s = 0; s < C::KV_STAGES; ++s) {
            mbar_init(bar0 + 8 * (C::B_KV_FULL + s), 1);
            mbar_init(bar0 + 8 * (C::B_KV_FREE + s), 1);
        }
        for (int s = 0; s < C::KV_STAGES; ++s) reinterpret_cast<uint32_t*>(smem + C::LOADED_OFF)[s] = 0;
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == WARP_K && lane_id() == 0) {
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    if (warp == WARP_MMA_S) {
        tmem_alloc(smem_addr(tmem_holder), TMEM_COLS);
        tmem_relinquish();
    }
    // Q rows past tokens * G (G does not divide 128): no copy writes them, their scores are read and dropped
    const int q_rows = args.tile.tokens * args.G;
    for (int i = threadIdx.x; i < (BLOCK_M - q_rows) * C::Q_BUFS * C::PANELS * 8; i += NUM_THREADS) {
        const int r = q_rows + i / (C::Q_BUFS * C::PANELS * 8), p = i / 8 % (C::Q_BUFS * C::PANELS);
        *reinterpret_cast<uint4*>(smem + C::Q_OFF + p * PANEL_BYTES + r * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    pdl_wait();

    if (warp < NUM_SOFTMAX_WARPS)
        softmax_role<D, F16>(args, smem, bar0, tmem_base, abort_flag);
    else if (warp == WARP_K)
        producer_k_role<D>(&tq, &tk, args, smem, bar0, abort_flag);
    else if (warp == WARP_V)
        producer_v_role<D>(&tv, args, smem, bar0, abort_flag);
    else if (warp == WARP_MMA_PV)
        mma_pv_role<D, F16>(args, smem, bar0, tmem_base, abort_flag);
    else if (warp == WARP_MMA_S && lane_id() == 0)
        mma_s_role<D, F16>(args, smem, bar0, tmem_base, abort_flag);
    __syncwarp();

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == WARP_MMA_S) tmem_dealloc(tmem_base, TMEM_COLS);
    if (*abort_flag && threadIdx.x == 0) {   // copies already issued land before the CTA exits
        const uint32_t* loaded = reinterpret_cast<const uint32_t*>(smem + C::LOADED_OFF);
        for (int s = 0; s < C::KV_STAGES; ++s)
            if (loaded[s] > 0) drain_wait(bar0 + 8 * (C::B_KV_FULL + s), (loaded[s] - 1) & 1, 20000000ull);
    }
}

template <int D, bool F16>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a,
                   cudaStream_t stream) {
    auto kern = attn_paged_kernel<D, F16>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM_ALLOC);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kern, dim3(static_cast<unsigned>(a.tile.grid)), NUM_THREADS, Cfg<D>::SMEM_ALLOC, stream, tq, tk,
                             tv, a);
}

}  // namespace

cudaError_t launch_attn_paged(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const PagedAttnArgs& a, int dtype, cudaStream_t stream) {
    if (a.D == 128) return dtype == 0 ? launch<128, false>(tq, tk, tv, a, stream) : launch<128, true>(tq, tk, tv, a, stream);
    return dtype == 0 ? launch<64, false>(tq, tk, tv, a, stream) : launch<64, true>(tq, tk, tv, a, stream);
}

cudaError_t paged_error_words(ErrorWords* w) { return error_words_here(w); }

cudaError_t read_and_clear_paged_error(int* value, DeviceErrorInfo* info, int* drain_failed, unsigned long long* when) {
    return read_and_clear_error_words(value, info, drain_failed, when);
}

}  // namespace xs
