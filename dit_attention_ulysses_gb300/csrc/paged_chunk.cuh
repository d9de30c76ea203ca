// Pieces of the tcgen05 attention over a paged cache that do not depend on the cache's type: the
// descriptors of a CTA's work, the walk over its part of the plan, and what becomes of a
// finished or unfinished tile.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "attn_tile.cuh"
#include "device_wait.cuh"
#include "kernels.h"
#include "paged.h"
#include "paged_walk.cuh"
#include "ptx.cuh"

namespace xs {
namespace {

constexpr int NUM_SOFTMAX_WARPS = 8;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t S_COL = 0;     // + 128 * buffer; P(g) over the first 64 columns of buffer g % 3
constexpr int S_BUFS = 3;
constexpr uint32_t O_COL = 384;
constexpr float RESCALE_THRESHOLD = 8.0f;   // log2 units
constexpr float NO_MAX = -3.402823466e38f;            // running maximum of a row that has seen nothing
constexpr int PIECES = 4;                   // descriptors in flight (see producer_k_role)

// One piece of work: key blocks of one tile, written by the producer.
struct Piece {
    int nb;         // key blocks; 0: no more work
    int key0;       // first key
    int kv_len;     // keys of the sequence
    int row0;       // packed row of the tile's first token
    int n_rows;     // packed query rows (tokens * G)
    int pos0;       // position of the tile's first token (negative: it sees no key when causal)
    int head;       // KV head
    int part;       // workspace slot of an unfinished tile; -1: the whole tile
    int c0, c1;     // CTAs of an unfinished tile
    int index;      // row of the block table
    int lo_key;     // first key that some row sees
    int unseen;     // keys below it: no row of the sequence sees them
    int unseen_rows;   // so many of them, right below it, come in with the first block (the others read as zeros)
    int unused[2];
};
static_assert(sizeof(Piece) == 64, "descriptor");

__device__ __forceinline__ const Piece& piece_of(const uint8_t* smem, int piece_off, int u) {
    return *reinterpret_cast<const Piece*>(smem + piece_off + (u % PIECES) * 64);
}

// Page numbers of a piece's blocks: lane 8 j + i holds page i of block 4 m + j of group m.
// Past the keys, before the window and past the table: -1, a page out of range, which
// reads as zeros.
__device__ __forceinline__ int load_pages(const PagedAttnArgs& a, const int* table, int m, int key0, int nb, int kv_len,
                                          int lo_key, int boxes, int box) {
    const int lane = static_cast<int>(lane_id());
    const int blk = 4 * m + (lane >> 3);
    const int key = key0 + blk * BLOCK_N + (lane & 7) * box;
    if ((lane & 7) >= boxes || blk >= nb || key >= kv_len || key + box <= lo_key) return -1;
    const int col = key >> a.page_shift;
    return static_cast<unsigned>(col) < static_cast<unsigned>(a.width) ? table[col] : -1;
}

// A CTA's part of the plan, walked by one warp: whole tiles in waves, then its range of the rest.
struct PieceWalk {
    PagedRange range;
    PagedPos pos;
    PagedSeq seq;
    const PagedSlot* slots;
    int n_seqs, per_slot, waves;
    int wave, left;        // slot `wave` has `left` tiles to go
    bool in_wave, cut_end; // of the piece described last

    __device__ __forceinline__ PieceWalk(const PagedAttnArgs& a, int cache8) {
        range = a.work.ranges[blockIdx.x];
        const PagedHeader& h = *a.work.header;
        n_seqs = h.n_seqs;
        per_slot = h.slot;
        waves = h.waves - (static_cast<int>(blockIdx.x) >= h.slot_ctas ? 1 : 0);
        if (h.n != a.n || h.H != a.H || h.Hkv != a.Hkv || h.D != a.D || h.tokens != a.tile.tokens || h.block != BLOCK_N ||
            h.grid != a.tile.grid || h.causal != a.causal || h.window != a.window || h.cache8 != cache8) {
            if (lane_id() == 0) report_error(XS_DEVICE_BOUNDS_CODE, PAGED_MAGIC_SITE, h.n, h.tokens, h.grid);
            range.end = range.start;
            waves = 0;
        }
        slots = a.work.slots + static_cast<size_t>(blockIdx.x) * MAX_PAGED_WAVES;
        wave = left = 0;
        in_wave = cut_end = false;
        begin();
    }

    __device__ __forceinline__ void begin() {
        if (wave < waves) {
            pos = slots[wave].pos;
            seq = slots[wave].seq;
            left = per_slot;
        } else {
            pos = range.start;
            seq = range.first;
        }
    }

    // The next piece, for copies of `box` keys; false: there is none (d.nb == 0).
    __device__ __forceinline__ bool describe(const PagedAttnArgs& a, int box, Piece& d) {
        const int tokens = a.tile.tokens;
        in_wave = wave < waves;
        cut_end = false;
        if (!in_wave && !paged_before(pos, range.end)) return false;
        if (!paged_valid(pos, seq, n_seqs, tokens, a.Hkv)) {
            if (lane_id() == 0) report_error(XS_DEVICE_BOUNDS_CODE, PAGED_MAGIC_SITE, pos.seq, pos.head, pos.tile);
            return false;
        }
        int b0, count, hi_tile;
        paged_tile_blocks(seq, pos.tile, a.tile, a.causal, a.window, b0, count);
        paged_tile_keys(seq, pos.tile, tokens, a.causal, a.window, d.lo_key, hi_tile);
        cut_end = !in_wave && paged_same_tile(pos, range.end);
        const int k1 = cut_end && range.end.k < count ? range.end.k : count;
        const int tok0 = pos.tile * tokens;
        const int n_tok = seq.q_len - tok0 < tokens ? seq.q_len - tok0 : tokens;
        d.nb = k1 - pos.k;
        d.key0 = (b0 + pos.k) * BLOCK_N;
        d.kv_len = seq.kv_len;
        d.row0 = seq.q_start + tok0;
        d.n_rows = n_tok * a.G;
        d.pos0 = seq.kv_len - seq.q_len + tok0;
        d.head = pos.head;
        d.index = seq.index;
        d.unseen = paged_unseen(seq, a.window);
        d.unseen_rows = pos.k == 0 ? max(d.unseen - (d.lo_key & ~(box - 1)), 0) : 0;
        const bool whole = pos.k == 0 && !cut_end;
        d.part = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (pos.k == 0 ? 1 : 0);
        d.c0 = pos.k == 0 ? static_cast<int>(blockIdx.x) : range.c0;
        d.c1 = pos.k == 0 ? range.c1_last : range.c1;
        if (d.nb < 1 || (!whole && (d.c0 < 0 || d.c1 < d.c0 || d.c1 >= a.tile.grid))) {
            if (lane_id() == 0) report_error(XS_DEVICE_BOUNDS_CODE, PAGED_MAGIC_SITE, d.nb, d.c0, d.c1);
            d.nb = 0;
            return false;
        }
        return true;
    }

    __device__ __forceinline__ void advance(const PagedAttnArgs& a) {
        if (in_wave && --left == 0) {
            ++wave;
            begin();
        } else if (cut_end) {
            pos = range.end;   // the rest of the tile is the next CTA's
        } else if (paged_next(pos, seq, a.tile.tokens, a.Hkv) && (in_wave || paged_before(pos, range.end)) && pos.seq < n_seqs) {
            seq = a.work.seqs[pos.seq];
        }
    }
};

// ------------------------------------------------------------------ finished tiles
// Destination of packed row r of a piece (this lane's row of all `D` channels); null past the rows.
__device__ __forceinline__ uint16_t* dest_row(const PagedAttnArgs& a, const Piece& d, int r, int& token, int& head) {
    int t, gh;
    fdivmod(r, a.fd_G, t, gh);
    token = d.row0 + t;
    head = d.head * a.G + gh;
    if (r >= d.n_rows || token >= a.T) return nullptr;
    int ps, s, ph, h;
    fdivmod(token, a.epi.fd_Sl, ps, s);
    fdivmod(head, a.epi.fd_Hl, ph, h);
    const int p = ps + ph;
    if (p >= MAX_PTRS || a.epi.ptr[p] == nullptr) {
        report_error(XS_DEVICE_BOUNDS_CODE, 2, p, token, head);
        return nullptr;
    }
    return reinterpret_cast<uint16_t*>(a.epi.ptr[p]) + (static_cast<size_t>(s) * a.epi.Hl + h) * a.D;
}

// Log-sum-exp of a row from its maximum (log2 units) and its sum: -infinity if it saw no key, NaN if its sum is.
__device__ __forceinline__ float log_sum(float m, float l) {
    return l == 0.0f ? __int_as_float(0xff800000) : (m + log2f(l)) * 0.6931471805599453f;
}

// The join of a tile of up to 128 / SHARE rows: SHARE warps for every 16 rows, each with a share of the channels of
// both half rows and SHARE parts in flight, in CTA order (past the last: the last, at weight 0).
template <int D, bool F16, int SHARE>
__device__ __forceinline__ bool join_few_rows(const PagedAttnArgs& a, const Piece& d, int warp) {
    constexpr int CHUNKS = D / 8 / SHARE;   // four channels each
    constexpr int SOFTMAX_THREADS = NUM_SOFTMAX_WARPS * 32;
    const int lane = static_cast<int>(lane_id());
    const int owner = (warp & 4) | (warp & (4 / SHARE - 1)), sub = (warp & 3) / (4 / SHARE);
    const int row = (owner & 3) * 32 + (owner >> 2) * 16 + (lane & 15);
    int token, head;
    uint16_t* const dst = dest_row(a, d, row, token, head);
    if (dst == nullptr) return true;
    const float4* const from = reinterpret_cast<const float4*>(a.work.part_o) + owner * 32 + lane;
    float4 acc[CHUNKS];
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float m_all = NO_MAX, l_all = 0.0f;
#pragma unroll 1
    for (int c = d.c0; c <= d.c1; c += SHARE) {
        float2 ml[SHARE];
        float4 v[SHARE][CHUNKS];
#pragma unroll
        for (int j = 0; j < SHARE; ++j) {
            const int cj = c + j <= d.c1 ? c + j : d.c1, slot = 2 * cj + (cj == d.c0 ? 1 : 0);
            ml[j] = __ldcg(a.work.part_ml + static_cast<size_t>(slot) * BLOCK_M + row);
#pragma unroll
            for (int k = 0; k < CHUNKS; ++k)
                v[j][k] = __ldcg(from + (static_cast<size_t>(slot) * (D / 8) + sub * CHUNKS + k) * SOFTMAX_THREADS);
            if (c + j > d.c1) ml[j] = make_float2(NO_MAX, 0.0f);
        }
        float m_new = m_all;
#pragma unroll
        for (int j = 0; j < SHARE; ++j) m_new = fmaxf(m_new, ml[j].x);
        const float f0 = ex2_approx(m_all - m_new);
        m_all = m_new;
        l_all *= f0;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) acc[k] = make_float4(acc[k].x * f0, acc[k].y * f0, acc[k].z * f0, acc[k].w * f0);
#pragma unroll
        for (int j = 0; j < SHARE; ++j) {
            const float f = c + j <= d.c1 ? ex2_approx(ml[j].x - m_all) : 0.0f;
            l_all += ml[j].y * f;
#pragma unroll
            for (int k = 0; k < CHUNKS; ++k) {
                acc[k].x += v[j][k].x * f;
                acc[k].y += v[j][k].y * f;
                acc[k].z += v[j][k].z * f;
                acc[k].w += v[j][k].w * f;
            }
        }
    }
    const float inv = l_all > 0.0f ? 1.0f / l_all : 0.0f;
    if (sub == 0 && lane < 16 && a.lse != nullptr) a.lse[static_cast<size_t>(token) * a.H + head] = log_sum(m_all, l_all);
    uint16_t* const out = dst + (lane >> 4) * (D / 2) + sub * CHUNKS * 4;
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
        uint2 w;
        w.x = F16 ? pack_f16x2(acc[k].x * inv, acc[k].y * inv) : pack_bf16x2(acc[k].x * inv, acc[k].y * inv);
        w.y = F16 ? pack_f16x2(acc[k].z * inv, acc[k].w * inv) : pack_bf16x2(acc[k].z * inv, acc[k].w * inv);
        *reinterpret_cast<uint2*>(out + k * 4) = w;
    }
    return true;
}

// Publishes this thread's half row of an unfinished tile (its O accumulator, maximum and
// sum), and, in the CTA that finishes last, joins the parts in CTA order and stores the
// row.  Out of line: at most twice per CTA and launch.
template <typename C, int D, bool F16>
__device__ __noinline__ bool part_epilogue(const PagedAttnArgs& a, const Piece& d, uint8_t* smem, uint32_t bar0,
                                           uint32_t o_base, int row, int half, int warp, float m, float l, int parity,
                                           volatile int* abort_flag) {
    constexpr int DH = D / 2;
    auto bar = [&](int i) { return bar0 + static_cast<uint32_t>(i) * 8u; };
    // A part is laid out by threads: the k-th four channels of all 256, one after the other, so that
    // every access is 512 contiguous bytes per warp (by rows, a join of two parts took 11 us)
    constexpr int SOFTMAX_THREADS = NUM_SOFTMAX_WARPS * 32;
    float4* const parts_o = reinterpret_cast<float4*>(a.work.part_o);
    auto at_o = [&](int slot, int k) {
        return (static_cast<size_t>(slot) * (DH / 4) + k) * SOFTMAX_THREADS + threadIdx.x;
    };
    auto at_ml = [&](int slot) { return static_cast<size_t>(slot) * BLOCK_M + row; };
#pragma unroll 1
    for (int q = 0; q < (row - (threadIdx.x & 15) < d.n_rows ? DH / 32 : 0); ++q) {   // (a warp without rows: none)
        uint32_t orr[32];
        tmem_ld16x2_32<DH>(o_base + q * 32, orr);
        tmem_wait_ld();
#pragma unroll
        for (int v4 = 0; v4 < 8; ++v4)
            st_global_v4(parts_o + at_o(d.part, q * 8 + v4), orr[4 * v4], orr[4 * v4 + 1], orr[4 * v4 + 2], orr[4 * v4 + 3]);
    }
    if (half == 0) a.work.part_ml[at_ml(d.part)] = make_float2(m, l);
    tc_fence_before();
    __threadfence();
    warp_arrive(bar(C::B_O_FREE));
    warp_arrive(bar(C::B_PART));
    volatile int* last = abort_flag + 1;
    if (warp == 0) {
        if (!warp_wait(bar(C::B_PART), parity, abort_flag, a.timeout_ns)) return false;
        if (lane_id() == 0) {
            __threadfence();
            const unsigned parts = static_cast<unsigned>(d.c1 - d.c0 + 1);
            const bool mine = atomicAdd(a.work.counters + d.c0, 1u) + 1u == parts;
            if (mine) a.work.counters[d.c0] = 0;   // for the next launch on this plan
            *last = mine ? 1 : 0;
            __threadfence();
            mbar_arrive(bar(C::B_JOIN));
        }
        __syncwarp();
    }
    if (!warp_wait(bar(C::B_JOIN), parity, abort_flag, a.timeout_ns)) return false;
    if (!*last) return true;
    __threadfence();   // the other CTAs' parts, published before their counts
    if (d.n_rows <= 32) return join_few_rows<D, F16, 4>(a, d, warp);
    if (d.n_rows <= 64) return join_few_rows<D, F16, 2>(a, d, warp);
    int token, head;
    uint16_t* const dst = dest_row(a, d, row, token, head);
    if (dst == nullptr) return true;
    float acc[DH];
#pragma unroll
    for (int i = 0; i < DH; ++i) acc[i] = 0.0f;
    float m_all = NO_MAX, l_all = 0.0f;
#pragma unroll 1
    for (int c = d.c0; c <= d.c1; ++c) {   // in CTA order
        const int slot = 2 * c + (c == d.c0 ? 1 : 0);
        const float2 ml = __ldcg(a.work.part_ml + at_ml(slot));
        float4 v[DH / 4];
#pragma unroll
        for (int k = 0; k < DH / 4; ++k) v[k] = __ldcg(parts_o + at_o(slot, k));
        const float m_new = fmaxf(m_all, ml.x);
        const float f0 = ex2_approx(m_all - m_new), f1 = ex2_approx(ml.x - m_new);
        m_all = m_new;
        l_all = l_all * f0 + ml.y * f1;
#pragma unroll
        for (int k = 0; k < DH / 4; ++k) {
            acc[4 * k + 0] = acc[4 * k + 0] * f0 + v[k].x * f1;
            acc[4 * k + 1] = acc[4 * k + 1] * f0 + v[k].y * f1;
            acc[4 * k + 2] = acc[4 * k + 2] * f0 + v[k].z * f1;
            acc[4 * k + 3] = acc[4 * k + 3] * f0 + v[k].w * f1;
        }
    }
    const float inv = l_all > 0.0f ? 1.0f / l_all : 0.0f;
    if (half == 0 && a.lse != nullptr) a.lse[static_cast<size_t>(token) * a.H + head] = log_sum(m_all, l_all);
#pragma unroll
    for (int q = 0; q < DH / 8; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = acc[8 * q + 2 * i] * inv, y = acc[8 * q + 2 * i + 1] * inv;
            w[i] = F16 ? pack_f16x2(x, y) : pack_bf16x2(x, y);
        }
        st_global_v4(dst + half * DH + q * 8, w[0], w[1], w[2], w[3]);
    }
    return true;
}

// Stores this thread's half row of a finished tile (O accumulator over the row's sum), and the row's log-sum-exp.
template <int D, bool F16>
__device__ __forceinline__ void store_tile(const PagedAttnArgs& a, const Piece& d, uint8_t* warp_stage, uint32_t o_base, int row,
                                           int half, float m_run, float l_row) {
    constexpr int DH = D / 2;
    const int lane = static_cast<int>(lane_id());
    int token, head;
    uint16_t* const mine = dest_row(a, d, row, token, head);
    const unsigned long long dst_row =
        mine == nullptr ? 0ull : reinterpret_cast<unsigned long long>(mine + half * DH);
    if (mine != nullptr && half == 0 && a.lse != nullptr)
        a.lse[static_cast<size_t>(token) * a.H + head] = log_sum(m_run, l_row);
    // Through a 2 KB stage per warp (32 half rows x 64 B, chunks XOR-swizzled), so that
    // 4 lanes write 64 contiguous bytes
    uint4* stage = reinterpret_cast<uint4*>(warp_stage);
    const float inv_l = l_row > 0.0f ? 1.0f / l_row : 0.0f;   // a row that saw no key: 0
#pragma unroll
    for (int q = 0; q < DH / 32; ++q) {
        uint32_t orr[32];
        tmem_ld16x2_32<DH>(o_base + q * 32, orr);
        tmem_wait_ld();
        uint32_t wv[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = __uint_as_float(orr[2 * i]) * inv_l, y = __uint_as_float(orr[2 * i + 1]) * inv_l;
            wv[i] = F16 ? pack_f16x2(x, y) : pack_bf16x2(x, y);
        }
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4)
            stage[lane * 4 + (c4 ^ (lane & 3))] =
                make_uint4(wv[4 * c4], wv[4 * c4 + 1], wv[4 * c4 + 2], wv[4 * c4 + 3]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = k * 8 + (lane >> 2);   // lane whose half row this lane stores a chunk of
            const int c4 = lane & 3;
            const uint4 v = stage[r * 4 + (c4 ^ (r & 3))];
            const unsigned long long rp = __shfl_sync(0xffffffffu, dst_row, r);
            if (rp) st_global_v4(reinterpret_cast<uint16_t*>(rp) + q * 32 + c4 * 8, v.x, v.y, v.z, v.w);
        }
        __syncwarp();   // the stage is rewritten by the next chunk
    }
}

}  // namespace
}  // namespace xs
