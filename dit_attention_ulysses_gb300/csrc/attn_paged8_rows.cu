// Attention of a few new tokens over an 8-bit paged cache: up to 8 packed query rows per KV head, 16 with heads of 64.
//
//   x_t = c 2^(E_q + E_k) <q, k_t> + E_v,  M = a running maximum of x_t,  l = sum_t 2^-E_v 2^(x_t - M),
//   O = sum_t 2^(x_t - M) v_t / l,  lse = (M + log2 l) ln 2,  c = scale log2(e),
//
// k_t and v_t the e4m3 numbers of a key, 2^E_k and 2^E_v the scales of its block, q the row as a sum
// of e4m3 numbers times 2^E_q (two for bf16, three for fp16: exact down to 2^-18 of the row's largest channel).
//
// What bounds it: the bytes of K and V, half as many as in 16 bits, so that the same card asks for twice the
// keys per second of its warps.  Hence every step of a key's way is short:
//   * both products are computed transposed, S^T = K Q^T and O^T = V^T P^T: the keys (and channels) fill the
//     m16 side of the instruction, and the query rows its n8 side, of which there are few.  A
//     row of 4 heads costs one n8 tile, where rows on the m16 side cost four times the
//     instructions and registers.
//   * K enters its product as it lies in shared memory (mma of e4m3, twice the fp16 rate).  V is
//     loaded transposed by bytes, four keys of a channel to a register, which are two cvt to fp16 and
//     no shuffle: its keys come in the order in which a thread's probabilities leave S^T and
//     the 8 x 8 transposition (see key_of_row).
//   * the ring, the pieces and their join as in attn_paged_rows.cu, except that the first copies
//     of a CTA's next piece are under way before it joins the current one (64 sequences of 8192 keys, 32 heads of 128
//     over 8, one token each: 203 -> 197 us with the transposed products, ragged 75 -> 71).
//
// The same batch with tiles of two heads: 181 us, 5.9 TB/s of 1.07 GB (158 us at the copy rate; over the 16-bit cache 324);
// 64 ragged sequences of up to 16385 keys, 126409 in all, 58.7 us, 4.4 TB/s (over the 16-bit cache 88.9, 5.8 TB/s: a tile's start
// and end, which the plan counts as 512 keys, weigh twice as much beside half the bytes); one sequence of
// 4096 keys 10.5 us, a chain of dependent trips to memory (plan, page, keys, parts), of which one of 300 keys has 7.7.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "codes8.cuh"
#include "device_wait.cuh"
#include "error_words.cuh"
#include "kernels.h"
#include "paged.h"
#include "paged_rows.cuh"
#include "paged_walk.cuh"
#include "ptx.cuh"
#include "rope_tile.cuh"

namespace xs {
namespace {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int GROUP = 32;                  // keys of a ring slot

// HP: KV heads of a tile, of up to 8 rows each (row 8 n + r: row r of head n); otherwise up to 8 NT rows of one head.
template <int D, bool F16, int NT, int HP>
struct Rows8Cfg {
    static_assert(HP == 1 || HP == NT, "");
    static constexpr int ROWS = 8 * NT;
    static constexpr int PARTS = F16 ? 3 : 2;          // numbers per channel of Q
    static constexpr int SLOT = HP * GROUP * D;
    static constexpr int SLOTS = 6 * 128 / D / HP;     // per warp
    static constexpr int RING = WARPS * SLOTS * SLOT;  // 96 KB
    static constexpr int Q_STRIDE = D + 16;            // bytes; keeps eight rows' words on different banks
    // a warp's results wait for their join in ring slots that the next piece's first copies do not use: SLOT_ROWS rows of
    // D floats to a slot, the channels of row r xor 8 (r / 2 % 4), which keeps a store's four rows on different banks
    static constexpr int SLOT_ROWS = 8 * HP;
    static constexpr int AHEAD = SLOTS - ROWS / SLOT_ROWS;
    static constexpr int Q_OFF = RING;
    static constexpr int ML_OFF = (Q_OFF + PARTS * ROWS * Q_STRIDE + 15) / 16 * 16;
    static constexpr int FACTOR_OFF = ML_OFF + WARPS * ROWS * 8;   // c 2^E_q of every row
    static constexpr int BAR_OFF = FACTOR_OFF + ROWS * 4;
    static constexpr int MISC_OFF = BAR_OFF + WARPS * SLOTS * 8;   // abort, last, first join slot of each warp
    static constexpr int SMEM = MISC_OFF + 32;
    static constexpr int ALLOC = SMEM + 1024;          // alignment of the swizzled slots
    static_assert(AHEAD >= 2, "a group of the next piece fits");
    static_assert(ALLOC <= 113 * 1024, "two CTAs per SM");
};

// e4m3 x e4m3, m16 n8 k32.
__device__ __forceinline__ void mma16832(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two 16 x 16 matrices of bytes, transposed: lane 4 g + c gets rows 4 c .. 4 c + 3 of columns g and g + 8 of each.  Rows
// of the first are at the addresses of lanes 0-15, of the second at those of lanes 16-31.
__device__ __forceinline__ void ldmatrix2_trans8(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(addr)
                 : "memory");
}

// 8 x 8 16-bit matrix over the warp, two elements of a row to a lane: transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The key, of 16, in row r of a tile of S^T: 0 .. 7, then 12 .. 15, 8 .. 11.  Lane 4 g + c then holds, once P is
// transposed, the probabilities of keys 2 c, 2 c + 1 (from rows 0-7) and of rows 8 + 2 c, 8 + 2 c + 1; V's
// bytes are loaded in the order of these (order_of_v), so that one register's four are a lane's four.  Among any
// eight rows that one step of a load touches, of K or V, no two keys are equal modulo 8: no bank conflicts.
__device__ __forceinline__ int key_of_row(int r) { return r < 8 ? r : 8 + ((r & 7) ^ 4); }
__device__ __forceinline__ int order_of_v(int r) {   // r = 4 c + s
    return key_of_row(2 * (r >> 2) + (r & 1) + ((r & 2) ? 8 : 0));
}

// Offset of the 16 channels `chunk` of a key of a slot, under TMA's swizzle of D-byte rows.
template <int D>
__device__ __forceinline__ uint32_t code_at(int key, int chunk) {
    return key * D + ((chunk ^ (D == 128 ? key & 7 : (key >> 1) & 3)) << 4);
}

template <int D, bool F16, int NT, int HP>
__global__ void __launch_bounds__(THREADS, 2)
    attn_paged8_rows_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                            const __grid_constant__ PagedAttn8Args a) {
    using C = Rows8Cfg<D, F16, NT, HP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, c4 = lane & 3;   // row and column pair of a thread in the instructions' fragments
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF);
    volatile int* last_flag = abort_flag + 1;
    volatile int* join_slot = abort_flag + 2;                            // [WARPS]
    const uint32_t ring = smem_addr(smem) + warp * C::SLOTS * C::SLOT;
    const uint32_t bars = smem_addr(smem + C::BAR_OFF) + warp * C::SLOTS * 8;
    float2* join_ml = reinterpret_cast<float2*>(smem + C::ML_OFF);       // [WARPS][ROWS]
    float* const factors = reinterpret_cast<float*>(smem + C::FACTOR_OFF);

    if (tid == 0) {
        *abort_flag = 0;
        for (int i = 0; i < WARPS * C::SLOTS; ++i) mbar_init(smem_addr(smem + C::BAR_OFF) + i * 8, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    pdl_wait();
    const PagedRange range = a.work.ranges[blockIdx.x];
    const int n_seqs = a.work.header->n_seqs, tile_heads = a.Hkv / HP;
    {
        const PagedHeader& h = *a.work.header;
        if (h.n != a.n || h.H != a.H || h.Hkv != tile_heads || h.D != D || h.tokens != a.tile.tokens ||
            h.block != a.tile.block || h.grid != a.tile.grid || h.causal != a.causal || h.window != a.window || h.cache8 != 1) {
            if (tid == 0) report_error(XS_DEVICE_BOUNDS_CODE, PAGED_MAGIC_SITE, h.n, h.tokens, h.grid);
            return;
        }
    }
    __syncthreads();

    const int page_size = 1 << a.page_shift;
    const int box = page_size < GROUP ? page_size : GROUP;   // rows of one TMA copy: 16 or 32
    const int halves = GROUP / box;
    // a slot holds units of 16 keys of a head: a copy's heads one after the other, its keys together
    const int unit_keys = halves == 2 ? HP * 16 * D : 16 * D, unit_head = halves == 2 ? 16 * D : GROUP * D;
    uint32_t k_at[D / 32], v_at[D / 32];   // a lane's offsets in a slot, by 32 channels
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        k_at[i] = code_at<D>(key_of_row((lane & 7) + (lane & 8)), 2 * i + (lane >> 4));
        v_at[i] = code_at<D>(order_of_v(lane & 15), 2 * i + (lane >> 4));
    }

    // ---- the open piece: blocks [k0, k1) of a tile; keys key0 + 32 (warp + 4 g), g < groups, are this warp's
    PagedPos pos = range.start;
    PagedSeq seq = range.first;
    int key0, groups, tok0, n_tok, lo_tile, unseen;
    bool cut_end, whole;
    uint32_t slot = 0, phase = 0;   // of the next item (K and V of a group alternately) to be waited for
    int issued;                     // items of the piece issued so far
    int pages = -1, pages_next = -1, page_base = 0, scales = 0, scales_next = 0;
    uint4 q_ahead[NT];
    const int* table;
    auto row_of = [](int r) { return HP == 1 ? r : r & 7; };                          // row of its head
    auto head_of = [](int head, int r) { return HP == 1 ? head : head * HP + (r >> 3); };   // KV head of a tile's row
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
    // scale bytes of the 16 keys `lane & 1` of group `first + lane / 2`: K's, V's << 8, the second head's << 16
    auto load_scales = [&](int first, int page) -> int {
        int w = 127 | 127 << 8 | 127 << 16 | 127 << 24;
        if (halves == 1) page = __shfl_sync(0xffffffffu, page, lane & ~1);
        if (static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages)) {
            const int off = (key_of(first + (lane >> 1)) + (lane & 1) * 16) & (page_size - 1);
            const int b = off >> a.block_shift;
            const uint8_t* k = a.k_scale + page * a.k_scale_strides[0] + b * a.k_scale_strides[1] + pos.head * HP * a.k_scale_strides[2];
            const uint8_t* v = a.v_scale + page * a.v_scale_strides[0] + b * a.v_scale_strides[1] + pos.head * HP * a.v_scale_strides[2];
            w = k[0] | v[0] << 8;
            if constexpr (HP == 2) w |= k[a.k_scale_strides[2]] << 16 | v[a.v_scale_strides[2]] << 24;
        }
        return w;
    };
    auto issue = [&](int i, uint32_t to) {   // item i of the piece, K (even) or V (odd) of group i / 2, into ring slot `to`
        const int g = i >> 1;
        const int from = ((g - page_base) & 15) * 2;
        const int src = g - page_base < 16 ? pages : pages_next;
        const int p0 = __shfl_sync(0xffffffffu, src, from), p1 = __shfl_sync(0xffffffffu, src, from + 1);
        if (lane == 0) {
            const uint32_t bar = bars + to * 8, dst = ring + to * C::SLOT;
            mbar_arrive_expect_tx(bar, C::SLOT);
            const int row = key_of(g) & (page_size - 1);
            const CUtensorMap* m = (i & 1) ? &tv : &tk;
            tma_load_4d(dst, m, bar, 0, row, pos.head * HP, p0);
            if (halves == 2) tma_load_4d(dst + C::SLOT / 2, m, bar, 0, row, pos.head * HP, p1);
        }
    };
    auto issue_up_to = [&](int most) {   // items in slots that have been read, counted from the next to be waited for
        for (; issued < most && issued < 2 * groups; ++issued) issue(issued, (slot + issued) % C::SLOTS);
    };
    // Opens the piece at `pos`; false: the plan names a tile that is not there.
    auto open_piece = [&]() -> bool {
        if (!paged_valid(pos, seq, n_seqs, a.tile.tokens, tile_heads)) {
            if (tid == 0) report_error(XS_DEVICE_BOUNDS_CODE, PAGED_MAGIC_SITE, pos.seq, pos.head, pos.tile);
            return false;
        }
        int blk0, count, hi_tile;
        paged_tile_blocks(seq, pos.tile, a.tile, a.causal, a.window, blk0, count);
        paged_tile_keys(seq, pos.tile, a.tile.tokens, a.causal, a.window, lo_tile, hi_tile);
        cut_end = paged_same_tile(pos, range.end);
        const int k1 = cut_end ? min(range.end.k, count) : count;
        whole = pos.k == 0 && !cut_end;
        key0 = (blk0 + pos.k) * a.tile.block;
        const int key1 = min((blk0 + k1) * a.tile.block, hi_tile);
        const int groups_all = key1 > key0 ? (key1 - key0 + GROUP - 1) / GROUP : 0;
        groups = groups_all > warp ? (groups_all - warp + WARPS - 1) / WARPS : 0;
        tok0 = pos.tile * a.tile.tokens;
        n_tok = min(a.tile.tokens, seq.q_len - tok0);
        unseen = paged_unseen(seq, a.window);
        table = a.table + static_cast<long long>(seq.index) * a.table_stride;
        page_base = 0;
        issued = 0;
        pages = load_pages(0);
        pages_next = load_pages(16);
#pragma unroll
        for (int i = 0; i < NT; ++i) {   // 8 channels of a row, D / 8 lanes side by side
            const int at = tid + i * THREADS, r = row_of(at / (D / 8));
            q_ahead[i] = make_uint4(0, 0, 0, 0);
            if (r < n_tok * a.G && at / (D / 8) < C::ROWS) {
                int t, gh;
                fdivmod(r, a.fd_G, t, gh);
                const long long token = static_cast<long long>(seq.q_start) + tok0 + t;
                if (token < a.T)
                    q_ahead[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + token * a.q_stride +
                                                                 (static_cast<long long>(head_of(pos.head, at / (D / 8))) * a.G + gh) * D + at % (D / 8) * 8);
            }
        }
        return true;
    };
    // Q's rows into shared memory as e4m3 numbers, rows past the tile as zeros
    auto store_q = [&]() {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int at = tid + i * THREADS, r = at / (D / 8);
            if (D == 64 && r >= C::ROWS) break;   // (whole warps)
            const uint32_t w[4] = {q_ahead[i].x, q_ahead[i].y, q_ahead[i].z, q_ahead[i].w};
            float x[8], m = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                widen<F16>(w[j], x[2 * j], x[2 * j + 1]);
                m = fmaxf(m, fmaxf(fabsf(x[2 * j]), fabsf(x[2 * j + 1])));
            }
#pragma unroll
            for (int d = D / 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            float f;
            const int e = row_scale(m, f);
            if (at % (D / 8) == 0) factors[r] = a.c * scale_value(e);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= f;
#pragma unroll
            for (int p = 0; p < C::PARTS; ++p) {
                uint32_t o[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    o[j] = to_codes(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
                    const float2 lo = f16x2_values(codes_to_f16x2(o[j])), hi = f16x2_values(codes_to_f16x2_high(o[j]));
                    x[4 * j] -= lo.x;
                    x[4 * j + 1] -= lo.y;
                    x[4 * j + 2] -= hi.x;
                    x[4 * j + 3] -= hi.y;
                }
                *reinterpret_cast<uint2*>(smem + C::Q_OFF + (p * C::ROWS + r) * C::Q_STRIDE + at % (D / 8) * 8) = make_uint2(o[0], o[1]);
            }
        }
    };

    if (!paged_before(pos, range.end) || !open_piece()) return;
    issue_up_to(C::SLOTS);
    scales = load_scales(0, pages);
    store_q();
    __syncthreads();
    bool ok = true;
    for (;;) {
        // the next piece's tile, its sequence fetched early
        PagedPos next = pos;
        PagedSeq next_seq = seq;
        bool more = false;
        if (!cut_end) {
            const bool other = paged_next(next, seq, a.tile.tokens, tile_heads);
            more = paged_before(next, range.end);
            if (other && more && next.seq < n_seqs) next_seq = a.work.seqs[next.seq];
        }
        const int n_rows = n_tok * a.G;   // of a head
        const long long base = static_cast<long long>(seq.kv_len) - seq.q_len;
        // keys [loaded, unseen) come in with the first copy although no row of the sequence sees them
        const int loaded = lo_tile & ~(box - 1);

        // this thread's rows of Q: 8 n + 2 c and 8 n + 2 c + 1
        float factor[NT][2];
        uint32_t qf[C::PARTS][NT][D / 32][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) factor[n][e] = factors[8 * n + 2 * c4 + e];
#pragma unroll
            for (int p = 0; p < C::PARTS; ++p)
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint8_t* w = smem + C::Q_OFF + (p * C::ROWS + 8 * n + g8) * C::Q_STRIDE + i * 32 + c4 * 4;
                    qf[p][n][i][0] = *reinterpret_cast<const uint32_t*>(w);
                    qf[p][n][i][1] = *reinterpret_cast<const uint32_t*>(w + 16);
                }
        }
        // keys that every row sees: [all_lo, all_hi)
        const long long all_hi = a.causal ? base + tok0 + 1 : seq.kv_len;
        const long long all_lo = a.window > 0 ? base + tok0 + n_tok - a.window : 0;

        float o[D / 16][NT][4], m_run[NT][2], l_run[NT][2];   // o: channels 16 i + g8 (+ 8) of rows 2 c, 2 c + 1
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][n][e] = 0.0f;
            m_run[n][0] = m_run[n][1] = NO_MAX;
            l_run[n][0] = l_run[n][1] = 0.0f;
        }
        scales_next = scales;

        int waited = 0;
        for (int g = 0; g < groups && ok; ++g) {
            if (g == page_base + 16) {
                pages = pages_next;
                page_base = g;
                pages_next = load_pages(g + 16);
                scales = scales_next;
            }
            if (g == page_base + 1) scales_next = load_scales(page_base + 16, pages_next);   // (the pages have arrived)
            const int key = key_of(g);
            // ---- S^T = K Q^T
            ok = ring_wait(bars + slot * 8, phase, abort_flag, a.timeout_ns, pos.seq, g);
            if (!ok) break;
            ++waited;
            float s[2][NT][4];   // keys key_of_row(g8), key_of_row(g8 + 8) of 16, rows 2 c, 2 c + 1
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[b][n][e] = 0.0f;
            const uint32_t kbase = ring + slot * C::SLOT;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int hp = 0; hp < HP; ++hp) {
                        uint32_t k[4];
                        ldmatrix4(kbase + k_at[i] + b * unit_keys + hp * unit_head, k[0], k[1], k[2], k[3]);
#pragma unroll
                        for (int p = 0; p < C::PARTS; ++p)
#pragma unroll
                            for (int n = hp; n < (HP == 1 ? NT : hp + 1); ++n)
                                mma16832(s[b][n], k, qf[p][n][i][0], qf[p][n][i][1]);
                    }
            __syncwarp();   // every lane has read the slot
            if (issued < 2 * groups) issue(issued++, slot);
            if (++slot == C::SLOTS) {
                slot = 0;
                phase ^= 1u;
            }
            // ---- softmax of the group
            const bool masked = key + GROUP > all_hi || key < all_lo;
            float v_inv[2][HP];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint32_t w = __shfl_sync(0xffffffffu, scales, (g - page_base) * 2 + b);
#pragma unroll
                for (int hp = 0; hp < HP; ++hp) {
                    // (of a block that no row sees: anything)
                    const int v = min(max(static_cast<int>(w >> (16 * hp + 8) & 255), LEAST_SCALE), 254);
                    const float k = scale_value(w >> 16 * hp & 255), v_exp = static_cast<float>(v - 127);
                    v_inv[b][hp] = inverse_scale(v);
#pragma unroll
                    for (int n = hp; n < (HP == 1 ? NT : hp + 1); ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[b][n][e] = fmaf(s[b][n][e], factor[n][e & 1] * k, v_exp);
                }
            }
            if (masked) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = row_of(8 * n + 2 * c4 + e);
                        const long long p = base + tok0 + fdiv(r, a.fd_G);
                        long long h = a.causal ? p + 1 : seq.kv_len;   // the row sees keys [l, h)
                        const long long l = a.window > 0 ? p - a.window + 1 : 0;
                        if (r >= n_rows) h = 0;
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int f = 0; f < 2; ++f) {
                                const int t = key + b * 16 + key_of_row(g8 + f * 8);
                                if (t >= h || t < l) s[b][n][2 * f + e] = __int_as_float(0xff800000);
                            }
                    }
            }
            bool moved = false;
            float alpha[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mx = fmaxf(fmaxf(s[0][n][e], s[0][n][e + 2]), fmaxf(s[1][n][e], s[1][n][e + 2]));
                    alpha[n][e] = mx;
                }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) alpha[n][e] = fmaxf(alpha[n][e], __shfl_xor_sync(0xffffffffu, alpha[n][e], d));
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mx = alpha[n][e];
                    alpha[n][e] = 1.0f;
                    if (mx - m_run[n][e] > RESCALE_THRESHOLD + HEADROOM) {
                        const float m = mx - HEADROOM;
                        alpha[n][e] = ex2_approx(m_run[n][e] - m);
                        m_run[n][e] = m;
                        moved = true;
                    }
                }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    l_run[n][0] *= alpha[n][0];
                    l_run[n][1] *= alpha[n][1];
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[i][n][e] *= alpha[n][e & 1];
                }
            }
            // P in fp16 (up to 2^15; its relative rounding, half a step, is at most of the size of the output's own), keys
            // side by side; the sum takes the fp32 values
            uint32_t pf[2][NT][2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = ex2_approx(s[b][n][e] - m_run[n][e & 1]);
                    l_run[n][0] = fmaf(p[0] + p[2], v_inv[b][HP == 1 ? 0 : n], l_run[n][0]);
                    l_run[n][1] = fmaf(p[1] + p[3], v_inv[b][HP == 1 ? 0 : n], l_run[n][1]);
                    pf[b][n][0] = transposed(pack_f16x2(p[0], p[1]));
                    pf[b][n][1] = transposed(pack_f16x2(p[2], p[3]));
                }
            // ---- O^T += V^T P^T
            ok = ring_wait(bars + slot * 8, phase, abort_flag, a.timeout_ns, pos.seq, g);
            if (!ok) break;
            ++waited;
            if (key + GROUP > seq.kv_len || (key < unseen && loaded < unseen)) {
                // what no row of the sequence sees holds whatever was there (rows of a page past its end, keys of a page
                // before its first row's window): 0 * NaN must not reach the sum
                const int bad = seq.kv_len > key ? min(seq.kv_len - key, GROUP) : 0;
                const int from = max(loaded - key, 0), low = max(min(unseen - key, GROUP) - from, 0);   // rows
                for (int i = lane; i < (low + GROUP - bad) * (D / 16) * HP; i += 32) {
                    const int j = i / (D / 16) / HP, r = j + (j < low ? from : bad - low), hp = i / (D / 16) % HP;
                    *reinterpret_cast<uint4*>(smem + (ring - smem_addr(smem)) + slot * C::SLOT + (r >> 4) * unit_keys + hp * unit_head +
                                              (r & 15) * D + i % (D / 16) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();   // before the next TMA copy into the slot
                __syncwarp();
            }
            const uint32_t vbase = ring + slot * C::SLOT;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
#pragma unroll
                    for (int hp = 0; hp < HP; ++hp) {
                        uint32_t w[4];   // channels 32 i + g8 + (0, 8, 16, 24), a lane's four keys
                        ldmatrix2_trans8(vbase + v_at[i] + b * unit_keys + hp * unit_head, w[0], w[1], w[2], w[3]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t v[4] = {codes_to_f16x2(w[2 * h]), codes_to_f16x2(w[2 * h + 1]),
                                                   codes_to_f16x2_high(w[2 * h]), codes_to_f16x2_high(w[2 * h + 1])};
#pragma unroll
                            for (int n = hp; n < (HP == 1 ? NT : hp + 1); ++n)
                                mma16816<true>(o[2 * i + h][n], v, pf[b][n][0], pf[b][n][1]);
                        }
                    }
            __syncwarp();
            if (issued < 2 * groups) issue(issued++, slot);
            if (++slot == C::SLOTS) {
                slot = 0;
                phase ^= 1u;
            }
        }
        if (!ok) {   // copies in flight land before the CTA ends
            for (int i = waited; i < issued; ++i) {
                drain_wait(bars + slot * 8, phase, 20000000ull);
                if (++slot == C::SLOTS) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
            issued = 0;
        }

        if (cut_end) pdl_launch();   // the end is near

        // ---- the tile as it is to be joined, then the next piece's first copies
        const int head = pos.head, row0 = seq.q_start + tok0;
        const bool tile_whole = whole, starts = pos.k == 0;
        int opened = 0;
        if (ok && more) {
            pos = next;
            seq = next_seq;
            opened = open_piece() ? 1 : 0;
            if (opened) {
                issue_up_to(C::AHEAD);
                scales = load_scales(0, pages);
            }
        }
        if (!opened) issued = 0;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l_run[n][e] += __shfl_xor_sync(0xffffffffu, l_run[n][e], d);
        const uint32_t first_slot = (slot + C::AHEAD) % C::SLOTS;
        auto join_at = [&](int w, uint32_t first, int r, int channel) -> float* {   // row r of warp w's results
            const uint32_t at = (first + r / C::SLOT_ROWS) % C::SLOTS;
            return reinterpret_cast<float*>(smem + (w * C::SLOTS + at) * C::SLOT) + r % C::SLOT_ROWS * D + (channel ^ (r / 2 % 4 * 8));
        };
        if (lane == 0) join_slot[warp] = static_cast<int>(first_slot);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * n + 2 * c4 + e;
                if (row_of(r) >= n_rows) continue;
                if (g8 == 0) join_ml[warp * C::ROWS + r] = make_float2(m_run[n][e], l_run[n][e]);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    *join_at(warp, first_slot, r, i * 16 + g8) = o[i][n][e];
                    *join_at(warp, first_slot, r, i * 16 + 8 + g8) = o[i][n][e + 2];
                }
            }
        __syncthreads();
        if (*abort_flag) {   // the other warps' next copies land too
            for (int i = 0; i < issued; ++i) drain_wait(bars + (slot + i) % C::SLOTS * 8, phase ^ ((slot + i) / C::SLOTS), 20000000ull);
            return;
        }
        uint32_t firsts[WARPS];
#pragma unroll
        for (int w = 0; w < WARPS; ++w) firsts[w] = static_cast<uint32_t>(join_slot[w]);
        // this piece's CTA slot: 2c + 1 for a piece that starts its tile, 2c for one that continues it
        const size_t part = 2 * static_cast<size_t>(blockIdx.x) + (starts ? 1 : 0);
        for (int i = tid; i < n_rows * HP * (D / 4); i += THREADS) {
            const int hp = i / (D / 4) % HP, r = i / (D / 4) / HP + 8 * hp, q4 = i % (D / 4);
            float m = NO_MAX;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) m = fmaxf(m, join_ml[w * C::ROWS + r].x);
            float l = 0.0f;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float2 ml = join_ml[w * C::ROWS + r];
                const float f = ex2_approx(ml.x - m);
                const float4 v = *reinterpret_cast<const float4*>(join_at(w, firsts[w], r, q4 * 4));
                l += ml.y * f;
                acc.x += v.x * f;
                acc.y += v.y * f;
                acc.z += v.z * f;
                acc.w += v.w * f;
            }
            if (tile_whole) {
                int t, gh;
                fdivmod(row_of(r), a.fd_G, t, gh);
                const int token = row0 + t;
                if (token < a.T) store_out<F16>(a, token, head_of(head, r) * a.G + gh, q4, acc, m, l);
            } else {
                *reinterpret_cast<float4*>(a.work.part_o + (part * C::ROWS + r) * D + q4 * 4) = acc;
                if (q4 == 0) a.work.part_ml[part * C::ROWS + r] = make_float2(m, l);
            }
        }
        if (!tile_whole) {
            const int c0 = starts ? static_cast<int>(blockIdx.x) : range.c0;
            const int c1 = starts ? range.c1_last : range.c1;
            const bool there = c0 >= 0 && c1 >= c0 && c1 < a.tile.grid;
            if (!there && tid == 0) report_error(XS_DEVICE_BOUNDS_CODE, PAGED_MAGIC_SITE, c0, c1, tok0);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const unsigned n_parts = static_cast<unsigned>(c1 - c0 + 1);
                const bool last = there && atomicAdd(a.work.counters + c0, 1u) + 1u == n_parts;
                if (last) a.work.counters[c0] = 0;   // for the next launch on this plan
                *last_flag = last ? 1 : 0;
            }
            __syncthreads();
            if (*last_flag) {
                __threadfence();   // the other CTAs' parts, published before their counts
                join_parts<D, C::ROWS, THREADS, HP, F16>(a, row0, head, n_rows, c0, c1);
            }
        }
        if (opened) store_q();
        fence_proxy_async_smem();   // the joined results before the next copies into the ring
        __syncthreads();
        if (!opened) break;
        issue_up_to(C::SLOTS);
    }
}

template <int D, bool F16, int NT, int HP>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttn8Args& a, cudaStream_t stream) {
    auto kern = attn_paged8_rows_kernel<D, F16, NT, HP>;
    constexpr int smem = Rows8Cfg<D, F16, NT, HP>::ALLOC;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kern, dim3(static_cast<unsigned>(a.tile.grid)), THREADS, smem, stream, tk, tv, a);
}

template <int NT, int HP>
cudaError_t launch_any(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttn8Args& a, int dtype, cudaStream_t stream) {
    if (a.D == 128) return dtype == 0 ? launch<128, false, NT, HP>(tk, tv, a, stream) : launch<128, true, NT, HP>(tk, tv, a, stream);
    return dtype == 0 ? launch<64, false, NT, HP>(tk, tv, a, stream) : launch<64, true, NT, HP>(tk, tv, a, stream);
}

}  // namespace

cudaError_t launch_attn_paged8_rows(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttn8Args& a, int dtype,
                                    cudaStream_t stream) {
    if (a.tile.heads == 2) return launch_any<2, 2>(tk, tv, a, dtype, stream);
    if (a.tile.tokens * a.G <= 8) return launch_any<1, 1>(tk, tv, a, dtype, stream);
    return dtype == 0 ? launch<64, false, 2, 1>(tk, tv, a, stream) : launch<64, true, 2, 1>(tk, tv, a, stream);
}

cudaError_t paged8_rows_error_words(ErrorWords* w) { return error_words_here(w); }

cudaError_t read_and_clear_paged8_rows_error(int* value, DeviceErrorInfo* info, int* drain_failed, unsigned long long* when) {
    return read_and_clear_error_words(value, info, drain_failed, when);
}

}  // namespace xs
