// Attention of chunks of new tokens over an 8-bit paged cache on the tcgen05 tensor cores.
//
//   x_t = c 2^(E_k) <Q, k_t> + E_v,  M = a running maximum of x_t,  l = sum_t 2^-E_v 2^(x_t - M),
//   O = sum_t 2^(x_t - M) v_t / l,  lse = (M + log2 l) ln 2,  c = scale log2(e),
//
// k_t and v_t the e4m3 numbers of a key, 2^E_k and 2^E_v the scales of its block of K and V (one
// factor and one addend per 16 scores, no work per element).  One pass over the cache in blocks of
// 128 keys; tiles, plan and TMEM as in attn_paged.cu.
//
// K enters its product as it lies in the cache (kind::f8f6f4), and Q as a sum of e4m3 numbers:
// q = 2^E_q (q_0 + q_1 (+ q_2)), q_i the nearest number to what the ones before leave, E_q the
// row's.  Each has four significant bits, so two hold a bf16 channel and three an fp16 one
// exactly, down to 2^-10 of the scale (2^-18 of the row's largest channel).  At twice the
// 16-bit rate, two products take the time of one, and K needs no conversion.
//
// V's numbers are converted to fp16 (exact) on their way: four warps read a block from the
// ring of copies and write it as the fp16 operand, keys that no row may see as zeros.  The
// probabilities go in as fp16, up to 2^15.  (As sums of e4m3 numbers they would cost the
// softmax two conversions back and forth per pair, 12 of its issue cycles, where V's
// conversion takes 2 and is another warp's.)
//
// What bounds it: 2 sequences' 2048 new tokens after 14336 each (causal, 32 heads of 128 over 8) take 785 us,
// 1310 TFLOP/s, 70 % of the measured bf16 rate; 4608 over 18432 keys, not causal, 24 heads, 793 us.  (attn_paged.cu, over
// twice the bytes: 749 and 743.)  Heads of 64, whose products are half as large: 2 x 2048 after 8192 452 us (353).  As there
// it is the softmax's chain, with two of its warps to a scheduler, and a converter beside them: the issue slots
// are busy for 57 % of the time, the tensor pipes for 58 %, the warps wait for their own results.
//
// The loops of five roles have to share the SM's instruction cache.  While they did not (MMA issuers of one lane
// each, whose operands every instruction moved to uniform registers; 90 to 94 % of the fetches hit, and the cache
// behind it, which the SMs of a GPC share, ran at 84 to 91 % of its rate: 834 us) no part was the bound: 785 without V's
// conversion, 765 with one instruction for S in place of eight, 775 without exponentials, 783 without the maximum.  Now 99 %
// hit.  Measured and not kept: masks or rescaling out of the loop, the two producers as one, smaller unrollings, the
// epilogue out of line (1 % faster to 20 % slower, by where the code came to lie), the next piece's Q before V's last
// block (+1.5 %), S of the next piece before the last PV (+1 %), a softmax of half the code in two passes over TMEM (+25 %).
//
// Organisation (one persistent CTA per SM, 16 warps):
//   warps 0-7   softmax + epilogue, two threads per row
//   warp  8     producer of V and of the scales of K and V
//   warp  9     issuer of the S MMAs and TMEM owner
//   warp 10     issuer of the O += P V MMAs
//   warp 11     producer of K: walks the CTA's part of the plan
//   warps 12-15 converters: Q of the next tile, V block by block
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_tile.cuh"
#include "codes8.cuh"
#include "device_wait.cuh"
#include "error_words.cuh"
#include "kernels.h"
#include "paged.h"
#include "paged_chunk.cuh"
#include "paged_walk.cuh"
#include "ptx.cuh"
#include "rope_tile.cuh"

namespace xs {
namespace {

constexpr int NUM_THREADS = 512;
constexpr int WARP_V = 8;
constexpr int WARP_MMA_S = 9;
constexpr int WARP_MMA_PV = 10;
constexpr int WARP_K = 11;
constexpr int WARP_CONVERT = 12;
constexpr int CONVERTERS = 4;
// Registers of a thread by warpgroup: 2 * 168 + 80 + 96 = 4 * 128, what the block is launched with
constexpr int REGS_SOFTMAX = 168, REGS_ISSUE = 80, REGS_CONVERT = 96;
constexpr int SCALE_SLOTS = 8;      // blocks whose scales are kept (see load_blocks)

// Scales of 16 keys.
struct alignas(16) Scales {
    float k;       // 2^E_k
    float v;       // E_v
    float v_inv;   // 2^-E_v
    float unused;
};

template <int D, bool F16>
struct Cfg8 {
    static constexpr int PARTS = F16 ? 3 : 2;              // numbers per channel of Q
    static constexpr int Q_PANELS = (PARTS * D + 127) / 128;   // 128 rows x 128 bytes
    static constexpr int Q_BYTES = Q_PANELS * PANEL_BYTES;
    static constexpr int CODE_BYTES = BLOCK_N * D;         // a block of K or V in the cache's form: [key][D]
    static constexpr int V_BYTES = BLOCK_N * D * 2;        // as the fp16 operand: [8 keys][panel][key][64 channels]
    static constexpr int GROUP = D / 64 * 1024;
    static constexpr int K_STAGES = D == 128 ? (F16 ? 2 : 3) : 5;
    static constexpr int C_STAGES = D == 128 ? 3 : 4;      // copies of V
    static constexpr int V_STAGES = D == 128 ? 2 : 3;      // operands
    static constexpr int Q_OFF = 0;
    static constexpr int V_OFF = Q_OFF + Q_BYTES;
    static constexpr int K_OFF = V_OFF + V_STAGES * V_BYTES;
    static constexpr int C_OFF = K_OFF + K_STAGES * CODE_BYTES;
    static constexpr int STAGE_OFF = C_OFF + C_STAGES * CODE_BYTES;   // epilogue staging, 2 KB per softmax warp
    static constexpr int SCALES_OFF = STAGE_OFF + NUM_SOFTMAX_WARPS * 2048;
    static constexpr int FACTOR_OFF = SCALES_OFF + SCALE_SLOTS * 8 * 16;   // [2][128] c 2^E_q of every row
    static constexpr int BAR_OFF = FACTOR_OFF + 2 * BLOCK_M * 4;
    static constexpr int B_Q_FULL = 0;                 // [1]  converters -> MMA
    static constexpr int B_Q_FREE = 1;                 // [2]  MMA -> producer of K, converters, by piece
    static constexpr int B_FACTOR = 3;                 // [2]  converters -> softmax, by piece
    static constexpr int B_S_FULL = 5;                 // [3]  S MMA -> softmax, per S buffer
    static constexpr int B_P_FULL = 8;                 // [3]  softmax -> PV MMA
    static constexpr int B_P_FREE = 11;                // [3]  PV MMA -> S MMA / rescale
    static constexpr int B_O_FINAL = 14;               // [1]  MMA -> epilogue
    static constexpr int B_O_FREE = 15;                // [1]  epilogue -> MMA
    static constexpr int B_DRAIN = 16;                 // [1]  both issuers
    static constexpr int B_PIECE = 17;                 // [4]  producer -> all: descriptor written
    static constexpr int B_PART = 21;                  // [1]  softmax warps -> warp 0: part written
    static constexpr int B_JOIN = 22;                  // [1]  warp 0 -> softmax warps: who joins
    static constexpr int B_SCALES = 23;                // [8]  producer of V -> softmax
    static constexpr int B_K_FULL = 31;                // [K_STAGES] TMA -> MMA
    static constexpr int B_K_FREE = B_K_FULL + K_STAGES;
    static constexpr int B_C_FULL = B_K_FREE + K_STAGES;   // [C_STAGES] TMA -> converters
    static constexpr int B_C_FREE = B_C_FULL + C_STAGES;
    static constexpr int B_V_FULL = B_C_FREE + C_STAGES;   // [V_STAGES] converters -> MMA
    static constexpr int B_V_FREE = B_V_FULL + V_STAGES;
    static constexpr int NUM_BARS = B_V_FREE + V_STAGES;
    static constexpr int PIECE_OFF = (BAR_OFF + NUM_BARS * 8 + 63) / 64 * 64;
    static constexpr int MISC_OFF = PIECE_OFF + PIECES * 64;
    static constexpr int LOADED_OFF = MISC_OFF + 16;   // per stage of K, of V: one more than the round of its newest copy
    static constexpr int SMEM_BYTES = LOADED_OFF + (K_STAGES + C_STAGES) * 4;
    static constexpr int SMEM_ALLOC = SMEM_BYTES + 1024;
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
    static_assert(K_STAGES <= 5, "a block's scales are read before their slot is written again");
};

// kind::f8f6f4, both operands e4m3 and K-major, fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// kind::f16, fp16 operands, B MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N) {
    return (1u << 4) | (1u << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ void mma_ss_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of K-major rows of D bytes, 8-row atoms swizzled over them.
template <int D>
__device__ __forceinline__ uint64_t code_desc(uint32_t saddr) {
    const uint64_t d = smem_desc_sw128(saddr, 16, 8 * D);
    return D == 128 ? d : (d & ~(7ull << 61)) | (4ull << 61);   // 4: 64-byte swizzle
}

template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The waits of device_wait.cuh, in line as far as their first test.  With every wait in line (700 bytes each) and the
// producers' loops apart, 41 % of the warps' time went to instruction fetches (the causal chunk above: 1474 us).  Not the
// softmax's: a call in its loop moves its registers to memory and back (1488 us).
__device__ __noinline__ bool warp_wait_on(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t timeout_ns, int unit,
                                          int blk) {
    return warp_wait(bar, parity, abort_flag, timeout_ns, unit, blk);
}

__device__ __forceinline__ bool all_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t timeout_ns, int unit,
                                         int blk = -1) {
    return __all_sync(0xffffffffu, mbar_test_wait(bar, parity)) || warp_wait_on(bar, parity, abort_flag, timeout_ns, unit, blk);
}

// --------------------------------------------------------------- producers
// Loads the blocks of a piece: K's, or V's and the scales of both.  By a whole warp: a block's stage is waited for by
// one lane, then each of up to eight lanes issues one page's copy.
//
// Lane 8 j + i has the scales of keys 16 i .. 16 i + 15 of block 4 m + j; they are fetched a group of four blocks
// ahead of use, from the pages of that group, fetched one more ahead.  Those of block g (counted over the CTA's
// lifetime) lie in slot g % 8 until those of block g + 8 are written: after the stage of V(g + 8)'s copy was given back,
// V(g + 8 - C_STAGES) converted, hence (its operand's stage) PV(g + 8 - C_STAGES - V_STAGES) done, which is g or later:
// after the softmax of block g.
template <int D, bool F16>
__device__ __forceinline__ bool load_blocks(const CUtensorMap* map, const PagedAttn8Args& a, uint8_t* smem, uint32_t bar0,
                                         const Piece& piece, int u, uint32_t item, bool is_v, volatile int* abort_flag) {
    using C = Cfg8<D, F16>;
    static_assert(C::C_STAGES + C::V_STAGES <= SCALE_SLOTS, "see above");
    const int lane = static_cast<int>(lane_id());
    auto bar = [&](int i) { return bar0 + static_cast<uint32_t>(i) * 8u; };
    const Piece d = piece;
    const int box = 1 << (a.page_shift < 7 ? a.page_shift : 7);   // keys of one copy
    const int boxes = BLOCK_N / box;                              // 1 .. 8
    const uint32_t stages = is_v ? C::C_STAGES : C::K_STAGES;
    const uint32_t base = smem_addr(smem + (is_v ? C::C_OFF : C::K_OFF));
    const uint32_t full0 = bar(is_v ? C::B_C_FULL : C::B_K_FULL), free0 = bar(is_v ? C::B_C_FREE : C::B_K_FREE);
    volatile uint32_t* const loaded = reinterpret_cast<volatile uint32_t*>(smem + C::LOADED_OFF) + (is_v ? C::K_STAGES : 0);
    Scales* const scales = reinterpret_cast<Scales*>(smem + C::SCALES_OFF);
    const int* table = a.table + static_cast<long long>(d.index) * a.table_stride;
    auto scales_of = [&](int m, int pages) {   // bytes of K's, V's << 8
        const int page = __shfl_sync(0xffffffffu, pages, (lane & 24) + (lane & 7) * 16 / box);
        int w = 127 | 127 << 8;
        if (static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages)) {
            const int off = (d.key0 + (4 * m + (lane >> 3)) * BLOCK_N + (lane & 7) * 16) & ((1 << a.page_shift) - 1);
            const int b = off >> a.block_shift;
            w = a.k_scale[page * a.k_scale_strides[0] + b * a.k_scale_strides[1] + d.head * a.k_scale_strides[2]] |
                a.v_scale[page * a.v_scale_strides[0] + b * a.v_scale_strides[1] + d.head * a.v_scale_strides[2]] << 8;
        }
        return w;
    };
    int cur = -1, next = -1, after = -1, bytes = 0, bytes_next = 0;   // of groups m, m + 1, m + 2
    uint32_t stage = item % stages, round = item / stages;
#pragma unroll 1
    for (int j = -8; j < d.nb; ++j) {   // (two groups before the first block fill the pipeline)
        if ((j & 3) == 0) {
            cur = next;
            next = after;
            after = load_pages(a, table, (j >> 2) + 2, d.key0, d.nb, d.kv_len, d.lo_key, boxes, box);
            bytes = bytes_next;
            if (is_v && j >= -4) bytes_next = scales_of((j >> 2) + 1, next);
            if (j < 0) {
                j += 3;
                continue;
            }
        }
        const bool ok = round == 0 || all_wait(free0 + stage * 8u, (round - 1) & 1, abort_flag, a.timeout_ns, u, j);
        if (ok && lane == 0) {
            mbar_arrive_expect_tx(full0 + stage * 8u, BLOCK_N * D);
            loaded[stage] = round + 1;
        }
        const int page = __shfl_sync(0xffffffffu, cur, (j & 3) * 8 + (lane & 7));
        __syncwarp();
        if (!ok) return false;
        if (lane < boxes)
            tma_load_4d(base + stage * (BLOCK_N * D) + lane * box * D, map, full0 + stage * 8u, 0,
                        (d.key0 + j * BLOCK_N) & ((1 << a.page_shift) - 1), d.head, page);
        if (is_v) {
            const uint32_t slot = item % SCALE_SLOTS;
            if ((lane >> 3) == (j & 3)) {
                // (of keys that no row sees: anything; a factor that stays positive keeps their scores at -infinity)
                const int k = min(max(bytes & 255, 1), 254), v = min(max(bytes >> 8, LEAST_SCALE), 254);
                scales[slot * 8 + (lane & 7)] =
                    Scales{scale_value(k), static_cast<float>(v - 127), inverse_scale(v), 0.0f};
            }
            warp_arrive(bar(C::B_SCALES + slot));
        }
        ++item;
        if (++stage == stages) {
            stage = 0;
            ++round;
        }
    }
    return true;
}

// A descriptor slot is reused four pieces later: the producer is then past the S MMAs of piece u - 2, whose first
// one waited for the last PV of the piece before, so every role has left piece u - 4.
template <int D, bool F16>
__device__ void producer_k_role(const CUtensorMap* tk, const PagedAttn8Args& a, uint8_t* smem, uint32_t bar0,
                                volatile int* abort_flag) {
    using C = Cfg8<D, F16>;
    const int lane = static_cast<int>(lane_id());
    auto bar = [&](int i) { return bar0 + static_cast<uint32_t>(i) * 8u; };
    const int box = 1 << (a.page_shift < 7 ? a.page_shift : 7);
    PieceWalk walk(a, 1);
    uint32_t item = 0;
    bool ok = true;
#pragma unroll 1
    for (int u = 0;; ++u) {
        if (u >= 2) {
            ok = all_wait(bar(C::B_Q_FREE + (u & 1)), ((u >> 1) - 1) & 1, abort_flag, a.timeout_ns, u);
        }
        if (!ok) break;
        Piece d{};
        const bool more = walk.describe(a, box, d);
        if (lane == 0) {
            *reinterpret_cast<Piece*>(smem + C::PIECE_OFF + (u % PIECES) * 64) = d;
            mbar_arrive(bar(C::B_PIECE + u % PIECES));   // release: the descriptor is visible to whoever waits
        }
        __syncwarp();
        if (!more) break;
        if (walk.cut_end) pdl_launch();   // the CTA's last piece
        if (!load_blocks<D, F16>(tk, a, smem, bar0, piece_of(smem, C::PIECE_OFF, u), u, item, false, abort_flag)) break;
        item += d.nb;
        walk.advance(a);
    }
    __syncwarp();
}

template <int D, bool F16>
__device__ void producer_v_role(const CUtensorMap* tv, const PagedAttn8Args& a, uint8_t* smem, uint32_t bar0,
                                volatile int* abort_flag) {
    using C = Cfg8<D, F16>;
    uint32_t item = 0;
#pragma unroll 1
    for (int u = 0;; ++u) {
        if (!all_wait(bar0 + (C::B_PIECE + u % PIECES) * 8u, (u / PIECES) & 1, abort_flag, a.timeout_ns, u)) break;
        const Piece& d = piece_of(smem, C::PIECE_OFF, u);
        const int n = d.nb;
        if (n == 0 || !load_blocks<D, F16>(tv, a, smem, bar0, d, u, item, true, abort_flag)) break;
        item += n;
    }
    __syncwarp();
}

// --------------------------------------------------------------- converters
// Q of a piece: thread t holds 16 channels at a time, a row's D / 16 threads side by side.
template <int D, bool F16>
__device__ __forceinline__ void convert_q(const PagedAttn8Args& a, const Piece& d, uint8_t* smem, int tid, float* factor) {
    using C = Cfg8<D, F16>;
    constexpr int PER_ROW = D / 16, ROWS = CONVERTERS * 32 / PER_ROW, BATCH = 2;
    const int piece = tid % PER_ROW;
    uint4 w[BATCH][2], next[BATCH][2];
    auto fetch = [&](int r0) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = r0 + i * ROWS;
            int t, gh;
            fdivmod(r, a.fd_G, t, gh);
            const int token = d.row0 + t;
            next[i][0] = next[i][1] = make_uint4(0, 0, 0, 0);
            if (r < d.n_rows && token >= 0 && token < a.T) {
                const uint4* p = reinterpret_cast<const uint4*>(
                    static_cast<const uint16_t*>(a.q) + token * a.q_stride + (static_cast<long long>(d.head) * a.G + gh) * D + piece * 16);
                next[i][0] = p[0];
                next[i][1] = p[1];
            }
        }
    };
    fetch(tid / PER_ROW);
#pragma unroll 1
    for (int r0 = tid / PER_ROW; r0 < BLOCK_M; r0 += BATCH * ROWS) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            w[i][0] = next[i][0];
            w[i][1] = next[i][1];
        }
        fetch(r0 + BATCH * ROWS);   // (past the rows: nothing)
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = r0 + i * ROWS;
            float x[16], m = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint4& v = w[i][j >> 2];
                widen<F16>((j & 3) == 0 ? v.x : (j & 3) == 1 ? v.y : (j & 3) == 2 ? v.z : v.w, x[2 * j], x[2 * j + 1]);
                m = fmaxf(m, fmaxf(fabsf(x[2 * j]), fabsf(x[2 * j + 1])));
            }
#pragma unroll
            for (int s = PER_ROW / 2; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
            float f;
            const int e = row_scale(m, f);
            if (piece == 0) factor[r] = a.c * scale_value(e);
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] *= f;
#pragma unroll
            for (int k = 0; k < C::PARTS; ++k) {
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o[j] = to_codes(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
                    if (k + 1 < C::PARTS) {
                        const float2 lo = f16x2_values(codes_to_f16x2(o[j])), hi = f16x2_values(codes_to_f16x2_high(o[j]));
                        x[4 * j] -= lo.x;
                        x[4 * j + 1] -= lo.y;
                        x[4 * j + 2] -= hi.x;
                        x[4 * j + 3] -= hi.y;
                    }
                }
                const int at = k * D + piece * 16;
                *reinterpret_cast<uint4*>(smem + C::Q_OFF + (at >> 7) * PANEL_BYTES + r * 128 + ((((at >> 4) & 7) ^ (r & 7)) << 4)) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

// A thread's part of V's conversion: a 16-byte piece of every KEYS-th key, read at code + n KEYS D, written as two at
// lo and hi + n KEYS D 2 (KEYS a multiple of 8, so that the swizzles of all its keys are the same).  Eight lanes read
// and write different banks: two keys, with D = 128 the first half of one and the second half of the other.
template <int D>
struct ConvertV {
    static constexpr int GROUP = D / 64 * 1024, KEYS = CONVERTERS * 32 * 16 / D;
    uint32_t code, lo, hi;   // offsets
    int key;

    __device__ __forceinline__ explicit ConvertV(int tid) {
        const int pair = D == 128 ? tid >> 4 : tid >> 3, odd = (tid >> 2) & 1;
        const int piece = (tid & 3) + (D == 128 ? 4 * (odd ^ ((tid >> 3) & 1)) : 0);
        key = 2 * pair + odd;
        const int r = key & 7;
        code = key * D + ((piece ^ (D == 128 ? r : r >> 1)) << 4);
        const uint32_t row = (key >> 3) * GROUP + (piece >> 2) * 1024 + r * 128;
        lo = row + ((((2 * piece) & 7) ^ r) << 4);
        hi = row + ((((2 * piece + 1) & 7) ^ r) << 4);
    }

    // Keys outside [from, to) become zeros.
    __device__ __forceinline__ void block(const uint8_t* from_code, uint8_t* v, int from, int to) const {
        const bool edge = from > 0 || to < BLOCK_N;
#pragma unroll 4
        for (int n = 0; n < BLOCK_N / KEYS; ++n) {
            uint4 w = *reinterpret_cast<const uint4*>(from_code + code + n * (KEYS * D));
            if (edge && (key + n * KEYS < from || key + n * KEYS >= to)) w = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(v + lo + n * (KEYS * D * 2)) =
                make_uint4(codes_to_f16x2(w.x), codes_to_f16x2_high(w.x), codes_to_f16x2(w.y), codes_to_f16x2_high(w.y));
            *reinterpret_cast<uint4*>(v + hi + n * (KEYS * D * 2)) =
                make_uint4(codes_to_f16x2(w.z), codes_to_f16x2_high(w.z), codes_to_f16x2(w.w), codes_to_f16x2_high(w.w));
        }
    }
};

template <int D, bool F16>
__device__ void convert_role(const PagedAttn8Args& a, uint8_t* smem, uint32_t bar0, volatile int* abort_flag) {
    using C = Cfg8<D, F16>;
    const int tid = threadIdx.x - WARP_CONVERT * 32;
    const ConvertV<D> convert_v(tid);
    auto bar = [&](int i) { return bar0 + static_cast<uint32_t>(i) * 8u; };
    uint32_t item = 0;
    bool ok = true;
    for (int u = 0; ok; ++u) {
        ok = all_wait(bar(C::B_PIECE + u % PIECES), (u / PIECES) & 1, abort_flag, a.timeout_ns, u);
        if (!ok) break;
        const Piece d = piece_of(smem, C::PIECE_OFF, u);
        if (d.nb == 0) break;
        // the previous piece's S MMAs have read Q
        if (u > 0) ok = all_wait(bar(C::B_Q_FREE + ((u - 1) & 1)), ((u - 1) >> 1) & 1, abort_flag, a.timeout_ns, u);
        if (!ok) break;
        convert_q<D, F16>(a, d, smem, tid, reinterpret_cast<float*>(smem + C::FACTOR_OFF) + (u & 1) * BLOCK_M);
        fence_proxy_async_smem();   // before the MMAs read it
        __syncwarp();
        if (lane_id() == 0) {
            mbar_arrive(bar(C::B_Q_FULL));
            mbar_arrive(bar(C::B_FACTOR + (u & 1)));
        }
        for (int j = 0; j < d.nb; ++j, ++item) {
            const uint32_t cs = item % C::C_STAGES, vs = item % C::V_STAGES, cr = item / C::C_STAGES, vr = item / C::V_STAGES;
            if (vr > 0) ok = all_wait(bar(C::B_V_FREE + vs), (vr - 1) & 1, abort_flag, a.timeout_ns, u, j);
            if (ok) ok = all_wait(bar(C::B_C_FULL + cs), cr & 1, abort_flag, a.timeout_ns, u, j);
            if (!ok) break;
            convert_v.block(smem + C::C_OFF + cs * C::CODE_BYTES, smem + C::V_OFF + vs * C::V_BYTES,
                            d.unseen - d.key0 - j * BLOCK_N, d.kv_len - d.key0 - j * BLOCK_N);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane_id() == 0) {
                mbar_arrive(bar(C::B_V_FULL + vs));
                mbar_arrive(bar(C::B_C_FREE + cs));
            }
        }
    }
    __syncwarp();
}

// --------------------------------------------------------------------- MMA
// Both issuers run as whole warps, with one elected thread at the instructions: what these take (descriptors, TMEM
// addresses) is then uniform, in registers where they can use it.  With one lane in the role, a dozen instructions
// more per MMA moved it there (causal chunk 834 us, video 825, 24 mixed requests with heads of 64 25.6; now 788, 795, 22.2).
//
// Issuer of S(j) = Q K_j^T into S buffer (block index) % 3: the parts of Q one after the other.
template <int D, bool F16>
__device__ void mma_s_role(const PagedAttn8Args& a, uint8_t* smem, uint32_t bar0, uint32_t tmem_base, volatile int* abort_flag) {
    using C = Cfg8<D, F16>;
    auto bar = [&](int i) { return bar0 + static_cast<uint32_t>(i) * 8u; };
    constexpr uint32_t IDESC = idesc_e4m3(BLOCK_M, BLOCK_N);
    const uint64_t qdesc = smem_desc_sw128(smem_addr(smem + C::Q_OFF), 16, 1024);
    const uint64_t kdesc0 = code_desc<D>(smem_addr(smem + C::K_OFF));
    uint32_t g = 0;             // key blocks over the CTA's lifetime
    uint32_t sb = 0, sph = 0;   // S buffer of block g (g % 3) and its phase parity ((g / 3) & 1)
    bool ok = true;
    for (int u = 0; ok; ++u) {
        ok = all_wait(bar(C::B_PIECE + u % PIECES), (u / PIECES) & 1, abort_flag, a.timeout_ns, u);
        if (!ok) break;
        const int n = __shfl_sync(0xffffffffu, piece_of(smem, C::PIECE_OFF, u).nb, 0);
        if (n == 0) break;
        ok = all_wait(bar(C::B_Q_FULL), u & 1, abort_flag, a.timeout_ns, u);
        // the previous piece's last PV first: its epilogue waits for it
        if (ok && u > 0) ok = all_wait(bar(C::B_O_FINAL), (u - 1) & 1, abort_flag, a.timeout_ns, u);
        for (int j = 0; j < n && ok; ++j, ++g) {
            if (g >= S_BUFS) ok = all_wait(bar(C::B_P_FREE + sb), sph ^ 1u, abort_flag, a.timeout_ns, u, j);
            const uint32_t stage = g % C::K_STAGES;
            if (ok) ok = all_wait(bar(C::B_K_FULL + stage), (g / C::K_STAGES) & 1, abort_flag, a.timeout_ns, u, j);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kdesc = desc_add(kdesc0, stage * (C::CODE_BYTES >> 4));
            if (elect_one()) {
#pragma unroll
                for (int p = 0; p < C::PARTS; ++p)
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk) {
                        const int at = p * D + kk * 32;   // byte of a Q row
                        mma_ss_e4m3(tmem_base + S_COL + sb * 128u, desc_add(qdesc, ((at >> 7) * PANEL_BYTES + (at & 127)) >> 4),
                                    desc_add(kdesc, kk * 2), IDESC, p > 0 || kk > 0);
                    }
                mma_commit(bar(C::B_S_FULL + sb));
                mma_commit(bar(C::B_K_FREE + stage));
                if (j == n - 1) mma_commit(bar(C::B_Q_FREE + (u & 1)));
            }
            __syncwarp();
            if (++sb == S_BUFS) {
                sb = 0;
                sph ^= 1u;
            }
        }
    }
    // B_DRAIN completes when both issuers' MMAs have all completed (TMEM is freed after it)
    if (elect_one()) mma_commit(bar(C::B_DRAIN));
    __syncwarp();
    drain_wait(bar(C::B_DRAIN), 0, a.timeout_ns > 20000000ull ? a.timeout_ns : 20000000ull);
}

// Issuer of PV(j): O += P(j) V_j.
template <int D, bool F16>
__device__ void mma_pv_role(const PagedAttn8Args& a, uint8_t* smem, uint32_t bar0, uint32_t tmem_base, volatile int* abort_flag) {
    using C = Cfg8<D, F16>;
    auto bar = [&](int i) { return bar0 + static_cast<uint32_t>(i) * 8u; };
    constexpr uint32_t IDESC = idesc_f16(BLOCK_M, D);
    const uint64_t vdesc0 = smem_desc_sw128(smem_addr(smem + C::V_OFF), 1024, C::GROUP);
    uint32_t g = 0;
    uint32_t pb = 0, pph = 0;   // buffer of block g (g % 3) and its phase parity ((g / 3) & 1)
    bool ok = true;
    for (int u = 0; ok; ++u) {
        ok = all_wait(bar(C::B_PIECE + u % PIECES), (u / PIECES) & 1, abort_flag, a.timeout_ns, u);
        if (!ok) break;
        const int n = __shfl_sync(0xffffffffu, piece_of(smem, C::PIECE_OFF, u).nb, 0);
        if (n == 0) break;
        for (int j = 0; j < n && ok; ++j, ++g) {
            ok = all_wait(bar(C::B_P_FULL + pb), pph, abort_flag, a.timeout_ns, u, j);
            // the epilogue has read the previous piece's O (PV(0) overwrites it)
            if (ok && j == 0 && u > 0) ok = all_wait(bar(C::B_O_FREE), (u - 1) & 1, abort_flag, a.timeout_ns, u, j);
            const uint32_t stage = g % C::V_STAGES;
            if (ok) ok = all_wait(bar(C::B_V_FULL + stage), (g / C::V_STAGES) & 1, abort_flag, a.timeout_ns, u, j);
            if (!ok) break;
            tc_fence_after();
            const uint64_t vdesc = desc_add(vdesc0, stage * (C::V_BYTES >> 4));
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < BLOCK_N / 16; ++kk)
                    mma_ts(tmem_base + O_COL, tmem_base + S_COL + pb * 128u + kk * 8, desc_add(vdesc, kk * (2 * C::GROUP >> 4)),
                           IDESC, j > 0 || kk > 0);
                mma_commit(bar(C::B_P_FREE + pb));
                mma_commit(bar(C::B_V_FREE + stage));
                if (j == n - 1) mma_commit(bar(C::B_O_FINAL));
            }
            __syncwarp();
            if (++pb == S_BUFS) {
                pb = 0;
                pph ^= 1u;
            }
        }
    }
    if (elect_one()) mma_commit(bar(C::B_DRAIN));
    __syncwarp();
    drain_wait(bar(C::B_DRAIN), 0, a.timeout_ns > 20000000ull ? a.timeout_ns : 20000000ull);
}

// ------------------------------------------------------- softmax + epilogue
// Maximum of 16 scores: two 3-input chains.
__device__ __forceinline__ float max16(const uint32_t* s) {
    float m0 = __uint_as_float(s[0]), m1 = __uint_as_float(s[1]);
#pragma unroll
    for (int i = 2; i < 14; i += 4) {
        m0 = fmax3(m0, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
        m1 = fmax3(m1, __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
    }
    return fmax3(m0, m1, fmaxf(__uint_as_float(s[14]), __uint_as_float(s[15])));
}

// 2^(s f + add) of 16 scores, packed to fp16 pairs (off by half a step relative to each: of the size of the output's
// own rounding in fp16, an eighth of it in bf16); returns their sum.
__device__ __forceinline__ float exp16(const uint32_t* s, float f, float add, uint32_t* pk) {
    const uint64_t ff = f2_pack(f, f), dd = f2_pack(add, add);
    uint64_t sum[2] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f)};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float x0, x1;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), ff, dd), x0, x1);
        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
        sum[i & 1] = f2_add(sum[i & 1], f2_pack(p0, p1));
        pk[i] = pack_f16x2(p0, p1);
    }
    float a0, a1;
    f2_unpack(f2_add(sum[0], sum[1]), a0, a1);
    return a0 + a1;
}

template <int D, bool F16>
__device__ void softmax_role(const PagedAttn8Args& a, uint8_t* smem, uint32_t bar0, uint32_t tmem_base,
                             volatile int* abort_flag) {
    using C = Cfg8<D, F16>;
    constexpr int DH = D / 2;  // O columns owned by each of a row's two threads
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = static_cast<int>(lane_id());
    const int quarter = warp & 3;             // TMEM lane quarter this warp may access
    const int half = lane >> 4;               // key columns [64*half, 64*half + 64), O columns [DH*half, +DH)
    const int warp_row = quarter * 32 + (warp >> 2) * 16;   // the warp's first row
    const int row = warp_row + (lane & 15);
    const uint32_t t_base = tmem_base + (static_cast<uint32_t>(warp_row) << 16);
    auto bar = [&](int i) { return bar0 + static_cast<uint32_t>(i) * 8u; };
    const Scales* const all_scales = reinterpret_cast<const Scales*>(smem + C::SCALES_OFF) + half * 4;

    uint32_t g = 0;              // key blocks over the CTA's lifetime
    uint32_t sb = 0, sph = 0;    // S buffer of block g (g % 3) and its phase parity ((g / 3) & 1)
    uint32_t pb = 2, pph = 1;    // the same for block g - 1 (the O rescale waits for PV(g-1))
    int u = 0, n_parts = 0;
    bool ok = true;
    for (; ok; ++u) {
        ok = warp_wait(bar(C::B_PIECE + u % PIECES), (u / PIECES) & 1, abort_flag, a.timeout_ns, u);
        if (!ok) break;
        const Piece& d = piece_of(smem, C::PIECE_OFF, u);
        const int n = __shfl_sync(0xffffffffu, d.nb, 0);
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
        ok = warp_wait(bar(C::B_FACTOR + (u & 1)), (u >> 1) & 1, abort_flag, a.timeout_ns, u);
        if (!ok) break;
        const float factor = reinterpret_cast<const float*>(smem + C::FACTOR_OFF)[(u & 1) * BLOCK_M + row];
        float m_run = NO_MAX, l_run = 0.0f;
        for (int j = 0; j < n; ++j, ++g) {
            const uint32_t slot = g % SCALE_SLOTS;
            ok = warp_wait(bar(C::B_SCALES + slot), (g / SCALE_SLOTS) & 1, abort_flag, a.timeout_ns, u, j);
            if (ok) ok = warp_wait(bar(C::B_S_FULL + sb), sph, abort_flag, a.timeout_ns, u, j);
            if (!ok) break;
            if (!idle) {
                tc_fence_after();
                uint32_t sr[2][32];
                tmem_ld16x2_32<64>(t_base + S_COL + sb * 128u, sr[0]);
                tmem_ld16x2_32<64>(t_base + S_COL + sb * 128u + 32, sr[1]);
                Scales z[4];
                float f[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    z[b] = all_scales[slot * 8 + b];
                    f[b] = fmaxf(factor * z[b].k, 1.17549435e-38f);   // never 0: a masked score is -infinity and stays so
                }
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
                float m_half = NO_MAX;
#pragma unroll
                for (int b = 0; b < 4; ++b) m_half = fmaxf(m_half, fmaf(max16(&sr[b >> 1][(b & 1) * 16]), f[b], z[b].v));
                const float m_blk = fmaxf(m_half, __shfl_xor_sync(0xffffffffu, m_half, 16));
                float m_use = m_run, alpha = 1.0f;
                bool rescale = false;
                if (m_blk - m_run > RESCALE_THRESHOLD) {
                    m_use = m_blk;
                    alpha = ex2_approx(m_run - m_blk);
                    rescale = j > 0;
                }
                uint32_t pk[32];
                float sum = 0.0f;
                const float ref = m_use - HEADROOM;   // what P, l and O are relative to
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    sum = fmaf(exp16(&sr[b >> 1][(b & 1) * 16], f[b], z[b].v - ref, pk + b * 8), z[b].v_inv, sum);
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
        m_run -= HEADROOM;
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
    attn_paged8_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                       const __grid_constant__ PagedAttn8Args args) {
    using C = Cfg8<D, F16>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t bar0 = smem_addr(smem + C::BAR_OFF);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);   // [1]: who joins a cut tile
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);   // (uniform, as the compiler sees)

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NUM_BARS; ++i) {
            const bool by_warp = i == C::B_Q_FULL || (i >= C::B_FACTOR && i < C::B_FACTOR + 2) ||
                                 (i >= C::B_C_FREE && i < C::B_C_FREE + C::C_STAGES) ||
                                 (i >= C::B_V_FULL && i < C::B_V_FULL + C::V_STAGES);   // the converters
            const bool by_softmax = (i >= C::B_P_FULL && i < C::B_P_FULL + S_BUFS) || i == C::B_O_FREE || i == C::B_PART;
            mbar_init(bar0 + 8 * i, by_warp ? CONVERTERS : by_softmax ? NUM_SOFTMAX_WARPS : i == C::B_DRAIN ? 2 : 1);
        }
        for (int s = 0; s < C::K_STAGES + C::C_STAGES; ++s) reinterpret_cast<uint32_t*>(smem + C::LOADED_OFF)[s] = 0;
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == WARP_K && lane_id() == 0) {
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    if (warp == WARP_MMA_S) {
        tmem_alloc(smem_addr(tmem_holder), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    pdl_wait();

    if (warp < NUM_SOFTMAX_WARPS) {
        regs_up<REGS_SOFTMAX>();
        softmax_role<D, F16>(args, smem, bar0, tmem_base, abort_flag);
    } else if (warp < WARP_CONVERT) {
        regs_down<REGS_ISSUE>();
        if (warp == WARP_K)
            producer_k_role<D, F16>(&tk, args, smem, bar0, abort_flag);
        else if (warp == WARP_V)
            producer_v_role<D, F16>(&tv, args, smem, bar0, abort_flag);
        else if (warp == WARP_MMA_PV)
            mma_pv_role<D, F16>(args, smem, bar0, tmem_base, abort_flag);
        else if (warp == WARP_MMA_S)
            mma_s_role<D, F16>(args, smem, bar0, tmem_base, abort_flag);
    } else {
        regs_down<REGS_CONVERT>();
        convert_role<D, F16>(args, smem, bar0, abort_flag);
    }
    __syncwarp();

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == WARP_MMA_S) tmem_dealloc(tmem_base, TMEM_COLS);
    if (*abort_flag && threadIdx.x == 0) {   // copies already issued land before the CTA exits
        const uint32_t* loaded = reinterpret_cast<const uint32_t*>(smem + C::LOADED_OFF);
        for (int s = 0; s < C::K_STAGES + C::C_STAGES; ++s) {
            const int full = s < C::K_STAGES ? C::B_K_FULL + s : C::B_C_FULL + s - C::K_STAGES;
            if (loaded[s] > 0) drain_wait(bar0 + 8 * full, (loaded[s] - 1) & 1, 20000000ull);
        }
    }
}

template <int D, bool F16>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttn8Args& a, cudaStream_t stream) {
    auto kern = attn_paged8_kernel<D, F16>;
    constexpr int smem = Cfg8<D, F16>::SMEM_ALLOC;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kern, dim3(static_cast<unsigned>(a.tile.grid)), NUM_THREADS, smem, stream, tk, tv, a);
}

}  // namespace

cudaError_t launch_attn_paged8(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttn8Args& a, int dtype,
                               cudaStream_t stream) {
    if (a.D == 128) return dtype == 0 ? launch<128, false>(tk, tv, a, stream) : launch<128, true>(tk, tv, a, stream);
    return dtype == 0 ? launch<64, false>(tk, tv, a, stream) : launch<64, true>(tk, tv, a, stream);
}

cudaError_t paged8_error_words(ErrorWords* w) { return error_words_here(w); }

cudaError_t read_and_clear_paged8_error(int* value, DeviceErrorInfo* info, int* drain_failed, unsigned long long* when) {
    return read_and_clear_error_words(value, info, drain_failed, when);
}

}  // namespace xs
