// Pieces of the tcgen05 attention kernels that do not depend on where a tile comes from:
// tile sizes, the order of the K/V ring, operand descriptor steps, and a thread's part of
// the softmax of a score block.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace xs {

constexpr int BLOCK_M = 128;
constexpr int BLOCK_N = 128;
constexpr int PANEL_BYTES = BLOCK_M * 128;  // 128 rows x 64 16-bit elements

// Ring position of K(j) / V(j) within a unit of n key blocks (consumption order
// K0, K1, V0, K2, V1, K3, ..., V(n-3), K(n-1), V(n-2), V(n-1)).
static __device__ __forceinline__ uint32_t ring_pos_k(int j) { return j < 2 ? j : 2 * j - 1; }
static __device__ __forceinline__ uint32_t ring_pos_v(int j, int n) { return (j + 2 < n) ? 2 * j + 2 : n + j; }

// Ring item `i` of a unit with n key blocks, in the consumption order
// K0, K1, V0, K2, V1, K3, ..., V(n-3), K(n-1), V(n-2), V(n-1): the block index
// and whether it is a V block.
static __device__ __forceinline__ void ring_item(int i, int n, int& blk, bool& is_v) {
    if (n == 1) {
        blk = 0;
        is_v = (i == 1);
        return;
    }
    if (i < 2) {
        blk = i;
        is_v = false;
        return;
    }
    const int r = i - 2;  // pairs (V_j, K_{j+2}) for j + 2 < n, then V(n-2), V(n-1)
    const int pairs = n - 2;
    if (r < 2 * pairs) {
        is_v = (r & 1) == 0;
        blk = is_v ? (r >> 1) : (r >> 1) + 2;
    } else {
        is_v = true;
        blk = n - 2 + (r - 2 * pairs);
    }
}

// Shared-memory operand descriptors (128-byte swizzle) are built once per role;
// a k-step or a ring stage only moves the start address (desc_add, one 32-bit
// add), which keeps the issuing threads to a few instructions per MMA.
// Q / K operand (K-major): k-step kk covers 16 columns of D, 32 B within the
// 128-B rows of a 64-column panel; panels are PANEL_BYTES apart.
static __device__ __forceinline__ constexpr uint32_t k_step16(int kk) {
    return static_cast<uint32_t>((kk >> 2) * (PANEL_BYTES >> 4) + (kk & 3) * 2);
}
// V operand (MN-major = D contiguous): k-step kk covers 16 keys = two 8-key
// groups of 1024 B (SBO); 64-wide D panels are PANEL_BYTES apart (LBO).
static __device__ __forceinline__ constexpr uint32_t v_step16(int kk) { return static_cast<uint32_t>(kk * (2048 >> 4)); }

// Maximum of a thread's 64 scores: four independent 3-input chains.
static __device__ __forceinline__ float max64(const uint32_t (&sr)[2][32]) {
    float mx[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) mx[r] = __uint_as_float(sr[r >> 1][(r & 1) * 16]);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const int r = q * 2 + (i >> 4);
            mx[r] = fmax3(mx[r], __uint_as_float(sr[q][i]), __uint_as_float(sr[q][i + 1]));
            mx[r] = fmax3(mx[r], __uint_as_float(sr[q][i + 2]), __uint_as_float(sr[q][i + 3]));
        }
    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// p = 2^(s*c - m) for a thread's 64 scores: one packed f32x2 FMA per pair of
// scores and one MUFU ex2 each, packed to bf16 pairs; the fp32 values are summed
// with packed f32x2 adds in two independent chains (half the FP32-pipe
// instructions of scalar FMAs and adds).  The second product takes its operands in
// the type of V: rounding p to it is off by half a step relative to p, which is of
// the size of the output's own rounding.
// TAIL: columns at or past `valid` (keys past the sequence) get p = 0.
// F16: p in fp16 instead of bf16.
template <bool TAIL, bool F16 = false>
static __device__ __forceinline__ float exp64(const uint32_t (&sr)[2][32], float c, float m, int col0, int valid,
                                       uint32_t (&pk)[32]) {
    const float neg_m = -m;
    const uint64_t cc = f2_pack(c, c), mm = f2_pack(neg_m, neg_m);
    uint64_t acc2[2] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f)};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int q = i >> 4;
        const int e = (i & 15) * 2;
        float x0, x1;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[q][e]), __uint_as_float(sr[q][e + 1])), cc, mm), x0, x1);
        float p0 = ex2_approx(x0);
        float p1 = ex2_approx(x1);
        if (TAIL) {
            const int col = col0 + q * 32 + e;
            if (col >= valid) p0 = 0.0f;
            if (col + 1 >= valid) p1 = 0.0f;
        }
        acc2[i & 1] = f2_add(acc2[i & 1], f2_pack(p0, p1));
        pk[i] = F16 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
    }
    float a0, a1, b0, b1;
    f2_unpack(acc2[0], a0, a1);
    f2_unpack(acc2[1], b0, b1);
    return (a0 + a1) + (b0 + b1);
}

}  // namespace xs
