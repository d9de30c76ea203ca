// Pieces of the mma.sync attention of a few tokens over a paged cache that do not depend on the
// cache's type: fragments, waits on a warp's ring of copies, and finished rows.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "device_wait.cuh"
#include "kernels.h"
#include "paged.h"
#include "ptx.cuh"

namespace xs {
namespace {

constexpr float NO_MAX = -3.402823466e38f;           // running maximum of a row that has seen nothing
constexpr float RESCALE_THRESHOLD = 8.0f;  // log2 units; P stays below 2^8

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(addr)
                 : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return F16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

// warp_wait, except that a limit of 0 gives up at the first test that finds the copy not
// landed: the wait's own first probe may be suspended until it has.
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t timeout_ns,
                                          int unit, int blk) {
    if (timeout_ns == 0 && !__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) {
        *abort_flag = 1;
        report_error(XS_DEVICE_TIMEOUT_CODE, static_cast<int>(bar), static_cast<int>(parity), unit, blk);
        return false;
    }
    return warp_wait(bar, parity, abort_flag, timeout_ns, unit, blk);
}

// Destination of output row (token, head) in the call's layout.
__device__ __forceinline__ uint16_t* out_row(const PagedAttnArgs& a, int token, int head) {
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

// Four channels and, once per row, the log-sum-exp of a finished row.
template <bool F16>
__device__ __forceinline__ void store_out(const PagedAttnArgs& a, int token, int head, int c4, float4 o, float m,
                                          float l) {
    uint16_t* p = out_row(a, token, head);
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;   // a row that saw no key: 0
    if (p != nullptr) {
        uint2 w;
        w.x = pack2<F16>(o.x * inv, o.y * inv);
        w.y = pack2<F16>(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2*>(p + c4 * 4) = w;
    }
    // (-infinity if the row saw no key, NaN if its sum is)
    if (c4 == 0 && a.lse != nullptr)
        a.lse[static_cast<size_t>(token) * a.H + head] =
            l == 0.0f ? __int_as_float(0xff800000) : (m + log2f(l)) * 0.6931471805599453f;
}

// The parts of CTAs c0 .. c1 of a cut tile, joined in CTA order and stored; by a whole CTA.  A tile of HP KV heads
// holds n_rows rows of each, row 8 h + r of its parts row r of head h.
constexpr int JOIN_BATCH = 16;             // parts read at once
template <int D, int ROWS, int THREADS, int HP, bool F16>
__device__ __forceinline__ void join_parts(const PagedAttnArgs& a, int row0, int kv_head, int n_rows, int c0, int c1) {
    for (int i = threadIdx.x; i < n_rows * HP * (D / 4); i += THREADS) {
        const int hp = i / (D / 4) % HP, r = i / (D / 4) / HP + 8 * hp, c4 = i % (D / 4);
        float m = NO_MAX, l = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        // a batch at a time in flight (past the last: the last once more, at weight 0)
        for (int cb = c0; cb <= c1; cb += JOIN_BATCH) {
            float2 ml[JOIN_BATCH];
            float4 v[JOIN_BATCH];
#pragma unroll
            for (int j = 0; j < JOIN_BATCH; ++j) {
                const int c = min(cb + j, c1);
                const size_t at = (2 * static_cast<size_t>(c) + (c == c0 ? 1 : 0)) * ROWS + r;
                ml[j] = __ldcg(a.work.part_ml + at);
                v[j] = __ldcg(reinterpret_cast<const float4*>(a.work.part_o + at * D + c4 * 4));
                if (cb + j > c1) ml[j] = make_float2(NO_MAX, 0.0f);
            }
            float m_new = m;
#pragma unroll
            for (int j = 0; j < JOIN_BATCH; ++j) m_new = fmaxf(m_new, ml[j].x);
            const float f0 = ex2_approx(m - m_new);
            m = m_new;
            l *= f0;
            acc.x *= f0;
            acc.y *= f0;
            acc.z *= f0;
            acc.w *= f0;
#pragma unroll
            for (int j = 0; j < JOIN_BATCH; ++j) {
                const float f = cb + j > c1 ? 0.0f : ex2_approx(ml[j].x - m);
                l += ml[j].y * f;
                acc.x += v[j].x * f;
                acc.y += v[j].y * f;
                acc.z += v[j].z * f;
                acc.w += v[j].w * f;
            }
        }
        int t, gh;
        fdivmod(r - 8 * hp, a.fd_G, t, gh);
        const int token = row0 + t;
        if (token < a.T) store_out<F16>(a, token, (kv_head * HP + hp) * a.G + gh, c4, acc, m, l);
    }
}

}  // namespace
}  // namespace xs
