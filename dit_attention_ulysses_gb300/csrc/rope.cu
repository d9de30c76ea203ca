// Rotary positions of Q and K, alone or fused with the append of K and V to a
// paged cache.
//
//   (a, b) -> m (a cos t - b sin t, a sin t + b cos t),   t = position * theta_i
//
// for the i-th pair of the first `rot` channels of every head; pairs are channels
// (i, i + rot/2) (half) or (2i, 2i + 1) (interleaved).  The gradient direction
// applies the transposed map, the rotation by -t.
//
// Angles: theta_i arrives as turns per position in 64-bit fixed point
// (theta / 2 pi * 2^64).  position * turns modulo 2^64 is then the exact fraction
// of a turn, whatever the position, in one integer product; its upper 32 bits,
// taken as signed, are the angle in half turns times 2^31, which sincospif takes
// in [-1, 1) with no range reduction.  A product in fp32 would be off by 0.06
// radians at position 2^20.
//
// What bounds it: the bytes (every element read once and written once).  A thread
// owns two 16-byte chunks of a head (both members of its 8 pairs), computes their
// 8 sines and cosines once and walks the heads with them in registers, four heads
// in flight.  Eight (D = 128) or four (D = 64) threads hold a head, so a load
// instruction of a warp covers 128-byte segments.  75776 x 40 x 128: 230 us, 6.76 TB/s,
// as fast as the card copies; 4608 x 24 x 128: 11.7 us from DRAM (8.3 at that rate, the
// rest is the start and end of one wave); the append of 8192 tokens, 32 + 8 + 8 heads:
// 34 us, 5.85 TB/s; a single small launch: 2.1 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged.h"
#include "ptx.cuh"

namespace xs {
namespace {

constexpr int ROPE_THREADS = 128;
constexpr int ROPE_UNROLL = 4;
constexpr int ROPE_RESIDENT = 5;   // blocks that an SM holds (88 .. 96 registers)

template <bool F16>
__device__ __forceinline__ void widen(uint32_t w, float& lo, float& hi) {
    if constexpr (F16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        lo = f.x;
        hi = f.y;
    } else {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xffff0000u);
    }
}

// Round to nearest even: the one rounding of the operator.
template <bool F16>
__device__ __forceinline__ uint32_t narrow(float lo, float hi) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

struct Chunk2 {
    uint4 a, b;
};

template <bool F16, bool INTERLEAVED>
__device__ __forceinline__ void turn(Chunk2& x, const float (&c)[8], const float (&s)[8], bool rot_a, bool rot_b) {
    uint32_t* wa = reinterpret_cast<uint32_t*>(&x.a);
    uint32_t* wb = reinterpret_cast<uint32_t*>(&x.b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a0, a1, b0, b1;
        widen<F16>(wa[j], a0, a1);
        widen<F16>(wb[j], b0, b1);
        if constexpr (INTERLEAVED) {   // pairs inside each chunk
            const uint32_t ra = narrow<F16>(a0 * c[j] - a1 * s[j], a0 * s[j] + a1 * c[j]);
            const uint32_t rb = narrow<F16>(b0 * c[4 + j] - b1 * s[4 + j], b0 * s[4 + j] + b1 * c[4 + j]);
            if (rot_a) wa[j] = ra;
            if (rot_b) wb[j] = rb;
        } else {                       // pairs across the two chunks
            const float c0 = c[2 * j], c1 = c[2 * j + 1], s0 = s[2 * j], s1 = s[2 * j + 1];
            if (rot_a) {
                wa[j] = narrow<F16>(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
                wb[j] = narrow<F16>(a0 * s0 + b0 * c0, a1 * s1 + b1 * c1);
            }
        }
    }
}

// Block: 128 / units tokens (blockIdx.x) x one group of heads (blockIdx.y).
// Heads are numbered q 0 .. H-1, then (APPEND) k H .. H+Hkv-1, v H+Hkv .. H+2Hkv-1.
template <bool F16, bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(ROPE_THREADS, 1) rope_kernel(const __grid_constant__ RopeArgs g) {
    pdl_launch();
    pdl_wait();
    const int units = g.D >> 4;
    const int tl = threadIdx.x / units, u = threadIdx.x - tl * units;
    const long long t = static_cast<long long>(blockIdx.x) * (ROPE_THREADS / units) + tl;
    if (t >= g.T) return;
    // channel offsets of the thread's two chunks, and whether they rotate
    int oa, ob;
    bool rot_a, rot_b;
    if constexpr (INTERLEAVED) {
        oa = u * 8;
        ob = (g.D >> 1) + u * 8;
        rot_a = oa < g.rot;
        rot_b = ob < g.rot;
    } else {
        const int ru = g.rot >> 4;   // rotating units; the others copy the rest of the head
        const int base = u < ru ? 0 : g.rot, span = u < ru ? g.rot >> 1 : (g.D - g.rot) >> 1;
        oa = base + (u < ru ? u : u - ru) * 8;
        ob = oa + span;
        rot_a = rot_b = u < ru;
    }
    float c[8], s[8];
    if (rot_a || rot_b) {
        const unsigned long long pos = static_cast<unsigned long long>(static_cast<long long>(g.positions[t]));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int pair = INTERLEAVED ? ((j < 4 ? oa : ob) >> 1) + (j & 3) : oa + j;
            const unsigned long long turn64 = pos * g.turns[pair < 64 ? pair : 63];
            const float half_turns = static_cast<float>(static_cast<int>(turn64 >> 32)) * 4.656612873077393e-10f;
            sincospif(half_turns, &s[j], &c[j]);
            c[j] *= g.magnitude;
            s[j] *= g.grad ? -g.magnitude : g.magnitude;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = s[j] = 0.0f;   // not used
    }
    using E = uint16_t;   // both types have 2-byte elements
    long long at = -1, off = 0;
    if constexpr (APPEND) {
        const long long slot = g.slots[t];
        if (slot >= 0 && slot < g.n_slots) {
            at = slot >> g.page_shift;
            off = slot & ((1 << g.page_shift) - 1);
        }
    }
    const int total = APPEND ? g.H + 2 * g.Hkv : g.H;
    const int h0 = blockIdx.y * g.heads_per, h1 = min(total, h0 + g.heads_per);
    auto src = [&](int h) -> const E* {
        if (!APPEND || h < g.H) return static_cast<const E*>(g.q) + t * g.q_stride + static_cast<long long>(h) * g.D;
        h -= g.H;
        if (h < g.Hkv) return static_cast<const E*>(g.k) + t * g.k_stride + static_cast<long long>(h) * g.D;
        return static_cast<const E*>(g.v) + t * g.v_stride + static_cast<long long>(h - g.Hkv) * g.D;
    };
    auto dst = [&](int h) -> E* {
        if (!APPEND || h < g.H) return static_cast<E*>(g.q_out) + t * g.qo_stride + static_cast<long long>(h) * g.D;
        if (at < 0) return nullptr;
        h -= g.H;
        if (h < g.Hkv) return static_cast<E*>(g.k_cache) + at * g.ks[0] + off * g.ks[1] + h * g.ks[2];
        return static_cast<E*>(g.v_cache) + at * g.vs[0] + off * g.vs[1] + (h - g.Hkv) * g.vs[2];
    };
    for (int h = h0; h < h1; h += ROPE_UNROLL) {
        Chunk2 x[ROPE_UNROLL];
#pragma unroll
        for (int i = 0; i < ROPE_UNROLL; ++i)
            if (h + i < h1) {
                const E* p = src(h + i);
                x[i].a = *reinterpret_cast<const uint4*>(p + oa);
                x[i].b = *reinterpret_cast<const uint4*>(p + ob);
            }
#pragma unroll
        for (int i = 0; i < ROPE_UNROLL; ++i)
            if (h + i < h1) {
                if (!APPEND || h + i < g.H + g.Hkv) turn<F16, INTERLEAVED>(x[i], c, s, rot_a, rot_b);
                E* p = dst(h + i);
                if (p != nullptr) {
                    *reinterpret_cast<uint4*>(p + oa) = x[i].a;
                    *reinterpret_cast<uint4*>(p + ob) = x[i].b;
                }
            }
    }
}

}  // namespace

// Heads per thread: as few as four (the loads in flight), at most twelve, and in between the fewest with which all
// blocks run side by side; eight where they do not anyway, twelve again from four rounds on.  Few tokens spread
// their heads further.  Append of 512 / 2048 / 8192 / 32768 tokens, 32 + 8 + 8 heads: 4.8 us (4 heads per thread; 5.4
// with 12), 11.5 (12; 12.3 with 8), 34.4 (8; 36 with 48), 123.4 (12; 125.5 with 8); 64 tokens: 2.7 (2; 3.0 with 4);
// 4608 x 24 x 128: 11.7 (12; 12.4 with 8).  With registers limited to 64, for eight blocks per SM: 6.1, 12.1, 38,
// 131; 3.1; 12.0.
cudaError_t launch_rope(const RopeArgs& args, int dtype, int layout, bool append, int num_sms, cudaStream_t stream) {
    RopeArgs a = args;
    const int units = a.D / 16, tokens = ROPE_THREADS / units;
    const int total = append ? a.H + 2 * a.Hkv : a.H;
    const long long rows = (static_cast<long long>(a.T) + tokens - 1) / tokens;
    auto blocks = [&](int heads) { return rows * ((total + heads - 1) / heads); };
    int heads = 4;
    while (heads < 12 && blocks(heads) > static_cast<long long>(num_sms) * ROPE_RESIDENT) heads += 4;
    if (blocks(heads) > static_cast<long long>(num_sms) * ROPE_RESIDENT)
        heads = blocks(heads) > 4ll * num_sms * ROPE_RESIDENT ? 12 : 8;
    while (heads > 1 && blocks(heads) < num_sms / 2) heads /= 2;
    a.heads_per = heads;
    const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>((total + heads - 1) / heads));
    auto launch = [&](auto kernel) { return launch_overlapped(kernel, grid, ROPE_THREADS, 0, stream, a); };
    switch (dtype * 4 + layout * 2 + (append ? 1 : 0)) {
        case 0: return launch(rope_kernel<false, false, false>);
        case 1: return launch(rope_kernel<false, false, true>);
        case 2: return launch(rope_kernel<false, true, false>);
        case 3: return launch(rope_kernel<false, true, true>);
        case 4: return launch(rope_kernel<true, false, false>);
        case 5: return launch(rope_kernel<true, false, true>);
        case 6: return launch(rope_kernel<true, true, false>);
        default: return launch(rope_kernel<true, true, true>);
    }
}

}  // namespace xs
