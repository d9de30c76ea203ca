// A thread's part of the rotary kernels: two 16-byte chunks of a head that hold both members
// of their 8 pairs, the pairs' sines and cosines, and the rotation.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace xs {

// Channel offsets of the two chunks of thread u of the D / 16 of a head, and whether they rotate.
template <bool INTERLEAVED>
__device__ __forceinline__ void rope_chunks(int u, int D, int rot, int& oa, int& ob, bool& rot_a, bool& rot_b) {
    if constexpr (INTERLEAVED) {
        oa = u * 8;
        ob = (D >> 1) + u * 8;
        rot_a = oa < rot;
        rot_b = ob < rot;
    } else {
        const int ru = rot >> 4;   // rotating units; the others copy the rest of the head
        const int base = u < ru ? 0 : rot, span = u < ru ? rot >> 1 : (D - rot) >> 1;
        oa = base + (u < ru ? u : u - ru) * 8;
        ob = oa + span;
        rot_a = rot_b = u < ru;
    }
}

// Cosines (times cos_by) and sines (times sin_by) of the chunks' pairs at a position.
template <bool INTERLEAVED>
__device__ __forceinline__ void rope_angles(int position, const unsigned long long (&turns)[64], int oa, int ob, float cos_by,
                                            float sin_by, float (&c)[8], float (&s)[8]) {
    const unsigned long long pos = static_cast<unsigned long long>(static_cast<long long>(position));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int pair = INTERLEAVED ? ((i < 4 ? oa : ob) >> 1) + (i & 3) : oa + i;
        const unsigned long long turn64 = pos * turns[pair < 64 ? pair : 63];
        const float half_turns = static_cast<float>(static_cast<int>(turn64 >> 32)) * 4.656612873077393e-10f;
        sincospif(half_turns, &s[i], &c[i]);
        c[i] *= cos_by;
        s[i] *= sin_by;
    }
}

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

// The same in fp32: channels oa .. oa + 7 and ob .. ob + 7.
template <bool F16, bool INTERLEAVED>
__device__ __forceinline__ void turn_wide(const Chunk2& x, const float (&c)[8], const float (&s)[8], bool rot_a, bool rot_b,
                                          float (&a)[8], float (&b)[8]) {
    const uint32_t wa[4] = {x.a.x, x.a.y, x.a.z, x.a.w}, wb[4] = {x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        widen<F16>(wa[j], a[2 * j], a[2 * j + 1]);
        widen<F16>(wb[j], b[2 * j], b[2 * j + 1]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = 2 * j;
        const float a0 = a[i], a1 = a[i + 1], b0 = b[i], b1 = b[i + 1];
        if constexpr (INTERLEAVED) {
            if (rot_a) {
                a[i] = a0 * c[j] - a1 * s[j];
                a[i + 1] = a0 * s[j] + a1 * c[j];
            }
            if (rot_b) {
                b[i] = b0 * c[4 + j] - b1 * s[4 + j];
                b[i + 1] = b0 * s[4 + j] + b1 * c[4 + j];
            }
        } else if (rot_a) {
            a[i] = a0 * c[i] - b0 * s[i];
            a[i + 1] = a1 * c[i + 1] - b1 * s[i + 1];
            b[i] = a0 * s[i] + b0 * c[i];
            b[i + 1] = a1 * s[i + 1] + b1 * c[i + 1];
        }
    }
}

}  // namespace xs
