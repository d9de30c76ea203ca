// The 8-bit paged cache: the append that quantises K and V, and elements read back.
//
// An element is an e4m3 number times 2^E, E of its block of tokens and its head.  Per head,
// with a = max |x| over the rows that a block gets and o the tokens that it keeps:
//     e = the least exponent >= -64 with a <= 448 2^e,   E = o > 0 ? max(E, e) : e,
//     kept numbers /= 2^(E - E_before),   new numbers = round(x 2^-E).
//
// Append.  A thread block owns a window of rows: the runs (adjacent rows whose slots follow one
// another in one block) that begin there, which end at most block - 1 rows past it.  It takes two passes over
// them, the maximum and the numbers, with the largest magnitudes of its runs and heads in
// shared memory between; the second pass reads k and v from L2 and turns them again, which
// costs less than holding up to 255 rows in registers would in occupancy.  Other blocks of the
// launch turn q.  Threads hold two 16-byte chunks of a row as in rope.cu.
#include <cuda_runtime.h>

#include <cstdint>

#include "codes8.cuh"
#include "paged.h"
#include "ptx.cuh"
#include "rope_tile.cuh"

namespace xs {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_WINDOW = 128;   // rows of a window; with the rows past it at most THREADS
constexpr int MAX_KV_PER = 4;
constexpr int UNROLL = 4;

template <bool F16, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) append8_kernel(const __grid_constant__ Append8Args g) {
    __shared__ long long s_slot[THREADS];
    __shared__ short s_lead[THREADS];                          // first row of a row's run; -1: not this block's
    __shared__ int s_last[WARPS];
    __shared__ uint32_t s_largest[MAX_WINDOW * MAX_KV_PER];    // per run (at its first row) and head
    __shared__ float s_inverse[MAX_WINDOW * MAX_KV_PER];       // 2^-E
    __shared__ int s_again[MAX_WINDOW * MAX_KV_PER];           // runs and heads whose kept numbers move
    __shared__ int s_n_again;
    using E = uint16_t;
    pdl_launch();
    pdl_wait();
    const int tid = threadIdx.x, units = g.D >> 4;
    const int tl = tid / units, u = tid - tl * units, rows_at_once = THREADS / units;
    const long long base = static_cast<long long>(blockIdx.x) * g.window;
    int oa, ob;
    bool rot_a, rot_b;
    rope_chunks<INTERLEAVED>(u, g.D, g.rot, oa, ob, rot_a, rot_b);
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = s[j] = 0.0f;

    if (static_cast<int>(blockIdx.y) >= g.kv_groups) {   // q
        const int h0 = (blockIdx.y - g.kv_groups) * g.q_per, h1 = min(g.H, h0 + g.q_per);
        for (int r = tl; r < g.window; r += rows_at_once) {
            const long long t = base + r;
            if (t >= g.T) break;
            if (rot_a || rot_b)
                rope_angles<INTERLEAVED>(g.positions[t], g.turns, oa, ob, g.magnitude, g.magnitude, c, s);
            const E* src = static_cast<const E*>(g.q) + t * g.q_stride;
            E* dst = static_cast<E*>(g.q_out) + t * g.qo_stride;
            for (int h = h0; h < h1; h += UNROLL) {
                Chunk2 x[UNROLL];
#pragma unroll
                for (int i = 0; i < UNROLL; ++i)
                    if (h + i < h1) {
                        x[i].a = *reinterpret_cast<const uint4*>(src + static_cast<long long>(h + i) * g.D + oa);
                        x[i].b = *reinterpret_cast<const uint4*>(src + static_cast<long long>(h + i) * g.D + ob);
                    }
#pragma unroll
                for (int i = 0; i < UNROLL; ++i)
                    if (h + i < h1) {
                        turn<F16, INTERLEAVED>(x[i], c, s, rot_a, rot_b);
                        *reinterpret_cast<uint4*>(dst + static_cast<long long>(h + i) * g.D + oa) = x[i].a;
                        *reinterpret_cast<uint4*>(dst + static_cast<long long>(h + i) * g.D + ob) = x[i].b;
                    }
            }
        }
        return;
    }

    // ---- runs
    const int block = 1 << g.block_shift, rows = g.window + block - 1;
    const int h0 = blockIdx.y * g.kv_per, heads = min(2 * g.Hkv, h0 + g.kv_per) - h0;   // K 0 .. Hkv - 1, then V
    {
        const long long t = base + tid;
        const bool here = tid < rows && t < g.T;
        const long long slot = here ? g.slots[t] : -1, before = here && t > 0 ? g.slots[t - 1] : -2;
        const bool stored = slot >= 0 && slot < g.n_slots;
        const bool begins = !stored || before + 1 != slot || (slot & (block - 1)) == 0;
        const unsigned flags = __ballot_sync(0xffffffffu, begins);
        const unsigned mine = flags & (0xffffffffu >> (31 - (tid & 31)));
        if ((tid & 31) == 0) {
            s_last[tid >> 5] = flags ? (tid & ~31) + 31 - __clz(flags) : -1;
            if (tid == 0) s_n_again = 0;
        }
        for (int i = tid; i < g.window * heads; i += THREADS) s_largest[i] = 0;
        __syncthreads();
        int lead = mine ? (tid & ~31) + 31 - __clz(mine) : -1;
        for (int w = (tid >> 5) - 1; w >= 0 && lead < 0; --w) lead = s_last[w];
        s_slot[tid] = slot;
        s_lead[tid] = static_cast<short>(stored && lead < g.window ? lead : -1);
    }
    __syncthreads();
    auto scale_at = [&](int row, int hh) -> uint8_t* {
        const long long slot = s_slot[row];
        const int h = h0 + hh, off = static_cast<int>(slot & ((1 << g.page_shift) - 1));
        const Codes8& x = h < g.Hkv ? g.kc : g.vc;
        return x.scale + (slot >> g.page_shift) * x.ss[0] + (off >> g.block_shift) * x.ss[1] +
               (h < g.Hkv ? h : h - g.Hkv) * x.ss[2];
    };
    auto source = [&](long long t, int hh) -> const E* {
        const int h = h0 + hh;
        if (h < g.Hkv) return static_cast<const E*>(g.k) + t * g.k_stride + static_cast<long long>(h) * g.D;
        return static_cast<const E*>(g.v) + t * g.v_stride + static_cast<long long>(h - g.Hkv) * g.D;
    };
    // scales of the blocks that keep tokens
    constexpr int PAIRS = MAX_WINDOW * MAX_KV_PER / THREADS;
    int kept_scale[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        const int pair = tid + i * THREADS, row = pair / heads;
        kept_scale[i] = -1;
        if (pair < g.window * heads && s_lead[row] == row && (s_slot[row] & (block - 1)) != 0)
            kept_scale[i] = *scale_at(row, pair - row * heads);
    }

    // ---- largest magnitudes
    const bool turns = h0 < g.Hkv && (rot_a || rot_b);
    for (int r = tl; r - tl < rows; r += rows_at_once) {   // (every lane takes part in the shuffles)
        const int lead = r < rows ? s_lead[r] : -1;
        if (!__any_sync(0xffffffffu, lead >= 0)) continue;
        const long long t = base + r;
        if (turns && lead >= 0) rope_angles<INTERLEAVED>(g.positions[t], g.turns, oa, ob, g.magnitude, g.magnitude, c, s);
        Chunk2 x[MAX_KV_PER];
#pragma unroll
        for (int i = 0; i < MAX_KV_PER; ++i) {
            x[i].a = x[i].b = make_uint4(0, 0, 0, 0);
            if (i < heads && lead >= 0) {
                const E* p = source(t, i);
                x[i].a = *reinterpret_cast<const uint4*>(p + oa);
                x[i].b = *reinterpret_cast<const uint4*>(p + ob);
            }
        }
#pragma unroll
        for (int i = 0; i < MAX_KV_PER; ++i) {
            if (i >= heads) break;
            float a[8], b[8], m = 0.0f;
            const bool k = h0 + i < g.Hkv;
            turn_wide<F16, INTERLEAVED>(x[i], c, s, k && rot_a, k && rot_b, a, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(a[j]), fabsf(b[j])));
            for (int d = units >> 1; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            if (u == 0 && lead >= 0) atomicMax(&s_largest[lead * heads + i], __float_as_uint(m));
        }
    }
    __syncthreads();

    // ---- scales
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        const int pair = tid + i * THREADS, row = pair / heads;
        if (pair >= g.window * heads || s_lead[row] != row) continue;
        const int before = kept_scale[i];
        int now = scale_byte(s_largest[pair]);
        if (before >= 0 && now > before) s_again[atomicAdd(&s_n_again, 1)] = (pair << 8) | (now - before);
        now = max(now, before);
        if (now != before) *scale_at(row, pair - row * heads) = static_cast<uint8_t>(now);
        s_inverse[pair] = scale_value(254 - now);
    }
    __syncthreads();

    // ---- numbers that a block keeps under a larger scale
    for (int i = tid >> 5; i < s_n_again; i += WARPS) {
        const int pair = s_again[i] >> 8, by = s_again[i] & 255, row = pair / heads, h = h0 + pair - row * heads;
        const float f = by < 127 ? scale_value(127 - by) : 0.0f;
        const long long slot = s_slot[row];
        const int keep = static_cast<int>(slot & (block - 1));
        const Codes8& x = h < g.Hkv ? g.kc : g.vc;
        uint8_t* p = x.code + (slot >> g.page_shift) * x.cs[0] + (h < g.Hkv ? h : h - g.Hkv) * x.cs[2];
        const long long token0 = (slot & ((1 << g.page_shift) - 1)) - keep;
        for (int j = tid & 31; j < keep * units; j += 32) {
            const int token = j / units;
            uint4* at = reinterpret_cast<uint4*>(p + (token0 + token) * x.cs[1] + (j - token * units) * 16);
            uint4 w = *at;
            uint32_t* const ws = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 lo = f16x2_values(codes_to_f16x2(ws[e])), hi = f16x2_values(codes_to_f16x2_high(ws[e]));
                ws[e] = to_codes(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
            }
            *at = w;
        }
    }

    // ---- new numbers
    for (int r = tl; r < rows; r += rows_at_once) {
        const int lead = s_lead[r];
        if (lead < 0) continue;
        const long long t = base + r, slot = s_slot[r];
        const long long page = slot >> g.page_shift, off = slot & ((1 << g.page_shift) - 1);
        if (turns) rope_angles<INTERLEAVED>(g.positions[t], g.turns, oa, ob, g.magnitude, g.magnitude, c, s);
        Chunk2 x[MAX_KV_PER];
#pragma unroll
        for (int i = 0; i < MAX_KV_PER; ++i)
            if (i < heads) {
                const E* p = source(t, i);
                x[i].a = *reinterpret_cast<const uint4*>(p + oa);
                x[i].b = *reinterpret_cast<const uint4*>(p + ob);
            }
#pragma unroll
        for (int i = 0; i < MAX_KV_PER; ++i) {
            if (i >= heads) break;
            float a[8], b[8];
            const int h = h0 + i;
            const bool k = h < g.Hkv;
            turn_wide<F16, INTERLEAVED>(x[i], c, s, k && rot_a, k && rot_b, a, b);
            const float f = s_inverse[lead * heads + i];
            const Codes8& z = k ? g.kc : g.vc;
            uint8_t* p = z.code + page * z.cs[0] + off * z.cs[1] + (k ? h : h - g.Hkv) * z.cs[2];
            uint2 wa, wb;
            wa.x = to_codes(a[0] * f, a[1] * f, a[2] * f, a[3] * f);
            wa.y = to_codes(a[4] * f, a[5] * f, a[6] * f, a[7] * f);
            wb.x = to_codes(b[0] * f, b[1] * f, b[2] * f, b[3] * f);
            wb.y = to_codes(b[4] * f, b[5] * f, b[6] * f, b[7] * f);
            *reinterpret_cast<uint2*>(p + oa) = wa;
            *reinterpret_cast<uint2*>(p + ob) = wb;
        }
    }
}

// ------------------------------------------------------------------- read back
// A thread block gathers READ_ROWS rows: their sequences, pages and offsets once, into shared
// memory, then 16-channel pieces of K and V.
constexpr int READ_ROWS = 32;
constexpr int READ_UNROLL = 4;

// The last sequence i of [0, n) with cu[i] <= r (empty ones behind it excluded), by a warp: 32 places at once.
__device__ __forceinline__ int find_sequence(const int* cu, int n, int r) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;   // cu[lo] <= r, the answer in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const bool below = at < hi && (lane == 0 || cu[at] <= r);
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, below));
        lo += last * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

template <bool F16>
__device__ __forceinline__ uint32_t value_pair(uint32_t f16x2, float scale) {
    const float2 f = f16x2_values(f16x2);
    const float most = F16 ? 65504.0f : 3.3895313892515355e38f;
    return narrow<F16>(fminf(fmaxf(f.x * scale, -most), most), fminf(fmaxf(f.y * scale, -most), most));
}

template <bool F16>
__global__ void __launch_bounds__(THREADS) read8_kernel(const __grid_constant__ Read8Args g) {
    __shared__ int s_page[READ_ROWS];   // -1: zeros
    __shared__ int s_off[READ_ROWS];
    pdl_launch();
    pdl_wait();
    const int base = blockIdx.x * READ_ROWS, tid = threadIdx.x;
    const int total = g.cu[g.n];
    const int rows = min(min(g.T, total) - base, READ_ROWS);
    if (rows <= 0) return;
    if (tid < 32) {
        int i = find_sequence(g.cu, g.n, base);
        const int r = base + tid;
        if (tid < rows) {
            // the sequences of the rows behind the first: the next ones, of any length
            if (i + 1 < g.n && g.cu[i + 1] <= r) {
                int hi = g.n;
                while (hi - i > 1) {
                    const int mid = i + (hi - i) / 2;
                    if (g.cu[mid] <= r) i = mid;
                    else hi = mid;
                }
            }
            const long long p = static_cast<long long>(g.first ? g.first[i] : 0) + r - g.cu[i];
            const long long col = p >> g.page_shift;
            const int page = p >= 0 && col < g.width ? g.table[i * g.table_stride + col] : -1;
            s_page[tid] = page >= 0 && page < g.n_pages ? page : -1;
            s_off[tid] = static_cast<int>(p & ((1 << g.page_shift) - 1));
        }
    }
    __syncthreads();
    const int pieces = g.fd_row.d, shift = g.D == 128 ? 3 : 2;   // of a row; a head has 1 << shift
    for (int i0 = tid; i0 < 2 * rows * pieces; i0 += READ_UNROLL * THREADS) {
        uint4 w[READ_UNROLL];
        uint32_t scale[READ_UNROLL];
        int row[READ_UNROLL], piece[READ_UNROLL];
#pragma unroll
        for (int j = 0; j < READ_UNROLL; ++j) {
            const int i = i0 + j * THREADS;
            w[j] = make_uint4(0, 0, 0, 0);
            scale[j] = 0;
            row[j] = -1;
            if (i >= 2 * rows * pieces) continue;
            fdivmod(i, g.fd_row, row[j], piece[j]);   // K rows, then V rows
            const bool k = row[j] < rows;
            const int r = k ? row[j] : row[j] - rows, page = s_page[r], off = s_off[r];
            if (page < 0) continue;
            const Codes8& x = k ? g.kc : g.vc;
            const int h = piece[j] >> shift, part = piece[j] & ((1 << shift) - 1);
            w[j] = *reinterpret_cast<const uint4*>(x.code + page * x.cs[0] + off * x.cs[1] + h * x.cs[2] + part * 16);
            scale[j] = x.scale[page * x.ss[0] + (off >> g.block_shift) * x.ss[1] + h * x.ss[2]];
        }
#pragma unroll
        for (int j = 0; j < READ_UNROLL; ++j) {
            if (row[j] < 0) continue;
            const bool k = row[j] < rows;
            const int r = k ? row[j] : row[j] - rows;
            const float f = scale_value(scale[j]);
            const uint32_t ws[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[2 * e] = value_pair<F16>(codes_to_f16x2(ws[e]), f);
                o[2 * e + 1] = value_pair<F16>(codes_to_f16x2_high(ws[e]), f);
            }
            uint16_t* p = static_cast<uint16_t*>(k ? g.k_out : g.v_out) + (base + r) * (k ? g.k_stride : g.v_stride) +
                          piece[j] * 16;
            st_global_v4(p, o[0], o[1], o[2], o[3]);
            st_global_v4(p + 8, o[4], o[5], o[6], o[7]);
        }
    }
}

}  // namespace

cudaError_t launch_append8(const Append8Args& args, int dtype, int layout, int num_sms, cudaStream_t stream) {
    Append8Args a = args;
    const int block = 1 << a.block_shift, at_once = THREADS * 16 / a.D;
    a.window = block > at_once ? block : at_once;
    const long long windows = (static_cast<long long>(a.T) + a.window - 1) / a.window;
    auto groups = [](int heads, int per) { return (heads + per - 1) / per; };
    a.kv_per = MAX_KV_PER;
    while (a.kv_per > 1 && windows * groups(2 * a.Hkv, a.kv_per) < num_sms) a.kv_per /= 2;
    a.q_per = 8;
    while (a.q_per > 1 && windows * groups(a.H, a.q_per) < 2 * num_sms) a.q_per /= 2;
    a.kv_groups = groups(2 * a.Hkv, a.kv_per);
    const dim3 grid(static_cast<unsigned>(windows), static_cast<unsigned>(a.kv_groups + groups(a.H, a.q_per)));
    auto launch = [&](auto kernel) { return launch_overlapped(kernel, grid, THREADS, 0, stream, a); };
    switch (dtype * 2 + layout) {
        case 0: return launch(append8_kernel<false, false>);
        case 1: return launch(append8_kernel<false, true>);
        case 2: return launch(append8_kernel<true, false>);
        default: return launch(append8_kernel<true, true>);
    }
}

cudaError_t launch_read8(const Read8Args& args, int dtype, int num_sms, cudaStream_t stream) {
    Read8Args a = args;
    a.fd_row = make_fastdiv(a.Hkv * a.D / 16);
    const dim3 grid(static_cast<unsigned>((a.T + READ_ROWS - 1) / READ_ROWS));
    return dtype == 0 ? launch_overlapped(read8_kernel<false>, grid, THREADS, 0, stream, a)
                      : launch_overlapped(read8_kernel<true>, grid, THREADS, 0, stream, a);
}

}  // namespace xs
