// The 8-bit paged cache: the append that quantises K and V, and elements read back.
//
// An element is an e4m3 number times 2^E, E of its block of tokens and its head.  Per head,
// with a = max |x| over the rows that a block gets and o the tokens that it keeps:
//     e = the least exponent >= -64 with a <= 448 2^e,   E = o > 0 ? max(E, e) : e,
//     kept numbers /= 2^(E - E_before),   new numbers = round(x 2^-E).
//
// Append.  A thread block owns a window of rows and some heads of q, k or v.  D / 16 threads hold a row as in rope.cu, and
// its sines and cosines serve all heads of the block.  Each thread's parts of its row come into
// shared memory by asynchronous copies of its own (256 bytes to a thread at most): bytes in flight cost no
// registers, so that several blocks share an SM, and a thread waits for nobody's copies but its own.  A window of k
// or v is at least as many rows as tokens share a scale, with fewer heads where the threads do not hold them all at once.
// Of k and v a block writes the runs (adjacent rows whose slots follow one another in one block of the cache) that begin in its
// window: their largest magnitudes, their scales, the numbers.  Rows of a run past the window (none in a
// prompt whose windows are blocks) are loaded beside the window's where there is room, else in their place, and
// those again after them.
//
// 8192 tokens (32 heads of 128 over 8, blocks of 16): 38.4 us, 4.8 TB/s of 186 MB (27.4 us at the copy rate).  A block
// runs once through long code, and fetching it holds it up beside its trips to memory (92 % of the fetches hit the SM's
// cache; loops over heads unrolled by two: 40.6 us).  Rows held in registers: 53 us.  64 tokens, one to a sequence: 5.1 us
// where no kept number moves, 10.4 where those of every block do (calls whose magnitudes double each time).  Positions,
// slots, a block's scale and its kept numbers are loaded one after the other, though their addresses depend on the slots
// alone.
#include <cuda_runtime.h>

#include <cstdint>

#include "codes8.cuh"
#include "paged.h"
#include "ptx.cuh"
#include "rope_tile.cuh"

namespace xs {
namespace {

constexpr int MAX_BLOCK = 128;   // tokens of a scale

template <int D, int THREADS>
struct AppendCfg {
    static constexpr int UNITS = D / 16;                      // threads of a row
    static constexpr int ROWS = THREADS / UNITS;              // rows that the threads hold at once
    static constexpr int HEADS = 8;                           // of so many rows, at most
    static constexpr int BYTES = THREADS * HEADS * 32;
    static constexpr int ALL = 2 * (ROWS > MAX_BLOCK ? ROWS : MAX_BLOCK);   // rows of the runs of a window
    static constexpr int SLOT_OFF = BYTES;                    // [ALL] slots
    static constexpr int LARGEST_OFF = SLOT_OFF + ALL * 8;    // [heads][window] largest magnitude of a run, at its first row
    static constexpr int INVERSE_OFF = LARGEST_OFF + ROWS * HEADS * 4;  // [heads][window] 2^-E
    static constexpr int AGAIN_OFF = INVERSE_OFF + ROWS * HEADS * 4;    // runs and heads whose kept numbers move, by how much
    static constexpr int LEAD_OFF = AGAIN_OFF + ROWS * HEADS * 4;       // [ALL] first row of a row's run; -1: not this block's
    static constexpr int MISC_OFF = LEAD_OFF + ALL * 2;
    static constexpr int SMEM = MISC_OFF + 48;
    static_assert(ALL <= 256, "eight warps' rows");
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(__cvta_generic_to_global(src)) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <int D, bool F16, bool INTERLEAVED, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 128 ? 5 : 2)
    append8_kernel(const __grid_constant__ Append8Args g) {
    using C = AppendCfg<D, THREADS>;
    constexpr int UNITS = C::UNITS, ROWS = C::ROWS;
    extern __shared__ __align__(128) uint8_t smem[];
    long long* const s_slot = reinterpret_cast<long long*>(smem + C::SLOT_OFF);
    unsigned* const s_largest = reinterpret_cast<unsigned*>(smem + C::LARGEST_OFF);
    float* const s_inverse = reinterpret_cast<float*>(smem + C::INVERSE_OFF);
    int* const s_again = reinterpret_cast<int*>(smem + C::AGAIN_OFF);
    short* const s_lead = reinterpret_cast<short*>(smem + C::LEAD_OFF);
    int* const s_rows = reinterpret_cast<int*>(smem + C::MISC_OFF);   // rows of the block's runs
    int* const s_n_again = s_rows + 1;
    int* const s_last = s_rows + 2;                                   // [8] last beginning of 32 rows
    using E = uint16_t;
    const int tid = threadIdx.x, lane = tid & 31, u = tid % UNITS, row = tid / UNITS;
    pdl_launch();
    pdl_wait();
    int window, group;   // a window's blocks side by side: what one row of a fused projection holds is read together
    fdivmod(static_cast<int>(blockIdx.x), g.fd_groups, window, group);
    // the block's heads of k, of v or of q (those of one part of the window), and its rows
    const int kind = group < g.kv_groups ? 0 : group < 2 * g.kv_groups ? 1 : 2;
    const int q_at = group - 2 * g.kv_groups, q_part = kind == 2 ? q_at / g.q_groups : 0;
    const int per = kind == 2 ? g.q_per : g.kv_per;
    const int h0 = (kind == 0 ? group : kind == 1 ? group - g.kv_groups : q_at - q_part * g.q_groups) * per;
    const int heads = min(kind == 2 ? g.H : g.Hkv, h0 + per) - h0;
    const int width = kind == 2 ? ROWS : g.window;
    const long long base = static_cast<long long>(window) * g.window + q_part * ROWS;
    if (base >= g.T) return;
    const E* const from = static_cast<const E*>(kind == 0 ? g.k : kind == 1 ? g.v : g.q) + static_cast<long long>(h0) * D;
    const long long stride = kind == 0 ? g.k_stride : kind == 1 ? g.v_stride : g.q_stride;

    int oa, ob;
    bool rot_a, rot_b;
    rope_chunks<INTERLEAVED>(u, D, g.rot, oa, ob, rot_a, rot_b);
    if (kind == 1) rot_a = rot_b = false;
    // the thread's parts of rows first + row, + ROWS .., up to first + n, to its places at, at + 1 ..
    const uint32_t mine = smem_addr(smem) + tid * 16;
    auto load = [&](int first, int n, int at) {
        for (int i = row; i < n; i += ROWS, ++at) {
            const E* p = from + (base + first + i) * stride;
            for (int h = 0; h < heads; ++h, p += D) {
                copy16(mine + (at * heads + h) * (2 * 16 * THREADS), p + oa);
                copy16(mine + (at * heads + h) * (2 * 16 * THREADS) + 16 * THREADS, p + ob);
            }
        }
    };
    auto element = [&](int at, int h) -> Chunk2 {
        const uint8_t* p = smem + tid * 16 + (at * heads + h) * (2 * 16 * THREADS);
        Chunk2 x;
        x.a = *reinterpret_cast<const uint4*>(p);
        x.b = *reinterpret_cast<const uint4*>(p + 16 * THREADS);
        return x;
    };
    const int here = static_cast<int>(min(static_cast<long long>(width), g.T - base));
    load(0, here, 0);
    float c[8] = {}, s[8] = {};
    int turned = -1;
    auto turn_to = [&](int r) {   // the sines and cosines of row r of the window
        const long long t = base + r;
        if (turned != r && (rot_a || rot_b) && t < g.T)
            rope_angles<INTERLEAVED>(g.positions[t], g.turns, oa, ob, g.magnitude, g.magnitude, c, s);
        turned = r;
    };
    turn_to(row);
    if (kind == 2) {
        copies_done();
        if (row >= here) return;
        E* const out = static_cast<E*>(g.q_out) + (base + row) * g.qo_stride + static_cast<long long>(h0) * D;
#pragma unroll 2
        for (int h = 0; h < heads; ++h) {
            Chunk2 x = element(0, h);
            turn<F16, INTERLEAVED>(x, c, s, rot_a, rot_b);
            *reinterpret_cast<uint4*>(out + h * D + oa) = x.a;
            *reinterpret_cast<uint4*>(out + h * D + ob) = x.b;
        }
        return;
    }

    if (tid == 0) *s_rows = *s_n_again = 0;
    for (int i = tid; i < width * heads; i += THREADS) s_largest[i] = 0;

    // ---- runs: a row that does not continue the one before begins one
    const int block = 1 << g.block_shift;
    constexpr int TURNS = C::ALL / THREADS;
    int lead[TURNS];
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int r = tid + i * THREADS, w = r >> 5;
        const long long t = base + r;
        const bool there = r < width + block - 1 && t < g.T;
        const long long slot = there ? g.slots[t] : -1, before = there && t > 0 ? g.slots[t - 1] : -2;
        const bool stored = slot >= 0 && slot < g.n_slots;
        const bool begins = !stored || before + 1 != slot || (slot & (block - 1)) == 0;
        const unsigned flags = __ballot_sync(0xffffffffu, begins), up_to = flags & (0xffffffffu >> (31 - lane));
        if (lane == 0) s_last[w] = flags ? w * 32 + 31 - __clz(flags) : -1;
        s_slot[r] = slot;
        lead[i] = !stored ? -2 : up_to ? w * 32 + 31 - __clz(up_to) : -1;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int r = tid + i * THREADS;
        for (int w = (r >> 5) - 1; w >= 0 && lead[i] == -1; --w) lead[i] = s_last[w];
        if (lead[i] >= width) lead[i] = -1;
        s_lead[r] = static_cast<short>(lead[i] < 0 ? -1 : lead[i]);
        const unsigned ours = __ballot_sync(0xffffffffu, lead[i] >= 0);
        if (lane == 0 && ours) atomicMax(s_rows, r + 32 - __clz(ours));
    }
    __syncthreads();
    const int rows = *s_rows, past = rows - width;   // past: rows past the window
    if (rows == 0) {
        copies_done();
        return;
    }
    // as many turns of the threads each; `place` of the rows past the window
    const int turns = (width + ROWS - 1) / ROWS;
    const bool both = past > 0 && (turns + (past + ROWS - 1) / ROWS) * heads <= C::HEADS;
    const int place = both ? turns : 0;
    copies_done();
    if (both) load(width, past, place);

    // ---- largest magnitudes
    auto largest = [&](int first, int n, int at) {
        for (int i = row; i - row < n; i += ROWS, ++at) {   // (whole warps: shuffles)
            const int r0 = i < n ? s_lead[first + i] : -1;
            if (!__any_sync(0xffffffffu, r0 >= 0)) continue;
            turn_to(first + i);
#pragma unroll 1
            for (int h = 0; h < heads; ++h) {
                float a[8], b[8], m = 0.0f;
                turn_wide<F16, INTERLEAVED>(element(at, h), c, s, rot_a, rot_b, a, b);
#pragma unroll
                for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(a[j]), fabsf(b[j])));
#pragma unroll
                for (int d = UNITS / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                if (u == 0 && r0 >= 0) atomicMax(&s_largest[h * width + r0], __float_as_uint(m));
            }
        }
    };
    largest(0, min(rows, width), 0);
    if (past > 0) {
        if (!both) load(width, past, place);
        copies_done();
        largest(width, past, place);
    }
    __syncthreads();

    // ---- scales of the runs
    const Codes8& to = kind == 0 ? g.kc : g.vc;
    for (int i = tid; i < width * heads; i += THREADS) {
        const int h = i / width, r0 = i - h * width;
        if (s_lead[r0] != r0) continue;
        const long long slot = s_slot[r0];
        const int off = static_cast<int>(slot & ((1 << g.page_shift) - 1));
        uint8_t* const at = to.scale + (slot >> g.page_shift) * to.ss[0] + (off >> g.block_shift) * to.ss[1] + (h0 + h) * to.ss[2];
        const int before = (off & (block - 1)) != 0 ? *at : -1;
        int now = scale_byte(s_largest[i]);
        if (before >= 0 && now > before) s_again[atomicAdd(s_n_again, 1)] = i << 8 | (now - before);
        now = max(now, before);
        if (now != before) *at = static_cast<uint8_t>(now);
        // (a block that keeps a scale of NaN: NaN)
        s_inverse[i] = now == 255 ? any_scale_value(255) : inverse_scale(now);
    }
    __syncthreads();

    // ---- numbers that a block keeps under a larger scale: 16 bytes to a thread at a time, MOVE of them on their way
    // (4: the loop is larger, 8192 tokens in blocks of 32 take 41.7 us instead of 38.3)
    constexpr int MOVE = 2;
    const int each = block * UNITS, all = *s_n_again * each;
    for (int i0 = tid; i0 < all; i0 += MOVE * THREADS) {
        uint4 w[MOVE];
        uint4* at[MOVE];
        float f[MOVE];
#pragma unroll
        for (int m = 0; m < MOVE; ++m) {
            const int i = i0 + m * THREADS, item = i >> (g.block_shift + (D == 128 ? 3 : 2)), k = i & (each - 1);
            at[m] = nullptr;
            if (i >= all) continue;
            const int pair = s_again[item] >> 8, by = s_again[item] & 255, h = pair / width;
            const long long slot = s_slot[pair - h * width];
            const int keep = static_cast<int>(slot & (block - 1)), token = k / UNITS;
            if (token >= keep) continue;
            f[m] = by < 127 ? scale_value(127 - by) : 0.0f;
            at[m] = reinterpret_cast<uint4*>(to.code + (slot >> g.page_shift) * to.cs[0] + (h0 + h) * to.cs[2] +
                                             ((slot & ((1 << g.page_shift) - 1)) - keep + token) * to.cs[1] + k % UNITS * 16);
            w[m] = *at[m];
        }
#pragma unroll
        for (int m = 0; m < MOVE; ++m) {
            if (at[m] == nullptr) continue;
            uint32_t* const ws = reinterpret_cast<uint32_t*>(&w[m]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 lo = f16x2_values(codes_to_f16x2(ws[e])), hi = f16x2_values(codes_to_f16x2_high(ws[e]));
                ws[e] = to_codes(lo.x * f[m], lo.y * f[m], hi.x * f[m], hi.y * f[m]);
            }
            *at[m] = w[m];
        }
    }

    // ---- new numbers, of the rows loaded last first
    auto store = [&](int first, int n, int at) {
        for (int i = row; i < n; i += ROWS, ++at) {
            const int r = first + i, r0 = s_lead[r];
            if (r0 < 0) continue;
            turn_to(r);
            const long long slot = s_slot[r];
            uint8_t* const p = to.code + (slot >> g.page_shift) * to.cs[0] + (slot & ((1 << g.page_shift) - 1)) * to.cs[1];
#pragma unroll 1
            for (int h = 0; h < heads; ++h) {
                float a[8], b[8];
                turn_wide<F16, INTERLEAVED>(element(at, h), c, s, rot_a, rot_b, a, b);
                const float f = s_inverse[h * width + r0];
                uint8_t* const q = p + (h0 + h) * to.cs[2];
                *reinterpret_cast<uint2*>(q + oa) = make_uint2(to_codes(a[0] * f, a[1] * f, a[2] * f, a[3] * f),
                                                               to_codes(a[4] * f, a[5] * f, a[6] * f, a[7] * f));
                *reinterpret_cast<uint2*>(q + ob) = make_uint2(to_codes(b[0] * f, b[1] * f, b[2] * f, b[3] * f),
                                                               to_codes(b[4] * f, b[5] * f, b[6] * f, b[7] * f));
            }
        }
    };
    if (past > 0) {
        store(width, past, place);
        if (!both) {
            load(0, width, 0);
            copies_done();
        }
    }
    store(0, min(rows, width), 0);
}

// ------------------------------------------------------------------- read back
// A thread block gathers ROWS rows, 8 or 16: their sequences, pages and offsets once, into
// shared memory, then 16-channel pieces of K and V.  Bound by HBM: 32768 rows of 8 x 128 take 35.4 us,
// 5.7 TB/s of 201 MB (29.6 us at the copy rate), with 8 rows to a block 36.2, with 32 38.2.  1000 sequences of 8
// rows take 12.1 us with 8 rows to a block (each waits for a search, a page, then the rows), 16.1 with 16 and 19.6
// with 32; 24 ragged ones of up to 500 rows of 6 x 64 4.5, 5.6 and 5.5.
constexpr int THREADS = 256;
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

// x, or the nearer end of [-most, most]; NaN stays NaN (fminf and fmaxf would give an end).
__device__ __forceinline__ float saturated(float x, float most) {
    float y;
    asm("{\n.reg .f32 t;\nmax.NaN.f32 t, %1, %2;\nmin.NaN.f32 %0, t, %3;\n}" : "=f"(y) : "f"(x), "f"(-most), "f"(most));
    return y;
}

template <bool F16>
__device__ __forceinline__ uint32_t value_pair(uint32_t f16x2, float scale) {
    const float2 f = f16x2_values(f16x2);
    const float most = F16 ? 65504.0f : 3.3895313892515355e38f;
    return narrow<F16>(saturated(f.x * scale, most), saturated(f.y * scale, most));
}

template <bool F16, int ROWS>
__global__ void __launch_bounds__(THREADS) read8_kernel(const __grid_constant__ Read8Args g) {
    __shared__ int s_page[ROWS];   // -1: zeros
    __shared__ int s_off[ROWS];
    pdl_launch();
    pdl_wait();
    const int base = blockIdx.x * ROWS, tid = threadIdx.x;
    const int total = g.cu[g.n];
    const int rows = min(min(g.T, total) - base, ROWS);
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
            const float f = any_scale_value(scale[j]);
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

namespace {

template <int D, int THREADS>
cudaError_t launch_append(const Append8Args& args, int dtype, int layout, int num_sms, cudaStream_t stream) {
    using C = AppendCfg<D, THREADS>;
    Append8Args a = args;
    const int parts = (1 << a.block_shift) > C::ROWS ? (1 << a.block_shift) / C::ROWS : 1;
    a.window = C::ROWS * parts;
    const long long windows = (static_cast<long long>(a.T) + a.window - 1) / a.window;
    // heads of a block: as many as fit, fewer where that leaves SMs without a block.  512 tokens (32 heads of 128 over 8):
    // 6.1 us, 7.0 if halved from half as many blocks on, 6.9 from twice as many, 8.1 if never; 7200 tokens at most, ragged
    // (12 of 64 over 6, blocks of 64): 7.9, 9.7, 10.1, 13.0; 256 tokens: 5.5, 5.7, 5.2, 7.0; 2048: 14.2, 14.1, 12.8, 14.1
    auto groups = [](int heads, int per) { return (heads + per - 1) / per; };
    auto per_block = [&](long long count, int heads, int most) {
        while (most > 1 && count * groups(heads, most) < num_sms) most /= 2;
        return most;
    };
    a.kv_per = per_block(2 * windows, a.Hkv, C::HEADS / parts);
    a.q_per = per_block(windows * parts, a.H, C::HEADS);
    a.kv_groups = groups(a.Hkv, a.kv_per);
    a.q_groups = groups(a.H, a.q_per);
    const int blocks = 2 * a.kv_groups + parts * a.q_groups;   // of a window
    if (windows * blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    a.fd_groups = make_fastdiv(blocks);
    auto launch = [&](auto kernel) {
        if (C::SMEM > 48 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
            if (e != cudaSuccess) return e;
        }
        return launch_overlapped(kernel, dim3(static_cast<unsigned>(windows * blocks)), THREADS, C::SMEM, stream, a);
    };
    switch (dtype * 2 + layout) {
        case 0: return launch(append8_kernel<D, false, false, THREADS>);
        case 1: return launch(append8_kernel<D, false, true, THREADS>);
        case 2: return launch(append8_kernel<D, true, false, THREADS>);
        default: return launch(append8_kernel<D, true, true, THREADS>);
    }
}

}  // namespace

cudaError_t launch_append8(const Append8Args& a, int dtype, int layout, int num_sms, cudaStream_t stream) {
    // 128 threads where they hold a block's rows (blocks of 16, D = 128: 256 tokens 5.5 us, 512 6.1, 8192 38.4; with 256
    // threads 6.3, 7.5, 42.1), else 256 (blocks of 128: 512 tokens 19.5 us, 8192 48.6, with 128 threads 30.5 and 55.2; blocks
    // of 32: 8.6 and 9.8, but 8192 42.1 and 39.2, heads first 38.4 and 39.4; the ragged batch above 7.9 and 11.4)
    const bool few = ((a.D / 16) << a.block_shift) <= 128;
    if (a.D == 64)
        return few ? launch_append<64, 128>(a, dtype, layout, num_sms, stream) : launch_append<64, 256>(a, dtype, layout, num_sms, stream);
    return few ? launch_append<128, 128>(a, dtype, layout, num_sms, stream) : launch_append<128, 256>(a, dtype, layout, num_sms, stream);
}

cudaError_t launch_read8(const Read8Args& args, int dtype, int num_sms, cudaStream_t stream) {
    Read8Args a = args;
    a.fd_row = make_fastdiv(a.Hkv * a.D / 16);
    auto launch = [&](auto kernel, int rows) {
        return launch_overlapped(kernel, dim3(static_cast<unsigned>((a.T - 1) / rows + 1)), THREADS, 0, stream, a);
    };
    // 8 rows to a block where all blocks are then on the SMs at once, eight to one (8000 rows of 8 x 128: 10.6 us, with 16
    // rows to a block 14.4; 12000 rows 17.0 and 17.3)
    if ((a.T - 1) / 8 < 8 * num_sms) return dtype == 0 ? launch(read8_kernel<false, 8>, 8) : launch(read8_kernel<true, 8>, 8);
    return dtype == 0 ? launch(read8_kernel<false, 16>, 16) : launch(read8_kernel<true, 16>, 16);
}

}  // namespace xs
