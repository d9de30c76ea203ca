// Internal interface of the paged-cache entry points (api_paged.cu) to their kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"

namespace xs {

// Launch whose prologue may overlap the end of the kernel before it on the stream; every
// thread of the kernel calls pdl_wait (ptx.cuh) before it touches global memory.
template <typename... Params, typename... Args>
inline cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                     const Args&... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// ---- rotary positions, and their fusion with the cache append (rope.cu)
struct RopeArgs {
    const void* q;            // [T, H, D], rows q_stride elements apart
    const void* k;            // append: [T, Hkv, D]
    const void* v;            // append: [T, Hkv, D]
    void* q_out;              // [T, H, D]
    void* k_cache;            // append: [n_pages, page, Hkv, D], strides ks
    void* v_cache;
    const int* positions;     // [T]
    const long long* slots;   // append: [T], page * page_size + offset; outside the cache: not stored
    long long q_stride, k_stride, v_stride, qo_stride;   // elements between rows
    long long ks[3], vs[3];                              // elements between pages, tokens of a page, heads
    long long n_slots;        // n_pages * page_size
    int T, H, Hkv, D, rot;
    int page_shift;
    int heads_per;            // heads per thread (set by the launch function)
    int grad;
    float magnitude;
    unsigned long long turns[64];   // turns per position of pair i, times 2^64
};

cudaError_t launch_rope(const RopeArgs& a, int dtype, int layout, bool append, int num_sms, cudaStream_t stream);

// ---- block tables and slot maps (paged_step.cu)
constexpr int MAX_PAGED_SEQS = 8192;
struct StepArgs {
    const int* cache_lens;   // [n]
    const int* new_lens;     // [n]; < 0: the request has ended
    int* table;              // [n][width]
    int* free_pages;         // [n_pages]
    const int* free_count;   // [1]
    int* kv_lens;            // [n]
    int* cu_q;               // [n + 1]
    int* positions;          // [rows]
    long long* slots;        // [rows]
    int* free_count_out;     // [1]
    int* status;             // [n]
    int n, width, n_pages, rows;
    int page_shift;
};

cudaError_t launch_paged_step(const StepArgs& a, int num_sms, cudaStream_t stream);

// ---- attention over a paged cache
// Query rows of one KV head are packed token-major, the G = H / Hkv query heads of a
// token side by side: a tile is `tokens` consecutive new tokens of one sequence and
// one KV head (up to tokens * G rows), and its keys are walked in blocks of `block`.
// Two kernels share plan and arguments: mma.sync on up to 16 rows (single tokens and
// short drafts) and tcgen05 on up to 128 rows (chunks).
struct PagedTiling {
    int tokens;     // new tokens per tile
    int block;      // keys per block
    int grid;       // CTAs
    int start_cost; // cost of a tile's start and end, in keys
    int snap;       // a cut leaves at least this many blocks on both sides
    int whole;      // a tile of fewer blocks is not cut
    int least;      // cost per CTA from which on another CTA takes part
    int join, join_rows;   // time that a part takes in the join of its tile, in keys, per join_rows rows
    int waves;      // whole tiles are dealt out in up to this many waves before the rest is cut (0: all is cut)
    int one_each;   // (waves) all tiles run whole if no CTA's cost more than this beyond its share
    int l2_bytes;   // (waves) keys and values beyond this do not stay in L2 for long
    // below few_keys keys per CTA on average (waves == 0) these replace start_cost and least
    int few_keys, few_start_cost, few_least;
};
constexpr int MAX_PAGED_WAVES = 64;

// A sequence of the step (those with new tokens only).  (Aligned, here and below: 16-byte loads and stores.)
struct alignas(16) PagedSeq {
    int q_start, q_len, kv_len;
    int index;      // row of the block table
};

// Position in the work: block k of tile `tile` of KV head `head` of sequence `seq`.
struct alignas(16) PagedPos {
    int seq, head, tile, k;
};

// `slot` consecutive tiles that a CTA runs whole in one wave, from `pos` on.
struct alignas(16) PagedSlot {
    PagedPos pos;
    PagedSeq seq;   // the sequence of `pos`
};

// The part of the work that is cut, for one CTA: from `start` (inclusive) to `end` (exclusive), plus what it
// needs to begin and to publish unfinished tiles.  A tile cut over CTAs c0 .. c1 is
// merged by the last of them to finish, in the order of the CTAs.
struct alignas(16) PagedRange {
    PagedPos start, end;
    PagedSeq first;       // the sequence of `start`
    int c0, c1;           // CTAs of the tile that `start` continues (start.k > 0)
    int c1_last;          // last CTA of the tile that the range leaves unfinished (end.k > 0)
    int unused;
};
static_assert(sizeof(PagedRange) == 64, "one range is one 64-byte line");

// What a plan was made for; a launch with other arguments does nothing and reports it.
struct alignas(16) PagedHeader {
    int n_seqs;           // sequences with new tokens
    int ranges;           // CTAs with work
    int n, H, Hkv, D, tokens, block, grid, causal, window;
    int waves;            // slots of every CTA before its range
    int slot;             // tiles per slot
    int slot_ctas;        // CTAs that have a slot in the last wave
    int unused[2];
};
constexpr int PAGED_MAGIC_SITE = 3;   // error record: the plan does not match the call

struct PagedWork {
    PagedHeader* header;
    unsigned* counters;   // [grid] pieces of a cut tile finished, indexed by its first CTA
    PagedRange* ranges;   // [grid]
    PagedSeq* seqs;       // [n]
    PagedSlot* slots;     // [grid][MAX_PAGED_WAVES]
    float2* part_ml;      // [2 grid][rows] running max (log2 units) and sum of a partial result
    float* part_o;        // [2 grid][rows][D] unnormalised partial result
};

struct PagedPlanArgs {
    const int* cu_q;      // [n + 1]
    const int* kv_lens;   // [n]
    int n, H, Hkv, D, causal, window;
    PagedTiling tile;
    PagedWork work;
};

cudaError_t launch_paged_plan(const PagedPlanArgs& a, cudaStream_t stream);

struct PagedAttnArgs {
    const void* q;              // [T, H, D], rows q_stride elements apart
    const int* table;           // [n], rows table_stride entries apart
    float* lse;                 // [T, H] or null
    long long q_stride, table_stride;
    int T, H, Hkv, G, D, n, width, page_shift, n_pages;
    int k_head, v_head;         // elements between the heads of a cache
    int causal, window;         // window: 0 for none
    float c;                    // scale * log2(e), positive
    EpiParams epi;
    PagedTiling tile;
    PagedWork work;
    unsigned long long timeout_ns;
    FastDiv fd_G;
};

// tk, tv: a cache as the 5-D tensor (element, token % 8, 64-channel panel, token / 8, page), the
// head in the first coordinate.  A box is one page's tokens of one head (at most a block's), and
// lands as [token / 8][panel][token % 8][64 channels]: 1024-byte swizzle atoms, so that any
// number of pages side by side form one operand tile, with one copy per page.
//
// Tiles of up to 16 packed rows.
cudaError_t launch_attn_paged_rows(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, int dtype,
                                   cudaStream_t stream);

// Tiles of up to 128 packed rows; tq covers [T, Hkv, G, D] in boxes of one tile's rows.
cudaError_t launch_attn_paged(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const PagedAttnArgs& a, int dtype, cudaStream_t stream);

cudaError_t read_and_clear_paged_error(int* value, DeviceErrorInfo* info, int* drain_failed, unsigned long long* when);
cudaError_t read_and_clear_paged_rows_error(int* value, DeviceErrorInfo* info, int* drain_failed, unsigned long long* when);

}  // namespace xs
