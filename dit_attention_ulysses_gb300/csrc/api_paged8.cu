// C ABI of the entry points of the 8-bit paged cache: host-side argument checks (everything is
// checked before any CUDA call), tensor maps and launches.  The declarations and their contracts
// are in include/xsattn.h.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <cstring>

#include "../../include/xsattn.h"
#include "host.h"
#include "paged.h"
#include "paged_host.h"

namespace {

using namespace xs::host;

// A cache's strides and address ranges: numbers of K, of V, scales of K, of V.
struct Checked8 {
    CacheStrides ks, vs, kss, vss;
    Range k, v, k_scales, v_scales;
};

int check_scale_strides(const int (&dims)[3], const long long* strides, CacheStrides* out) {
    for (int i = 0; i < 3; ++i) {
        const long long s = dims[i] == 1 ? 1 : strides[i];
        if (s < 1 || s > MAX_STRIDE) return XS_ERR_SHAPE;
        out->s[i] = s;
    }
    return XS_OK;
}

int check_cache8(const xs_paged_cache8& c, Checked8* x) {
    if (!c.k_scales || !c.v_scales) return XS_ERR_NULL;
    int rc = check_cache(view_of(c), &x->ks, &x->vs);
    if (rc != XS_OK) return rc;
    if (c.block < 16 || c.block > 128 || c.block > c.page_size || (c.block & (c.block - 1)) != 0) return XS_ERR_PAGE;
    const int dims[3] = {c.n_pages, c.page_size / c.block, c.Hkv};
    if ((rc = check_scale_strides(dims, c.k_scale_strides, &x->kss)) != XS_OK) return rc;
    if ((rc = check_scale_strides(dims, c.v_scale_strides, &x->vss)) != XS_OK) return rc;
    x->k = cache_span(c.k, x->ks, view_of(c));
    x->v = cache_span(c.v, x->vs, view_of(c));
    auto scales = [&](const void* p, const CacheStrides& s) {
        int64_t last = 1;
        for (int i = 0; i < 3; ++i) last += (dims[i] - 1) * static_cast<int64_t>(s.s[i]);
        return range_of(p, last);
    };
    x->k_scales = scales(c.k_scales, x->kss);
    x->v_scales = scales(c.v_scales, x->vss);
    return XS_OK;
}

xs::Codes8 codes_of(void* code, void* scale, const CacheStrides& cs, const CacheStrides& ss) {
    xs::Codes8 x;
    x.code = static_cast<uint8_t*>(code);
    x.scale = static_cast<uint8_t*>(scale);
    for (int i = 0; i < 3; ++i) {
        x.cs[i] = cs.s[i];
        x.ss[i] = ss.s[i];
    }
    return x;
}

// [n_pages, page, Hkv, D] as the 4-D tensor (element, token, head, page).  Box: `box_rows` tokens of `heads` heads.
int encode_cache8(CUtensorMap* m, const void* base, const CacheStrides& s, const xs_paged_cache8& c, int box_rows, int heads) {
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    int rc = get_encoder(&enc);
    if (rc != XS_OK) return rc;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.Hkv),
                                static_cast<cuuint64_t>(c.n_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(s.s[1]), static_cast<cuuint64_t>(s.s[2]), static_cast<cuuint64_t>(s.s[0])};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(c.D), static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(heads), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE,
                           c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                           c.D == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cuda_fail(cudaErrorInvalidValue);
    return XS_OK;
}

// Up to 8 packed rows (new tokens x heads to a KV head), with D = 64 up to 16, go to the kernel of few tokens, more to
// that of chunks.  12 and 16 rows of 128 (us, few tokens / chunks): 16 x 1000 keys 20.4 / 15.1 and 20.9 / 15.1, 1 x 32768
// 35.2 / 28.1 and 38.1 / 28.0, 64 x 8192 219 / 195 and 222 / 196 (fp16, whose Q has a part more, 266 / 238), 200 ragged
// sequences 78.5 / 75.3 and 79.2 / 77.7, but 1 x 4096 15.7 / 16.7 and 17.1 / 16.7, 64 ragged ones in fp16 66 / 72.  12 rows
// of 64: 1 x 4096 12.4 / 15.1, 64 x 4096 91.8 / 98.5, 200 ragged 56.9 / 67.6, but 16 x 1000 15.6 / 13.4.
Tiling make_tiling8(int n, int Hkv, int G, int D, int max_q, int sms) {
    Tiling x{};
    x.t.cache8 = 1;
    x.t.heads = 1;
    if (static_cast<int64_t>(G) * max_q > (D == 128 ? ROWS_FEW / 2 : ROWS_FEW)) {
        x.rows = ROWS_TILE;
        x.t.tokens = ROWS_TILE / G;
        x.t.block = 128;
        x.t.grid = sms;
        x.t.start_cost = 512;
        x.t.snap = 4;
        x.t.whole = 12;
        x.t.least = 512;        // (1 x 4096 keys, 32 rows: 18.6 us; with 1024 a fifth more, with 384 the same)
        x.t.join = 38;
        x.t.join_rows = 32;
        x.t.waves = xs::MAX_PAGED_WAVES;
        x.t.one_each = 2304;    // (24 rows: 64 x 2048 keys 79 us; with 1280 a fifth more, and 48 x 4096 5 %; ragged batches the same)
        // (8 x 96 new tokens over 2600 and 3800 keys, 43 and 61 MB: 50.3 and 60.3 us; with 32 MB 50.6 and 60.8)
        x.t.l2_bytes = 64 << 20;
        return x;
    }
    x.rows = static_cast<int64_t>(G) * max_q <= ROWS_FEW / 2 ? ROWS_FEW / 2 : ROWS_FEW;
    x.t.tokens = x.rows / G;
    // Pairs of KV heads (half the tiles, starts and joins, twice the work between waits) where a CTA still gets two of
    // them: 64 x 8192 keys 182 us, 199 with single heads; 200 ragged sequences 56 and 62.  With the heads of a page
    // apart in memory, which a plan does not know, they cost a little: 64 x 8192 178 and 171.
    if (x.rows == ROWS_FEW / 2 && Hkv % 2 == 0 && static_cast<int64_t>(n) * Hkv >= 2 * sms) x.t.heads = 2;
    x.t.block = 32;
    x.t.grid = 2 * sms;
    x.t.start_cost = 512;   // (64 ragged sequences: 60 us, 200 ragged: 56; 256: 71 and 61; 1024: 58 and 67)
    x.t.snap = 4;
    x.t.whole = 40;         // (16 x 1000 keys: 15.3 us; 20 and 30: 17.2; otherwise the same)
    x.t.least = 512;
    x.t.join = 4;
    x.t.join_rows = 512 / D;   // four channels to a thread
    x.t.few_keys = 512;
    x.t.few_start_cost = 128;
    x.t.few_least = 128;
    x.t.waves = 0;
    return x;
}

}  // namespace

extern "C" {

int xs_rope_append_paged8(const xs_rope_append8_args* args, void* stream) {
    if (!args) return XS_ERR_NULL;
    const xs_rope_append8_args& g = *args;
    const xs_paged_cache8& cache = g.cache;
    if (!g.k || !g.v || !g.slots) return XS_ERR_NULL;
    int rc;
    if (g.rope) {
        if (!g.q || !g.positions || !g.q_out) return XS_ERR_NULL;
        if ((rc = check_rope(g.rope)) != XS_OK) return rc;
    } else if (g.q || g.positions || g.q_out || g.H != 0) {
        return XS_ERR_ROPE;
    }
    Checked8 x;
    if ((rc = check_cache8(cache, &x)) != XS_OK) return rc;
    const int D = cache.D, T = g.T, H = g.H, Hkv = cache.Hkv;
    if (g.rope && g.rope->D != D) return XS_ERR_HEAD_DIM;
    if (g.rope) {
        if ((rc = check_rows(T, H, D, g.q_stride)) != XS_OK) return rc;
        if ((rc = check_rows(T, H, D, g.q_out_stride)) != XS_OK) return rc;
    }
    if ((rc = check_rows(T, Hkv, D, g.k_stride)) != XS_OK) return rc;
    if ((rc = check_rows(T, Hkv, D, g.v_stride)) != XS_OK) return rc;
    if (!aligned16(g.q) || !aligned16(g.k) || !aligned16(g.v) || !aligned16(g.q_out) || !aligned(g.positions, 4) ||
        !aligned(g.slots, 8))
        return XS_ERR_ALIGNMENT;
    const int n_q = g.rope ? T : 0;   // rows of q and q_out
    const Rows rq = rows_of(g.q, n_q, static_cast<int64_t>(H) * D, g.q_stride),
               rk = rows_of(g.k, T, static_cast<int64_t>(Hkv) * D, g.k_stride),
               rv = rows_of(g.v, T, static_cast<int64_t>(Hkv) * D, g.v_stride),
               ro = rows_of(g.q_out, n_q, static_cast<int64_t>(H) * D, g.q_out_stride);
    if (g.rope) {
        if (!(g.q == g.q_out && g.q_stride == g.q_out_stride) && rows_overlap(rq, ro)) return XS_ERR_OVERLAP;
        if (rows_overlap(rk, ro) || rows_overlap(rv, ro)) return XS_ERR_OVERLAP;
    }
    const int extents[3] = {cache.n_pages, cache.page_size, Hkv}, blocks[3] = {cache.n_pages, cache.page_size / cache.block, Hkv};
    if (!kv_apart(extents, D, 1, x.ks, x.vs, x.k, x.v) || !kv_apart(blocks, 1, 1, x.kss, x.vss, x.k_scales, x.v_scales))
        return XS_ERR_OVERLAP;
    for (const Range& s : {x.k_scales, x.v_scales})
        if (overlaps(s, x.k) || overlaps(s, x.v)) return XS_ERR_OVERLAP;
    const Range pos = range_of(g.positions, static_cast<int64_t>(n_q) * 4), sl = range_of(g.slots, static_cast<int64_t>(T) * 8);
    for (const Range& c : {x.k, x.v, x.k_scales, x.v_scales}) {
        for (const Rows* r : {&rq, &rk, &rv, &ro})
            if (overlaps(c, span(*r))) return XS_ERR_OVERLAP;
        if (overlaps(c, pos) || overlaps(c, sl)) return XS_ERR_OVERLAP;
    }
    if (overlaps(span(ro), pos) || overlaps(span(ro), sl)) return XS_ERR_OVERLAP;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != XS_OK) return rc;
    xs::Append8Args a;
    std::memset(&a, 0, sizeof a);
    a.q = g.q;
    a.k = g.k;
    a.v = g.v;
    a.q_out = g.q_out;
    a.positions = g.positions;
    a.slots = g.slots;
    a.kc = codes_of(cache.k, cache.k_scales, x.ks, x.kss);
    a.vc = codes_of(cache.v, cache.v_scales, x.vs, x.vss);
    a.q_stride = g.q_stride;
    a.k_stride = g.k_stride;
    a.v_stride = g.v_stride;
    a.qo_stride = g.q_out_stride;
    a.n_slots = static_cast<long long>(cache.n_pages) * cache.page_size;
    a.T = T;
    a.H = H;
    a.Hkv = Hkv;
    a.D = D;
    a.page_shift = log2_of(cache.page_size);
    a.block_shift = log2_of(cache.block);
    if (g.rope) {
        a.rot = g.rope->rot;
        a.magnitude = g.rope->magnitude;
        std::memcpy(a.turns, g.rope->turns, sizeof a.turns);
    }
    const cudaError_t e = xs::launch_append8(a, cache.dtype, g.rope ? g.rope->layout : XS_ROPE_HALF, dev.sms,
                                             static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : cuda_fail(e);
}

int xs_paged_read8(const xs_paged_read8_args* args, void* stream) {
    if (!args) return XS_ERR_NULL;
    const xs_paged_read8_args& g = *args;
    const xs_paged_cache8& cache = g.cache;
    if (!g.block_table || !g.cu_rows || !g.k_out || !g.v_out) return XS_ERR_NULL;
    Checked8 x;
    int rc = check_cache8(cache, &x);
    if (rc != XS_OK) return rc;
    const int D = cache.D, T = g.T, Hkv = cache.Hkv, n = g.n;
    if (n < 1 || n > xs::MAX_PAGED_SEQS) return XS_ERR_SHAPE;
    if (g.table_width < 1 || (n > 1 && g.table_stride < g.table_width) || g.table_stride > MAX_STRIDE) return XS_ERR_SHAPE;
    if ((rc = check_rows(T, Hkv, D, g.k_stride)) != XS_OK) return rc;
    if ((rc = check_rows(T, Hkv, D, g.v_stride)) != XS_OK) return rc;
    if (!aligned(g.block_table, 4) || !aligned(g.cu_rows, 4) || !aligned(g.first, 4) || !aligned16(g.k_out) || !aligned16(g.v_out))
        return XS_ERR_ALIGNMENT;
    const Rows ko = rows_of(g.k_out, T, static_cast<int64_t>(Hkv) * D, g.k_stride),
               vo = rows_of(g.v_out, T, static_cast<int64_t>(Hkv) * D, g.v_stride);
    if (rows_overlap(ko, vo)) return XS_ERR_OVERLAP;
    const int64_t n4 = static_cast<int64_t>(n) * 4;
    const Range ins[7] = {x.k, x.v, x.k_scales, x.v_scales, range_of(g.cu_rows, n4 + 4), range_of(g.first, g.first ? n4 : 0),
                          range_of(g.block_table, ((n > 1 ? (n - 1) * static_cast<int64_t>(g.table_stride) : 0) + g.table_width) * 4)};
    for (const Rows* r : {&ko, &vo})
        for (const Range& i : ins)
            if (overlaps(span(*r), i)) return XS_ERR_OVERLAP;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != XS_OK) return rc;
    xs::Read8Args a;
    std::memset(&a, 0, sizeof a);
    a.table = g.block_table;
    a.cu = g.cu_rows;
    a.first = g.first;
    a.k_out = g.k_out;
    a.v_out = g.v_out;
    a.kc = codes_of(cache.k, cache.k_scales, x.ks, x.kss);
    a.vc = codes_of(cache.v, cache.v_scales, x.vs, x.vss);
    a.k_stride = g.k_stride;
    a.v_stride = g.v_stride;
    a.table_stride = n > 1 ? g.table_stride : 0;
    a.T = T;
    a.n = n;
    a.width = g.table_width;
    a.n_pages = cache.n_pages;
    a.Hkv = Hkv;
    a.D = D;
    a.page_shift = log2_of(cache.page_size);
    a.block_shift = log2_of(cache.block);
    const cudaError_t e = xs::launch_read8(a, cache.dtype, dev.sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : cuda_fail(e);
}

int xs_attn_paged8_plan(const int* cu_q, const int* kv_lens, int n, int H, int Hkv, int D, int max_q, int causal,
                        int window, void* workspace, size_t workspace_bytes, void* stream) {
    return plan_attn(make_tiling8, cu_q, kv_lens, n, H, Hkv, D, max_q, causal, window, workspace, workspace_bytes, stream);
}

int xs_attn_paged8_fwd(const xs_attn_paged8_args* args, void* stream) {
    if (!args) return XS_ERR_NULL;
    const xs_paged_cache8& cache = args->cache;
    Checked8 x;
    int rc = check_cache8(cache, &x);
    if (rc != XS_OK) return rc;
    xs::PagedAttn8Args a;
    std::memset(&a, 0, sizeof a);
    const Range scales[2] = {x.k_scales, x.v_scales};
    Tiling tiling;
    if ((rc = prepare_attn(*args, make_tiling8, scales, 2, &a, &x.ks, &x.vs, &tiling)) != XS_OK) return rc;
    a.k_scale = static_cast<const uint8_t*>(cache.k_scales);
    a.v_scale = static_cast<const uint8_t*>(cache.v_scales);
    for (int i = 0; i < 3; ++i) {
        a.k_scale_strides[i] = x.kss.s[i];
        a.v_scale_strides[i] = x.vss.s[i];
    }
    a.block_shift = log2_of(cache.block);
    const int box_max = tiling.rows == ROWS_TILE ? 128 : 32;
    const int box = cache.page_size < box_max ? cache.page_size : box_max;
    CUtensorMap tk, tv;
    if ((rc = encode_cache8(&tk, cache.k, x.ks, cache, box, tiling.t.heads)) != XS_OK) return rc;
    if ((rc = encode_cache8(&tv, cache.v, x.vs, cache, box, tiling.t.heads)) != XS_OK) return rc;
    const auto launch = tiling.rows == ROWS_TILE ? xs::launch_attn_paged8 : xs::launch_attn_paged8_rows;
    const cudaError_t e = launch(tk, tv, a, cache.dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : cuda_fail(e);
}

}  // extern "C"
