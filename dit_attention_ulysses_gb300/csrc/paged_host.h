// Checks of arguments that the translation units of the paged-cache entry points share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/xsattn.h"
#include "host.h"
#include "kernels.h"
#include "paged.h"

namespace xs {
namespace host {

constexpr int64_t MAX_ELEMS = int64_t(1) << 40;
constexpr int64_t MAX_STRIDE = int64_t(1) << 35;   // elements: 8 tokens' TMA stride stays below 2^40 bytes

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// T rows of `width` elements, `stride` elements apart (2 bytes each).
struct Rows {
    uintptr_t base;
    int64_t n, width, stride;
};

inline Rows rows_of(const void* p, int64_t n, int64_t width, int64_t stride) {
    return Rows{reinterpret_cast<uintptr_t>(p), n, width * 2, stride * 2};
}

inline Range span(const Rows& r) {
    return Range{r.base, r.base + static_cast<uintptr_t>(r.n > 0 ? (r.n - 1) * r.stride + r.width : 0)};
}

// Rows of equal stride (columns of one wider matrix) overlap only where their
// columns do; otherwise the address ranges decide.
inline bool rows_overlap(const Rows& a, const Rows& b) {
    if (!overlaps(span(a), span(b))) return false;
    if (a.stride != b.stride || a.stride <= 0) return true;
    const int64_t d = b.base >= a.base ? static_cast<int64_t>((b.base - a.base) % static_cast<uintptr_t>(a.stride))
                                       : a.stride - 1 - static_cast<int64_t>((a.base - b.base - 1) %
                                                                             static_cast<uintptr_t>(a.stride));
    return d < a.width || a.stride - d < b.width;
}

inline int log2_of(int x) {
    int k = 0;
    while ((1 << k) < x) ++k;
    return k;
}

inline int check_page(int page_size, int n_pages) {
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return XS_ERR_PAGE;
    if (n_pages < 1 || static_cast<int64_t>(n_pages) * page_size > INT32_MAX) return XS_ERR_SHAPE;
    return XS_OK;
}

// A cache of elements of `bytes` bytes each.
struct CacheView {
    void *k, *v;
    const long long *k_strides, *v_strides;   // elements
    int n_pages, page_size, Hkv, D, dtype, bytes;
};

inline CacheView view_of(const xs_paged_cache& c) {
    return CacheView{c.k, c.v, c.k_strides, c.v_strides, c.n_pages, c.page_size, c.Hkv, c.D, c.dtype, 2};
}

inline CacheView view_of(const xs_paged_cache8& c) {
    return CacheView{c.k, c.v, c.k_strides, c.v_strides, c.n_pages, c.page_size, c.Hkv, c.D, c.dtype, 1};
}

// Strides (page, token, head) of a cache's K or V; those of an extent of one are not used.
struct CacheStrides {
    long long s[3];
};

inline int check_strides(const CacheView& c, const long long* strides, CacheStrides* out) {
    const int dims[3] = {c.n_pages, c.page_size, c.Hkv};
    for (int i = 0; i < 3; ++i) {
        const long long s = dims[i] == 1 ? c.D : strides[i];
        if (s < c.D || s > MAX_STRIDE) return XS_ERR_SHAPE;
        if (s * c.bytes % 16 != 0) return XS_ERR_ALIGNMENT;
        out->s[i] = s;
    }
    if ((c.Hkv - 1) * out->s[2] + c.D > INT32_MAX) return XS_ERR_SHAPE;   // a head's start is a TMA coordinate
    return XS_OK;
}

inline int check_cache(const CacheView& c, CacheStrides* ks, CacheStrides* vs) {
    if (!c.k || !c.v) return XS_ERR_NULL;
    if (c.D != 64 && c.D != 128) return XS_ERR_HEAD_DIM;
    if (c.dtype != XS_DTYPE_BF16 && c.dtype != XS_DTYPE_FP16) return XS_ERR_DTYPE;
    int rc = check_page(c.page_size, c.n_pages);
    if (rc != XS_OK) return rc;
    if (c.Hkv < 1 || c.Hkv > 4096) return XS_ERR_SHAPE;
    if ((rc = check_strides(c, c.k_strides, ks)) != XS_OK) return rc;
    if ((rc = check_strides(c, c.v_strides, vs)) != XS_OK) return rc;
    return aligned16(c.k) && aligned16(c.v) ? XS_OK : XS_ERR_ALIGNMENT;
}

inline Range cache_span(const void* p, const CacheStrides& s, const CacheView& c) {
    const int64_t last = (c.n_pages - 1) * static_cast<int64_t>(s.s[0]) + (c.page_size - 1) * static_cast<int64_t>(s.s[1]) +
                         (c.Hkv - 1) * static_cast<int64_t>(s.s[2]) + c.D;
    return range_of(p, last * c.bytes);
}

// Whether K and V of a cache share no element: apart in memory, or (one buffer for both, with
// equal strides) apart within every page, every token or every head, whatever holds both.  dims:
// pages, tokens (scales: blocks) and heads; `D` elements of `bytes` bytes each side by side.
inline bool kv_apart(const int (&dims)[3], int D, int bytes, const CacheStrides& ks, const CacheStrides& vs, const Range& k,
              const Range& v) {
    if (!overlaps(k, v)) return true;
    for (int i = 0; i < 3; ++i) {
        if (dims[i] > 1 && ks.s[i] != vs.s[i]) return false;
    }
    const uintptr_t lo = k.lo < v.lo ? k.lo : v.lo, hi = k.lo < v.lo ? v.lo : k.lo;
    for (int i = 0; i < 3; ++i) {
        if (dims[i] == 1) continue;
        int64_t width = D;   // span of the dimensions with smaller strides
        bool nested = true;
        for (int j = 0; j < 3; ++j) {
            if (j == i || dims[j] == 1) continue;
            if (ks.s[j] < ks.s[i]) width += (dims[j] - 1) * static_cast<int64_t>(ks.s[j]);
            else if (ks.s[j] % ks.s[i] != 0) nested = false;   // larger strides keep the offset's place
        }
        const int64_t stride = ks.s[i] * bytes, d = static_cast<int64_t>((hi - lo) % static_cast<uintptr_t>(stride));
        if (nested && d >= width * bytes && stride - d >= width * bytes) return true;
    }
    return false;
}

inline int check_rope(const xs_rope* rope) {
    if (!rope) return XS_ERR_NULL;
    if (rope->D != 64 && rope->D != 128) return XS_ERR_HEAD_DIM;
    if (rope->rot < 16 || rope->rot > rope->D || rope->rot % 16 != 0) return XS_ERR_ROPE;
    if (rope->layout != XS_ROPE_HALF && rope->layout != XS_ROPE_INTERLEAVED) return XS_ERR_LAYOUT;
    if (!std::isfinite(rope->magnitude)) return XS_ERR_ROPE;
    return XS_OK;
}

inline int check_rows(int T, int H, int D, long long stride) {
    if (T < 1 || H < 1 || H > 4096) return XS_ERR_SHAPE;
    if (stride < static_cast<long long>(H) * D || stride > MAX_STRIDE || T * static_cast<int64_t>(stride) > MAX_ELEMS)
        return XS_ERR_SHAPE;
    if (stride % 8 != 0) return XS_ERR_ALIGNMENT;
    return XS_OK;
}

inline void fill_rope(xs::RopeArgs* a, const xs_rope* rope, int T, int H, const int* positions) {
    std::memset(a, 0, sizeof *a);
    a->positions = positions;
    a->T = T;
    a->H = H;
    a->D = rope->D;
    a->rot = rope->rot;
    a->magnitude = rope->magnitude;
    std::memcpy(a->turns, rope->turns, sizeof a->turns);
}

// Packed query rows of a tile of the two attention kernels (attn_paged_rows.cu, attn_paged.cu).
constexpr int ROWS_FEW = 16, ROWS_TILE = 128;

struct Tiling {
    int rows;   // packed query rows of a tile
    xs::PagedTiling t;
};

inline int check_paged_shape(int n, int H, int Hkv, int D, int max_q, int causal, int window) {
    if (n < 1 || n > xs::MAX_PAGED_SEQS || H < 1 || Hkv < 1 || max_q < 1) return XS_ERR_SHAPE;
    if (D != 64 && D != 128) return XS_ERR_HEAD_DIM;
    if (H % Hkv != 0) return XS_ERR_DIVISIBILITY;
    if (H / Hkv > ROWS_TILE || H > 4096) return XS_ERR_SHAPE;
    if (window < 0 || (window > 0 && !causal)) return XS_ERR_SHAPE;
    return XS_OK;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace: header | counters | ranges | sequences | partial (m, l) | partial O.  Sized
// for every tiling of the shape, so one workspace serves steps of any max_q.
inline size_t paged_work(char* base, int n, int D, int sms, xs::PagedWork* w) {
    const size_t grid = 2 * static_cast<size_t>(sms);
    const size_t part_rows = 2 * static_cast<size_t>(sms) * ROWS_TILE;   // two parts per CTA
    static_assert(2 * 2 * ROWS_FEW <= 2 * ROWS_TILE, "the parts of both kernels fit");
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += align256(bytes);
        return base ? base + at : nullptr;
    };
    char* p;
    p = take(sizeof(xs::PagedHeader));
    if (w) w->header = reinterpret_cast<xs::PagedHeader*>(p);
    p = take(grid * sizeof(unsigned));
    if (w) w->counters = reinterpret_cast<unsigned*>(p);
    p = take(grid * sizeof(xs::PagedRange));
    if (w) w->ranges = reinterpret_cast<xs::PagedRange*>(p);
    p = take(static_cast<size_t>(n) * sizeof(xs::PagedSeq));
    if (w) w->seqs = reinterpret_cast<xs::PagedSeq*>(p);
    p = take(grid * xs::MAX_PAGED_WAVES * sizeof(xs::PagedSlot));
    if (w) w->slots = reinterpret_cast<xs::PagedSlot*>(p);
    p = take(part_rows * sizeof(float2));
    if (w) w->part_ml = reinterpret_cast<float2*>(p);
    p = take(part_rows * D * sizeof(float));
    if (w) w->part_o = reinterpret_cast<float*>(p);
    return off;
}

// Tiling of the paged attention, a function of the shape alone.
using TilingOf = Tiling (*)(int n, int Hkv, int G, int D, int max_q, int sms);

inline int plan_attn(TilingOf tiling_of, const int* cu_q, const int* kv_lens, int n, int H, int Hkv, int D, int max_q, int causal,
                     int window, void* workspace, size_t workspace_bytes, void* stream) {
    if (!cu_q || !kv_lens || !workspace) return XS_ERR_NULL;
    int rc = check_paged_shape(n, H, Hkv, D, max_q, causal, window);
    if (rc != XS_OK) return rc;
    if (!aligned(cu_q, 4) || !aligned(kv_lens, 4) || !aligned(workspace, 256)) return XS_ERR_ALIGNMENT;
    const Range w = range_of(workspace, static_cast<int64_t>(workspace_bytes));
    if (overlaps(w, range_of(cu_q, 4 * (static_cast<int64_t>(n) + 1))) || overlaps(w, range_of(kv_lens, 4 * static_cast<int64_t>(n))))
        return XS_ERR_OVERLAP;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != XS_OK) return rc;
    xs::PagedPlanArgs a;
    std::memset(&a, 0, sizeof a);
    if (workspace_bytes < paged_work(static_cast<char*>(workspace), n, D, dev.sms, &a.work)) return XS_ERR_WORKSPACE;
    a.cu_q = cu_q;
    a.kv_lens = kv_lens;
    a.n = n;
    a.H = H;
    a.D = D;
    a.causal = causal ? 1 : 0;
    a.window = window;
    a.tile = tiling_of(n, Hkv, H / Hkv, D, max_q, dev.sms).t;
    a.Hkv = Hkv / a.tile.heads;
    const cudaError_t e = xs::launch_paged_plan(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : cuda_fail(e);
}

// Checks the arguments of an attention over a cache of either kind (`more`: further inputs) and fills in what
// does not depend on it.
template <typename Args>
int prepare_attn(const Args& g, TilingOf tiling_of, const Range* more, int n_more, xs::PagedAttnArgs* a, CacheStrides* ks,
                 CacheStrides* vs, Tiling* tiling) {
    const auto& cache = g.cache;
    const int T = g.T, H = g.H, Hkv = cache.Hkv, D = cache.D, P = g.P, n = g.n;
    if (!g.q || !g.block_table || !g.workspace) return XS_ERR_NULL;
    if (T < 1) return XS_ERR_SHAPE;
    int rc = check_cache(view_of(cache), ks, vs);
    if (rc != XS_OK) return rc;
    if ((rc = check_paged_shape(n, H, Hkv, D, g.max_q, g.causal, g.window)) != XS_OK) return rc;
    int n_out = 0;
    int64_t out_bytes = 0;
    bool need_div = false;
    if ((rc = layout_epi(g.layout, g.outs, 1, T, H, D, P, &a->epi, &n_out, &out_bytes, &need_div)) != XS_OK) return rc;
    if (need_div) {
        if (P < 1) return XS_ERR_SHAPE;
        if (P > XS_MAX_P) return XS_ERR_TOO_MANY_RANKS;
        if (T % P != 0 || H % P != 0) return XS_ERR_DIVISIBILITY;
    }
    for (int i = 0; i < n_out; ++i)
        if (!g.outs[i]) return XS_ERR_NULL;
    if ((rc = check_rows(T, H, D, g.q_stride)) != XS_OK) return rc;
    if (g.table_width < 1 || (n > 1 && g.table_stride < g.table_width) || g.table_stride > MAX_STRIDE) return XS_ERR_SHAPE;
    if ((rc = check_scale(g.scale)) != XS_OK) return rc;
    if (!aligned16(g.q) || !aligned(g.block_table, 4) || !aligned(g.lse, 4) || !aligned(g.workspace, 256))
        return XS_ERR_ALIGNMENT;
    for (int i = 0; i < n_out; ++i)
        if (!aligned16(g.outs[i])) return XS_ERR_ALIGNMENT;
    const Range ins[4] = {span(rows_of(g.q, T, static_cast<int64_t>(H) * D, g.q_stride)),
                          cache_span(cache.k, *ks, view_of(cache)), cache_span(cache.v, *vs, view_of(cache)),
                          range_of(g.block_table, ((n > 1 ? (n - 1) * static_cast<int64_t>(g.table_stride) : 0) + g.table_width) * 4)};
    Range o[XS_MAX_P + 2];
    int n_all = 0;
    for (int i = 0; i < n_out; ++i) o[n_all++] = range_of(g.outs[i], out_bytes);
    if (g.lse) o[n_all++] = range_of(g.lse, static_cast<int64_t>(T) * H * 4);
    o[n_all++] = range_of(g.workspace, static_cast<int64_t>(g.workspace_bytes));
    for (int i = 0; i < n_all; ++i) {
        for (int j = i + 1; j < n_all; ++j)
            if (overlaps(o[i], o[j])) return XS_ERR_OVERLAP;
        for (const Range& r : ins)
            if (overlaps(o[i], r)) return XS_ERR_OVERLAP;
        for (int j = 0; j < n_more; ++j)
            if (overlaps(o[i], more[j])) return XS_ERR_OVERLAP;
    }
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != XS_OK) return rc;
    if (g.workspace_bytes < paged_work(static_cast<char*>(g.workspace), n, D, dev.sms, &a->work)) return XS_ERR_WORKSPACE;
    *tiling = tiling_of(n, Hkv, H / Hkv, D, g.max_q, dev.sms);
    a->q = g.q;
    a->table = g.block_table;
    a->lse = g.lse;
    a->q_stride = g.q_stride;
    a->table_stride = n > 1 ? g.table_stride : 0;
    a->T = T;
    a->H = H;
    a->Hkv = Hkv;
    a->G = H / Hkv;
    a->D = D;
    a->n = n;
    a->width = g.table_width;
    a->page_shift = log2_of(cache.page_size);
    a->n_pages = cache.n_pages;
    a->k_head = static_cast<int>(ks->s[2]);
    a->v_head = static_cast<int>(vs->s[2]);
    a->causal = g.causal ? 1 : 0;
    a->window = g.window;
    // never 0: a masked score is -infinity and stays so
    a->c = std::fmax(static_cast<float>(static_cast<double>(g.scale) * 1.4426950408889634), 1e-30f);
    a->tile = tiling->t;
    a->timeout_ns = timeout_ns();
    a->fd_G = xs::make_fastdiv(a->G);
    a->epi.fd_Sl = xs::make_fastdiv(a->epi.Sl);
    a->epi.fd_Hl = xs::make_fastdiv(a->epi.Hl);
    return XS_OK;
}

}  // namespace host
}  // namespace xs
