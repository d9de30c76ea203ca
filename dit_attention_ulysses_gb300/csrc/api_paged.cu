// C ABI of the paged-cache entry points: host-side argument checks (everything is
// checked before any CUDA call, so an invalid call launches nothing), tensor maps and
// launches.  The declarations and their contracts are in include/xsattn.h.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/xsattn.h"
#include "host.h"
#include "kernels.h"
#include "paged.h"

namespace {

using namespace xs::host;

constexpr int64_t MAX_ELEMS = int64_t(1) << 40;
constexpr int64_t MAX_STRIDE = int64_t(1) << 35;   // elements: 8 tokens' TMA stride stays below 2^40 bytes

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// T rows of `width` elements, `stride` elements apart (2 bytes each).
struct Rows {
    uintptr_t base;
    int64_t n, width, stride;
};

Rows rows_of(const void* p, int64_t n, int64_t width, int64_t stride) {
    return Rows{reinterpret_cast<uintptr_t>(p), n, width * 2, stride * 2};
}

Range span(const Rows& r) {
    return Range{r.base, r.base + static_cast<uintptr_t>(r.n > 0 ? (r.n - 1) * r.stride + r.width : 0)};
}

// Rows of equal stride (columns of one wider matrix) overlap only where their
// columns do; otherwise the address ranges decide.
bool rows_overlap(const Rows& a, const Rows& b) {
    if (!overlaps(span(a), span(b))) return false;
    if (a.stride != b.stride || a.stride <= 0) return true;
    const int64_t d = b.base >= a.base ? static_cast<int64_t>((b.base - a.base) % static_cast<uintptr_t>(a.stride))
                                       : a.stride - 1 - static_cast<int64_t>((a.base - b.base - 1) %
                                                                             static_cast<uintptr_t>(a.stride));
    return d < a.width || a.stride - d < b.width;
}

int log2_of(int x) {
    int k = 0;
    while ((1 << k) < x) ++k;
    return k;
}

int check_page(int page_size, int n_pages) {
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return XS_ERR_PAGE;
    if (n_pages < 1 || static_cast<int64_t>(n_pages) * page_size > INT32_MAX) return XS_ERR_SHAPE;
    return XS_OK;
}

// Strides (page, token, head) of a cache's K or V; those of an extent of one are not used.
struct CacheStrides {
    long long s[3];
};

int check_strides(const xs_paged_cache& c, const long long* strides, CacheStrides* out) {
    const int dims[3] = {c.n_pages, c.page_size, c.Hkv};
    for (int i = 0; i < 3; ++i) {
        const long long s = dims[i] == 1 ? c.D : strides[i];
        if (s < c.D || s > MAX_STRIDE) return XS_ERR_SHAPE;
        if (s % 8 != 0) return XS_ERR_ALIGNMENT;
        out->s[i] = s;
    }
    if ((c.Hkv - 1) * out->s[2] + c.D > INT32_MAX) return XS_ERR_SHAPE;   // a head's start is a TMA coordinate
    return XS_OK;
}

int check_cache(const xs_paged_cache& c, CacheStrides* ks, CacheStrides* vs) {
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

Range cache_span(const void* p, const CacheStrides& c, int n_pages, int page_size, int Hkv, int D) {
    const int64_t last = (n_pages - 1) * static_cast<int64_t>(c.s[0]) + (page_size - 1) * static_cast<int64_t>(c.s[1]) +
                         (Hkv - 1) * static_cast<int64_t>(c.s[2]) + D;
    return range_of(p, last * 2);
}

// Whether K and V of a cache share no element: apart in memory, or (one buffer for both, with
// equal strides) apart within every page, every token or every head, whatever holds both.
bool kv_apart(const xs_paged_cache& c, const CacheStrides& ks, const CacheStrides& vs, const Range& k, const Range& v) {
    if (!overlaps(k, v)) return true;
    const int dims[3] = {c.n_pages, c.page_size, c.Hkv};
    for (int i = 0; i < 3; ++i) {
        if (dims[i] > 1 && ks.s[i] != vs.s[i]) return false;
    }
    const uintptr_t lo = k.lo < v.lo ? k.lo : v.lo, hi = k.lo < v.lo ? v.lo : k.lo;
    for (int i = 0; i < 3; ++i) {
        if (dims[i] == 1) continue;
        int64_t width = c.D;   // span of the dimensions with smaller strides
        bool nested = true;
        for (int j = 0; j < 3; ++j) {
            if (j == i || dims[j] == 1) continue;
            if (ks.s[j] < ks.s[i]) width += (dims[j] - 1) * static_cast<int64_t>(ks.s[j]);
            else if (ks.s[j] % ks.s[i] != 0) nested = false;   // larger strides keep the offset's place
        }
        const int64_t stride = ks.s[i] * 2, d = static_cast<int64_t>((hi - lo) % static_cast<uintptr_t>(stride));
        if (nested && d >= width * 2 && stride - d >= width * 2) return true;
    }
    return false;
}

int check_rope(const xs_rope* rope) {
    if (!rope) return XS_ERR_NULL;
    if (rope->D != 64 && rope->D != 128) return XS_ERR_HEAD_DIM;
    if (rope->rot < 16 || rope->rot > rope->D || rope->rot % 16 != 0) return XS_ERR_ROPE;
    if (rope->layout != XS_ROPE_HALF && rope->layout != XS_ROPE_INTERLEAVED) return XS_ERR_LAYOUT;
    if (!std::isfinite(rope->magnitude)) return XS_ERR_ROPE;
    return XS_OK;
}

int check_rows(int T, int H, int D, long long stride) {
    if (T < 1 || H < 1 || H > 4096) return XS_ERR_SHAPE;
    if (stride < static_cast<long long>(H) * D || stride > MAX_STRIDE || T * static_cast<int64_t>(stride) > MAX_ELEMS)
        return XS_ERR_SHAPE;
    if (stride % 8 != 0) return XS_ERR_ALIGNMENT;
    return XS_OK;
}

void fill_rope(xs::RopeArgs* a, const xs_rope* rope, int T, int H, const int* positions) {
    std::memset(a, 0, sizeof *a);
    a->positions = positions;
    a->T = T;
    a->H = H;
    a->D = rope->D;
    a->rot = rope->rot;
    a->magnitude = rope->magnitude;
    std::memcpy(a->turns, rope->turns, sizeof a->turns);
}

// [n_pages, page, Hkv, D] as the 5-D tensor (element, token % 8, panel, token / 8, page); the heads
// lie along the first dimension, whatever their stride.  Box: `box_rows` tokens of one head.
int encode_cache(CUtensorMap* m, const void* base, const CacheStrides& c, const xs_paged_cache& cache, int box_rows) {
    const int n_pages = cache.n_pages, page_size = cache.page_size, Hkv = cache.Hkv, D = cache.D;
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    int rc = get_encoder(&enc);
    if (rc != XS_OK) return rc;
    const cuuint64_t dims[5] = {static_cast<cuuint64_t>((Hkv - 1) * c.s[2] + D), 8, static_cast<cuuint64_t>(D / 64),
                                static_cast<cuuint64_t>(page_size / 8), static_cast<cuuint64_t>(n_pages)};
    const cuuint64_t token = static_cast<cuuint64_t>(c.s[1]) * 2;
    const cuuint64_t strides[4] = {token, 128, 8 * token, static_cast<cuuint64_t>(c.s[0]) * 2};
    const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(D / 64), static_cast<cuuint32_t>(box_rows / 8), 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const CUtensorMapDataType type =
        cache.dtype == XS_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    // A row of 64 channels is 128 B: fetching 256 B brings another head's or token's row along, which is gone
    // from L2 when its turn comes (64 x 8192 keys, 8 heads side by side: 4.2 TB/s against 5.4)
    const CUtensorMapL2promotion l2 = D == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    const CUresult r = enc(m, type, 5, const_cast<void*>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, l2,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cuda_fail(cudaErrorInvalidValue);
    return XS_OK;
}

// q as a 4-D tensor (D, G, Hkv, T); box = 64 channels x the G heads of one KV head x `tokens`
// tokens: the packed rows of a tile, token-major.
int encode_q(CUtensorMap* m, const void* base, int T, int Hkv, int G, int D, long long stride, int tokens, int dtype) {
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    int rc = get_encoder(&enc);
    if (rc != XS_OK) return rc;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(G), static_cast<cuuint64_t>(Hkv),
                                static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(G) * D * 2,
                                   static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(G), 1, static_cast<cuuint32_t>(tokens)};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type =
        dtype == XS_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUresult r = enc(m, type, 4, const_cast<void*>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cuda_fail(cudaErrorInvalidValue);
    return XS_OK;
}

// ---- tiling of the paged attention, a function of the shape alone
// rows 16: attn_paged_rows.cu; 128: attn_paged.cu
constexpr int ROWS_FEW = 16, ROWS_TILE = 128;

struct Tiling {
    int rows;   // packed query rows of a tile
    xs::PagedTiling t;
};

Tiling make_tiling(int G, int D, int max_q, int sms) {
    Tiling x{};
    const int64_t need = static_cast<int64_t>(G) * max_q;
    // Few-tokens kernel against chunk kernel, us, by keys (which the host does not know):
    //   rows, heads    1 x 300   1 x 4096   1 x 32768  4 x 4096   16 x 1000  64 x 2048  32 x 8192  64 ragged
    //   16, 32 / 8     8.4/8.6   15.2/18.2  39.4/36.7  17.3/19.3  20.0/13.8  97.5/98.0  176/172    54.8/58.3
    //   16, 16 / 4     8.4/8.7   13.7/17.9  26.9/23.7  15.8/18.9  15.8/13.1  55.9/54.4  96.9/92.9  32.9/36.5
    //   16, 16 / 1     8.4/8.6   13.1/17.9  24.0/23.0  14.4/18.2  13.6/12.3  18.9/20.9  35.1/35.3  18.1/19.2
    //   12, 32 / 8     8.1/8.8   13.4/18.4  36.7/37.2  16.0/19.5  18.5/13.7  95.3/97.7  175/172    51.8/58.6
    // At 16 rows the chunk kernel wins with several short tiles to a CTA (16 x 1000) and on one long sequence, the other
    // elsewhere; at 12 to 15 rows that one is faster by 5 .. 15 % in the mean over these shapes.  Above 16 rows it would
    // need a second m16 tile: 20 rows, 64 x 2048 105 / 99, 16 x 1000 26 / 13.5, one of 32768 47 / 36
    if (need > ROWS_FEW) {
        x.rows = ROWS_TILE;
        x.t.tokens = ROWS_TILE / G;
        x.t.block = 128;
        x.t.grid = sms;
        x.t.start_cost = 512;
        x.t.snap = 4;
        x.t.whole = 12;
        x.t.least = 1024;
        // (per 32 rows) 40 new tokens over 20000 keys, 8 / 1 heads: 50 us at 0, 35 at 38, 42 at 125
        x.t.join = 38;
        x.t.join_rows = 32;
        x.t.waves = xs::MAX_PAGED_WAVES;
        x.t.one_each = 1280;      // a cut tile costs as much time as ten blocks (8 us)
        x.t.l2_bytes = 64 << 20;
        return x;
    }
    x.rows = ROWS_FEW;
    x.t.tokens = x.rows / G;
    x.t.block = 32;
    x.t.grid = 2 * sms;
    // 64 ragged sequences of 1 .. 16384 keys, 8 KV heads: 135 us at 128 keys, 105 at 256
    x.t.start_cost = 256;
    x.t.snap = 4;
    x.t.whole = 20;
    x.t.least = 512;
    // one token over 131072 keys, 8 / 1 heads: 43 us at 0, 29 at 4, 28 at 12; 4 x 2 over 1527, 8 / 1: 12.2, 12.7, 13.3
    x.t.join = 4;
    x.t.join_rows = 512 / D;   // four channels to a thread
    x.t.few_keys = 512;
    x.t.few_start_cost = 128;
    x.t.few_least = 128;
    x.t.waves = 0;   // one tile per sequence and KV head: no keys to share in L2
    return x;
}

int check_paged_shape(int n, int H, int Hkv, int D, int max_q, int causal, int window) {
    if (n < 1 || n > xs::MAX_PAGED_SEQS || H < 1 || Hkv < 1 || max_q < 1) return XS_ERR_SHAPE;
    if (D != 64 && D != 128) return XS_ERR_HEAD_DIM;
    if (H % Hkv != 0) return XS_ERR_DIVISIBILITY;
    if (H / Hkv > ROWS_TILE || H > 4096) return XS_ERR_SHAPE;
    if (window < 0 || (window > 0 && !causal)) return XS_ERR_SHAPE;
    return XS_OK;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace: header | counters | ranges | sequences | partial (m, l) | partial O.  Sized
// for every tiling of the shape, so one workspace serves steps of any max_q.
size_t paged_work(char* base, int n, int D, int sms, xs::PagedWork* w) {
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

}  // namespace

extern "C" {

int xs_rope_init(xs_rope* rope, int D, int rot, int layout, double base, int scaling, double factor, double context,
                 double low, double high, double magnitude) {
    if (!rope) return XS_ERR_NULL;
    if (D != 64 && D != 128) return XS_ERR_HEAD_DIM;
    if (rot < 16 || rot > D || rot % 16 != 0) return XS_ERR_ROPE;
    if (layout != XS_ROPE_HALF && layout != XS_ROPE_INTERLEAVED) return XS_ERR_LAYOUT;
    if (!std::isfinite(base) || base < 1.0 || !std::isfinite(magnitude) || std::fabs(magnitude) > 1e30)
        return XS_ERR_ROPE;
    if (scaling < XS_ROPE_PLAIN || scaling > XS_ROPE_BY_PARTS) return XS_ERR_ROPE;
    if (scaling != XS_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0)) return XS_ERR_ROPE;
    if (scaling == XS_ROPE_BY_PARTS && !(context >= 1.0 && std::isfinite(context) && high > low && std::isfinite(low) &&
                                         std::isfinite(high)))
        return XS_ERR_ROPE;
    const double tau = 6.283185307179586476925286766559;
    std::memset(rope, 0, sizeof *rope);
    rope->D = D;
    rope->rot = rot;
    rope->layout = layout;
    rope->magnitude = static_cast<float>(magnitude);
    if (scaling == XS_ROPE_STRETCH) base *= std::pow(factor, static_cast<double>(rot) / (rot - 2));
    for (int i = 0; i < rot / 2; ++i) {
        double theta = std::pow(base, -2.0 * i / rot);
        if (scaling == XS_ROPE_LINEAR) theta /= factor;
        if (scaling == XS_ROPE_BY_PARTS) {
            double keep = (theta * context / tau - low) / (high - low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            theta = theta * keep + theta / factor * (1.0 - keep);
        }
        rope->turns[i] = static_cast<unsigned long long>(theta / tau * 18446744073709551616.0 + 0.5);   // < 2^64 / 6
    }
    return XS_OK;
}

int xs_rope_fwd(const void* x, const int* positions, void* out, int T, int H, long long x_stride,
                long long out_stride, int dtype, int grad, const xs_rope* rope, void* stream) {
    if (!x || !positions || !out) return XS_ERR_NULL;
    int rc = check_rope(rope);
    if (rc != XS_OK) return rc;
    if (dtype != XS_DTYPE_BF16 && dtype != XS_DTYPE_FP16) return XS_ERR_DTYPE;
    if ((rc = check_rows(T, H, rope->D, x_stride)) != XS_OK) return rc;
    if ((rc = check_rows(T, H, rope->D, out_stride)) != XS_OK) return rc;
    if (!aligned16(x) || !aligned16(out) || !aligned(positions, 4)) return XS_ERR_ALIGNMENT;
    const int64_t width = static_cast<int64_t>(H) * rope->D;
    const Rows in = rows_of(x, T, width, x_stride), o = rows_of(out, T, width, out_stride);
    if (!(x == out && x_stride == out_stride) && rows_overlap(in, o)) return XS_ERR_OVERLAP;
    if (overlaps(span(o), range_of(positions, static_cast<int64_t>(T) * 4))) return XS_ERR_OVERLAP;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != XS_OK) return rc;
    xs::RopeArgs a;
    fill_rope(&a, rope, T, H, positions);
    a.q = x;
    a.q_out = out;
    a.q_stride = x_stride;
    a.qo_stride = out_stride;
    a.grad = grad ? 1 : 0;
    const cudaError_t e =
        xs::launch_rope(a, dtype, rope->layout, false, dev.sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : cuda_fail(e);
}

int xs_rope_append_paged(const xs_rope_append_args* args, void* stream) {
    if (!args) return XS_ERR_NULL;
    const xs_rope_append_args& g = *args;
    const xs_paged_cache& cache = g.cache;
    if (!g.q || !g.k || !g.v || !g.positions || !g.slots || !g.q_out) return XS_ERR_NULL;
    int rc = check_rope(g.rope);
    if (rc != XS_OK) return rc;
    CacheStrides ks, vs;
    if ((rc = check_cache(cache, &ks, &vs)) != XS_OK) return rc;
    const int D = cache.D, T = g.T, H = g.H, Hkv = cache.Hkv;
    if (g.rope->D != D) return XS_ERR_HEAD_DIM;
    if ((rc = check_rows(T, H, D, g.q_stride)) != XS_OK) return rc;
    if ((rc = check_rows(T, Hkv, D, g.k_stride)) != XS_OK) return rc;
    if ((rc = check_rows(T, Hkv, D, g.v_stride)) != XS_OK) return rc;
    if ((rc = check_rows(T, H, D, g.q_out_stride)) != XS_OK) return rc;
    if (!aligned16(g.q) || !aligned16(g.k) || !aligned16(g.v) || !aligned16(g.q_out) || !aligned(g.positions, 4) ||
        !aligned(g.slots, 8))
        return XS_ERR_ALIGNMENT;
    const Rows rq = rows_of(g.q, T, static_cast<int64_t>(H) * D, g.q_stride),
               rk = rows_of(g.k, T, static_cast<int64_t>(Hkv) * D, g.k_stride),
               rv = rows_of(g.v, T, static_cast<int64_t>(Hkv) * D, g.v_stride),
               ro = rows_of(g.q_out, T, static_cast<int64_t>(H) * D, g.q_out_stride);
    if (!(g.q == g.q_out && g.q_stride == g.q_out_stride) && rows_overlap(rq, ro)) return XS_ERR_OVERLAP;
    if (rows_overlap(rk, ro) || rows_overlap(rv, ro)) return XS_ERR_OVERLAP;
    const Range kc = cache_span(cache.k, ks, cache.n_pages, cache.page_size, Hkv, D),
                vc = cache_span(cache.v, vs, cache.n_pages, cache.page_size, Hkv, D);
    if (!kv_apart(cache, ks, vs, kc, vc)) return XS_ERR_OVERLAP;
    const Range pos = range_of(g.positions, static_cast<int64_t>(T) * 4),
                sl = range_of(g.slots, static_cast<int64_t>(T) * 8);
    for (const Range& c : {kc, vc}) {
        for (const Rows* r : {&rq, &rk, &rv, &ro})
            if (overlaps(c, span(*r))) return XS_ERR_OVERLAP;
        if (overlaps(c, pos) || overlaps(c, sl)) return XS_ERR_OVERLAP;
    }
    if (overlaps(span(ro), pos) || overlaps(span(ro), sl)) return XS_ERR_OVERLAP;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != XS_OK) return rc;
    xs::RopeArgs a;
    fill_rope(&a, g.rope, T, H, g.positions);
    a.q = g.q;
    a.k = g.k;
    a.v = g.v;
    a.q_out = g.q_out;
    a.k_cache = cache.k;
    a.v_cache = cache.v;
    a.slots = g.slots;
    a.q_stride = g.q_stride;
    a.k_stride = g.k_stride;
    a.v_stride = g.v_stride;
    a.qo_stride = g.q_out_stride;
    for (int i = 0; i < 3; ++i) {
        a.ks[i] = ks.s[i];
        a.vs[i] = vs.s[i];
    }
    a.n_slots = static_cast<long long>(cache.n_pages) * cache.page_size;
    a.Hkv = Hkv;
    a.page_shift = log2_of(cache.page_size);
    const cudaError_t e =
        xs::launch_rope(a, cache.dtype, g.rope->layout, true, dev.sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : cuda_fail(e);
}

int xs_paged_step(const int* cache_lens, const int* new_lens, int* block_table, int* free_pages,
                  const int* free_count, int n, int table_width, int n_pages, int page_size, int rows, int* kv_lens,
                  int* cu_q, int* positions, long long* slots, int* free_count_out, int* status, void* stream) {
    const void* all[] = {cache_lens, new_lens, free_count, block_table, free_pages, kv_lens, cu_q, positions,
                         free_count_out, status, slots};
    for (const void* p : all)
        if (!p) return XS_ERR_NULL;
    if (n < 1 || n > xs::MAX_PAGED_SEQS || table_width < 1 || rows < 1) return XS_ERR_SHAPE;
    int rc = check_page(page_size, n_pages);
    if (rc != XS_OK) return rc;
    if (static_cast<int64_t>(table_width) * page_size > INT32_MAX) return XS_ERR_SHAPE;
    for (const void* p : all)
        if (!aligned(p, 4)) return XS_ERR_ALIGNMENT;
    if (!aligned(slots, 8)) return XS_ERR_ALIGNMENT;
    const int64_t n4 = static_cast<int64_t>(n) * 4, r4 = static_cast<int64_t>(rows) * 4;
    const Range ins[3] = {range_of(cache_lens, n4), range_of(new_lens, n4), range_of(free_count, 4)};
    const Range outs[8] = {range_of(block_table, n4 * table_width), range_of(free_pages, static_cast<int64_t>(n_pages) * 4),
                           range_of(kv_lens, n4), range_of(cu_q, n4 + 4), range_of(positions, r4),
                           range_of(free_count_out, 4), range_of(status, n4), range_of(slots, 2 * r4)};
    for (int i = 0; i < 8; ++i) {
        for (int j = i + 1; j < 8; ++j)
            if (overlaps(outs[i], outs[j])) return XS_ERR_OVERLAP;
        for (const Range& r : ins)
            if (overlaps(outs[i], r)) return XS_ERR_OVERLAP;
    }
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != XS_OK) return rc;
    xs::StepArgs a;
    a.cache_lens = cache_lens;
    a.new_lens = new_lens;
    a.table = block_table;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.kv_lens = kv_lens;
    a.cu_q = cu_q;
    a.positions = positions;
    a.slots = slots;
    a.free_count_out = free_count_out;
    a.status = status;
    a.n = n;
    a.width = table_width;
    a.n_pages = n_pages;
    a.rows = rows;
    a.page_shift = log2_of(page_size);
    const cudaError_t e = xs::launch_paged_step(a, dev.sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : cuda_fail(e);
}

int xs_attn_paged_workspace_bytes(int n, int H, int Hkv, int D, size_t* bytes) {
    if (!bytes) return XS_ERR_NULL;
    int rc = check_paged_shape(n, H, Hkv, D, 1, 1, 0);
    if (rc != XS_OK) return rc;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != XS_OK) return rc;
    *bytes = paged_work(nullptr, n, D, dev.sms, nullptr);
    return XS_OK;
}

int xs_attn_paged_plan(const int* cu_q, const int* kv_lens, int n, int H, int Hkv, int D, int max_q, int causal,
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
    a.Hkv = Hkv;
    a.D = D;
    a.causal = causal ? 1 : 0;
    a.window = window;
    a.tile = make_tiling(H / Hkv, D, max_q, dev.sms).t;
    const cudaError_t e = xs::launch_paged_plan(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : cuda_fail(e);
}

int xs_attn_paged_fwd(const xs_attn_paged_args* args, void* stream) {
    if (!args) return XS_ERR_NULL;
    const xs_attn_paged_args& g = *args;
    const xs_paged_cache& cache = g.cache;
    const int T = g.T, H = g.H, Hkv = cache.Hkv, D = cache.D, P = g.P, n = g.n;
    if (!g.q || !g.block_table || !g.workspace) return XS_ERR_NULL;
    if (T < 1) return XS_ERR_SHAPE;
    CacheStrides ks, vs;
    int rc = check_cache(cache, &ks, &vs);
    if (rc != XS_OK) return rc;
    if ((rc = check_paged_shape(n, H, Hkv, D, g.max_q, g.causal, g.window)) != XS_OK) return rc;
    xs::PagedAttnArgs a;
    std::memset(&a, 0, sizeof a);
    int n_out = 0;
    int64_t out_bytes = 0;
    bool need_div = false;
    if ((rc = layout_epi(g.layout, g.outs, 1, T, H, D, P, &a.epi, &n_out, &out_bytes, &need_div)) != XS_OK) return rc;
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
                          cache_span(cache.k, ks, cache.n_pages, cache.page_size, Hkv, D),
                          cache_span(cache.v, vs, cache.n_pages, cache.page_size, Hkv, D),
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
    }
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != XS_OK) return rc;
    if (g.workspace_bytes < paged_work(static_cast<char*>(g.workspace), n, D, dev.sms, &a.work)) return XS_ERR_WORKSPACE;
    const Tiling tiling = make_tiling(H / Hkv, D, g.max_q, dev.sms);
    a.q = g.q;
    a.table = g.block_table;
    a.lse = g.lse;
    a.q_stride = g.q_stride;
    a.table_stride = n > 1 ? g.table_stride : 0;
    a.T = T;
    a.H = H;
    a.Hkv = Hkv;
    a.G = H / Hkv;
    a.D = D;
    a.n = n;
    a.width = g.table_width;
    a.page_shift = log2_of(cache.page_size);
    a.n_pages = cache.n_pages;
    a.k_head = static_cast<int>(ks.s[2]);
    a.v_head = static_cast<int>(vs.s[2]);
    a.causal = g.causal ? 1 : 0;
    a.window = g.window;
    // never 0: a masked score is -infinity and stays so
    a.c = std::fmax(static_cast<float>(static_cast<double>(g.scale) * 1.4426950408889634), 1e-30f);
    a.tile = tiling.t;
    a.timeout_ns = timeout_ns();
    a.fd_G = xs::make_fastdiv(a.G);
    a.epi.fd_Sl = xs::make_fastdiv(a.epi.Sl);
    a.epi.fd_Hl = xs::make_fastdiv(a.epi.Hl);
    const int box_max = tiling.rows == ROWS_TILE ? 128 : 32;
    const int box = cache.page_size < box_max ? cache.page_size : box_max;
    CUtensorMap tk, tv;
    if ((rc = encode_cache(&tk, cache.k, ks, cache, box)) != XS_OK) return rc;
    if ((rc = encode_cache(&tv, cache.v, vs, cache, box)) != XS_OK) return rc;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (tiling.rows == ROWS_TILE) {
        CUtensorMap tq;
        if ((rc = encode_q(&tq, g.q, T, Hkv, a.G, D, g.q_stride, tiling.t.tokens, cache.dtype)) != XS_OK) return rc;
        e = xs::launch_attn_paged(tq, tk, tv, a, cache.dtype, st);
    } else {
        e = xs::launch_attn_paged_rows(tk, tv, a, cache.dtype, st);
    }
    return e == cudaSuccess ? XS_OK : cuda_fail(e);
}

}  // extern "C"
