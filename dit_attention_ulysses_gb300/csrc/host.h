// Host-side helpers shared by the translation units of the C ABI (defined in api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "kernels.h"

namespace xs {
namespace host {

struct DeviceInfo {
    bool known = false;
    int sms = 0;
    int major = 0;
    int minor = 0;
    int coop = 0;   // cooperative launches supported
};

// Records a CUDA error for xs_attn_last_cuda_error and returns XS_ERR_CUDA.
int cuda_fail(cudaError_t e);

// Attributes of the current device; XS_ERR_UNSUPPORTED_DEVICE unless it is sm_103.
int device_info(DeviceInfo* out);

int get_encoder(PFN_cuTensorMapEncodeTiled_v12000* fn);

int check_scale(float scale);

unsigned long long timeout_ns();

// Output layout -> destination parameters and per-buffer byte size.
int layout_epi(int layout, void* const* outs, int B, int S, int H, int D, int P, EpiParams* epi, int* n_out,
               int64_t* out_bytes, bool* need_div);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

inline Range range_of(const void* p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, lo + static_cast<uintptr_t>(bytes)};
}

}  // namespace host
}  // namespace xs
