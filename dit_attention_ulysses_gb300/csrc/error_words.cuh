// Addresses of a translation unit's error words (device_wait.cuh), for one look at all families'.
#pragma once

#include <cuda_runtime.h>

#include "device_wait.cuh"
#include "paged.h"

namespace xs {

static inline cudaError_t error_words_here(ErrorWords* w) {
    void* p[2] = {};
    cudaError_t e = cudaGetSymbolAddress(&p[0], g_device_error);
    if (e == cudaSuccess) e = cudaGetSymbolAddress(&p[1], g_drain_failed);
    w->error = static_cast<const int*>(p[0]);
    w->drain = static_cast<const int*>(p[1]);
    return e;
}

}  // namespace xs
