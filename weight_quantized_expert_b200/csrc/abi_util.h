// Helpers of the C entry points that live beside their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/focr_moe.h"

namespace focr {

focr_status report_error(focr_status s, const char* msg);   // the library's focr_last_error() record

inline focr_status reportf(focr_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline focr_status reportf(focr_status s, const char* fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return report_error(s, msg);
}

inline focr_status report_launch(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return FOCR_OK;
    return reportf(FOCR_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

inline bool misaligned(const void* p, size_t a) { return (uintptr_t)p % a != 0; }

// Whether two byte ranges share a byte.
inline bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
    return (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

// A caller's buffer.
struct Span {
    const void* at;
    size_t bytes;
};
// Whether one of `n` outputs shares a byte with another one or with one of `m` inputs (NULL buffers share none).
inline bool outputs_overlap(const Span* out, int n, const Span* in, int m) {
    for (int i = 0; i < n; ++i) {
        if (!out[i].at) continue;
        for (int j = i + 1; j < n; ++j)
            if (out[j].at && ranges_overlap(out[i].at, out[i].bytes, out[j].at, out[j].bytes)) return true;
        for (int j = 0; j < m; ++j)
            if (in[j].at && ranges_overlap(out[i].at, out[i].bytes, in[j].at, in[j].bytes)) return true;
    }
    return false;
}

// Launch with programmatic stream serialisation; cluster > 1 sets the cluster's x extent.
inline cudaError_t launch_kernel(const void* fn, dim3 grid, dim3 block, size_t smem, int cluster, void** args,
                                 cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace focr
