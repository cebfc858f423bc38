// Argument checks that entry points share: alignment, extents, row distances, workspaces.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "lizard.h"

namespace lz {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

template <size_t n>
inline bool all_aligned(const void* const (&p)[n]) {
    for (const void* q : p)
        if (q != nullptr && !aligned16(q)) return false;
    return true;
}

inline lizard_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return LIZARD_OK;
    cudaGetLastError();
    return LIZARD_ERR_CUDA;
}

// Largest extents, so that no product of sizes below leaves 63 bits.
constexpr int64_t kMaxExtent = (int64_t)1 << 40;
inline bool extent(int64_t v, int64_t lo) { return v >= lo && v <= kMaxExtent; }

// A token distance: 0 selects the dense width; a row may not overlap the next.
inline bool row_stride(int64_t ld, int64_t width, int64_t* out) {
    *out = ld == 0 ? width : ld;
    return *out >= width && *out <= kMaxExtent;
}

// Checks an optional workspace and returns its header.
inline bool header_of(void* ws, size_t bytes, WsHeader** h) {
    *h = (WsHeader*)ws;
    return ws == nullptr || (aligned16(ws) && bytes >= kHeaderBytes);
}

inline bool batch_ok(int64_t B, int64_t L, int64_t C, int64_t nseq) {
    if (!extent(B, 1) || !extent(L, 0) || !extent(C, 1) || nseq < 0 || nseq > kMaxExtent) return false;
    if (L > 0x7fff0000) return false;  // the kernels count a row's tokens in 32 bits
    if (nseq > 0 && B != 1) return false;
    return (double)B * (double)(L > 0 ? L : 1) * (double)C < 9e15;
}

inline bool dtype_ok(int t) { return t == LIZARD_F32 || t == LIZARD_BF16; }

// Grids are one-dimensional and hold up to 2^31 - 1 CTAs.
inline bool grid_ok(double ctas) { return ctas < 2147483647.0; }

}  // namespace lz
