// Host-side argument checks shared by the C-ABI entry points.
#pragma once

#include <stdint.h>

#include "launch.hpp"
#include "trellis.h"

namespace trellis {

constexpr int32_t kMaxFeatures = 1 << 19;
constexpr uint64_t kMaxWeights = 1ull << 40;

struct Dims {
    int rows, cols, nb;
    CodeLayout lay;
};

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int check_geometry(const trellis_geometry* g, Dims* d) {
    if (!g) return TRELLIS_ERR_NULL;
    if (g->axis != 0 && g->axis != 1) return TRELLIS_ERR_GEOMETRY;
    if (g->T != 256 || g->L != 12) return TRELLIS_ERR_GEOMETRY;
    if (g->k < 2 || g->k > 4) return TRELLIS_ERR_GEOMETRY;
    if (g->in_features < 1 || g->out_features < 1) return TRELLIS_ERR_GEOMETRY;
    if (g->in_features > kMaxFeatures || g->out_features > kMaxFeatures) return TRELLIS_ERR_GEOMETRY;
    d->rows = g->axis == 1 ? g->out_features : g->in_features;
    d->cols = g->axis == 1 ? g->in_features : g->out_features;
    if (d->cols % g->T != 0) return TRELLIS_ERR_GEOMETRY;
    if (static_cast<uint64_t>(d->rows) * static_cast<uint64_t>(d->cols) > kMaxWeights)
        return TRELLIS_ERR_GEOMETRY;
    d->nb = d->cols / g->T;
    if (g->block_interleave != 0 && g->block_interleave != 2) return TRELLIS_ERR_GEOMETRY;
    if (g->block_interleave == 2 && d->nb % 2 != 0) return TRELLIS_ERR_GEOMETRY;
    d->lay = code_layout(g->block_interleave, d->rows, d->nb, g->k);
    return TRELLIS_OK;
}

// Operand checks shared by the compute entry points.
inline int check_operands(const void* codes, const float* scales, const float* lut) {
    if (!codes || !scales || !lut) return TRELLIS_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(lut, 16) || !aligned(scales, 4)) return TRELLIS_ERR_ALIGN;
    return TRELLIS_OK;
}

inline int check_io(const void* x, const void* y) {
    if (!x || !y) return TRELLIS_ERR_NULL;
    if (!aligned(x, 16) || !aligned(y, 16)) return TRELLIS_ERR_ALIGN;
    return TRELLIS_OK;
}

inline int status_of(hipError_t e) { return e == hipSuccess ? TRELLIS_OK : TRELLIS_ERR_HIP; }

}  // namespace trellis
