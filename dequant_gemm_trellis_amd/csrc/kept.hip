// Rows kept in 8 bits, and SwiGLU over many rows with its gradient
// (trellis_keep, trellis_restore, trellis_swiglu, trellis_swiglu_backward).
//
// Each reads its inputs once and writes its outputs once; the memory bounds them.
// A lane takes 8 adjacent columns of a row (of both halves of [g, u]), four lanes a
// group of 32, whose largest exponent they exchange in registers: no LDS, no second
// pass. Rows of any length start at any boundary: a wide access needs none.
//
// MI355X, us: [g, u] of 4096 x 17408 to h and 8 bits 101, and back through the gradient
// 100 (575 MB each, 5.7 TB/s, where a large copy reaches 5.2 to 5.5); 4096 x 5120 kept
// 12.9, restored 11.3; the gradient of 811 x 4112 with h made again 8.1 (40 MB), of rows
// that start off 16 bytes 10.9 (4111) and 10.2 (4110).
#include <algorithm>

#include "common.hpp"
#include "groups.hpp"
#include "kept.hpp"
#include "launch.hpp"

namespace trellis {
namespace {

constexpr int kThreads = 256;

// How rows of `width` values are dealt to workgroups: pieces of 8 values, a row's
// padded to whole groups of 32; several short rows make a bundle.
struct Deal {
    int rows, width;
    uint32_t pieces;   // of a row
    uint32_t inverse;  // ceil(2^32 / pieces): a piece's row in its bundle by a product
    uint32_t bundle;   // rows
    uint32_t groups;   // workgroups of a bundle
};

// A bundle has 2048 pieces at least (or all rows), so that at most 12% of its lanes are
// idle, in its last workgroup. They cost nothing that shows: the gradient of 811 rows of
// 4096 (none idle) and of 4112 (10%) takes 8.2 and 8.1 us. A piece's number in a bundle of several rows is below 4096, where
// the product with `inverse` gives the quotient exactly.
Deal deal(int rows, int width) {
    Deal d{rows, width, 4u * static_cast<uint32_t>((width + kKeptGroup - 1) / kKeptGroup), 0, 1, 0};
    if (d.pieces < 2048) d.bundle = (2048 + d.pieces - 1) / d.pieces;
    if (d.bundle > static_cast<uint32_t>(rows)) d.bundle = rows;
    d.inverse = static_cast<uint32_t>(((uint64_t{1} << 32) + d.pieces - 1) / d.pieces);
    d.groups = (d.bundle * d.pieces + kThreads - 1) / kThreads;
    return d;
}

dim3 grid_of(const Deal& d) { return dim3((d.rows + d.bundle - 1) / d.bundle * d.groups); }

// A lane's place: `left` of its 8 columns from `col` on are in the row (none or
// fewer for a padded piece); four lanes of a group are in or out together.
struct Place {
    int row, col, left, piece;
    bool in;
};
__device__ __forceinline__ Place place_of(const Deal& d) {
    const uint32_t bundle = blockIdx.x / d.groups;
    const uint32_t at = (blockIdx.x - bundle * d.groups) * kThreads + threadIdx.x;
    const uint32_t r = d.bundle > 1 ? __umulhi(at, d.inverse) : at >= d.pieces;
    const int row = static_cast<int>(bundle * d.bundle + r), piece = static_cast<int>(at - r * d.pieces);
    return {row, 8 * piece, d.width - 8 * piece, piece, r < d.bundle && row < d.rows};
}

__device__ __forceinline__ uint32_t exponent_at(const uint8_t* exponents, int row, const Deal& d, int piece) {
    return exponents[static_cast<size_t>(row) * (d.pieces / 4) + piece / 4];
}

// Keep a lane's 8 values of row `row`; every lane of the group calls it.
__device__ __forceinline__ void keep_piece(const u32x4& v, const Deal& d, size_t row, const Place& p,
                                           int8_t* __restrict__ codes, uint8_t* __restrict__ exponents) {
    const uint32_t e = largest_of_four(largest_exponent(v));
    if (p.piece % 4 == 0) exponents[row * (d.pieces / 4) + p.piece / 4] = static_cast<uint8_t>(e);
    if (p.left > 0) store_codes(codes + row * d.width + p.col, p.left, kept_codes(v, e));
}

__global__ __launch_bounds__(kThreads) void keep_kernel(const uint16_t* __restrict__ x, Deal d,
                                                        int8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ exponents) {
    const Place p = place_of(d);
    if (!p.in) return;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (p.left > 0) v = load_values(x + static_cast<size_t>(p.row) * d.width + p.col, p.left);
    keep_piece(v, d, p.row, p, codes, exponents);
}

__global__ __launch_bounds__(kThreads) void restore_kernel(KeptRows x, Deal d, uint16_t* __restrict__ out) {
    const Place p = place_of(d);
    if (!p.in || p.left <= 0) return;
    const size_t at = static_cast<size_t>(p.row) * d.width + p.col;
    const u32x2 q = load_codes(x.codes + at, p.left);
    store_values(out + at, p.left, kept_values(q, exponent_at(x.exponents, p.row, d, p.piece)));
}

// s = 1 / (1 + exp(-g)) of a bf16 value, formed 2^24 times smaller below: the denominator
// stays finite down to g = -105 and its reciprocal normal down to -103.97, where s is below
// float32's range (2^-150). exp(-g) is 2^t twice, which stays finite too, with t = -g times
// the upper 16 bits of log2(e) / 2, an exact product (g has 8), and once 1 - g c for the
// constant's rest. s is off by at most 10.5 2^-24 of it; from exp2(-g log2(e) - 24), whose
// argument is rounded once, it was by 2^-18.5. SwiGLU of 16384 x 768 takes 13.2 us with it
// and took 12.8, of 4096 x 17408 with [g, u] kept 102 and 102.
__device__ __forceinline__ float sigmoid(float g) {
    g = __builtin_amdgcn_fmed3f(g, -128.f, 128.f);  // no 0 times an infinite 1 - g c
    const float half = __builtin_amdgcn_exp2f(g * -0x1.7154p-1f);
    const float rest = fmaf(g, -0x1.480fb6p-42f, 0x1p-24f);
    const float denominator = fmaf(half * rest, half, 0x1p-24f);
    return __builtin_amdgcn_rcpf(denominator) * 0x1p-24f;
}

// h of 8 columns: each value in float32, rounded once.
__device__ __forceinline__ u32x4 swiglu8(const u32x4& g, const u32x4& u) {
    u32x4 h;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const float g0 = bf16_low(g[d]), g1 = bf16_high(g[d]);
        h[d] = pack_bf16(g0 * sigmoid(g0) * bf16_low(u[d]), g1 * sigmoid(g1) * bf16_high(u[d]));
    }
    return h;
}

template <bool KEEP>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(const uint16_t* __restrict__ gu, Deal d,
                                                          uint16_t* __restrict__ h,
                                                          int8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ exponents) {
    const Place p = place_of(d);
    if (!p.in) return;
    u32x4 g = {0u, 0u, 0u, 0u}, u = {0u, 0u, 0u, 0u};
    const size_t row = static_cast<size_t>(p.row);
    if (p.left > 0) {
        const uint16_t* at = gu + 2 * row * d.width + p.col;
        g = load_values(at, p.left);
        u = load_values(at + d.width, p.left);
        store_values(h + row * d.width + p.col, p.left, swiglu8(g, u));
    }
    if constexpr (KEEP) {
        keep_piece(g, d, 2 * row, p, codes, exponents);
        keep_piece(u, d, 2 * row + 1, p, codes, exponents);
    }
}

// d silu(g) / dg = s (1 + g (1 - s)).
template <bool KEPT, bool AGAIN>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(
    const uint16_t* __restrict__ dh, const uint16_t* __restrict__ gu, KeptRows kept, Deal d,
    uint16_t* __restrict__ dgu, uint16_t* __restrict__ h) {
    const Place p = place_of(d);
    if (!p.in || p.left <= 0) return;
    const size_t row = static_cast<size_t>(p.row), at = 2 * row * d.width + p.col;
    const u32x4 dv = load_values(dh + row * d.width + p.col, p.left);
    u32x4 g, u;
    if constexpr (KEPT) {
        const u32x2 qg = load_codes(kept.codes + at, p.left);
        const u32x2 qu = load_codes(kept.codes + at + d.width, p.left);
        const uint32_t eg = exponent_at(kept.exponents, 2 * p.row, d, p.piece);
        const uint32_t eu = exponent_at(kept.exponents, 2 * p.row + 1, d, p.piece);
        g = kept_values(qg, eg);
        u = kept_values(qu, eu);
    } else {
        g = load_values(gu + at, p.left);
        u = load_values(gu + at + d.width, p.left);
    }
    u32x4 dg, du;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        float og[2], ou[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float gv = i ? bf16_high(g[w]) : bf16_low(g[w]), uv = i ? bf16_high(u[w]) : bf16_low(u[w]);
            const float dhv = i ? bf16_high(dv[w]) : bf16_low(dv[w]);
            const float s = sigmoid(gv);
            og[i] = dhv * (s * fmaf(gv, 1.f - s, 1.f)) * uv;
            ou[i] = dhv * (gv * s);
        }
        dg[w] = pack_bf16(og[0], og[1]);
        du[w] = pack_bf16(ou[0], ou[1]);
    }
    store_values(dgu + at, p.left, dg);
    store_values(dgu + at + d.width, p.left, du);
    if constexpr (AGAIN) store_values(h + row * d.width + p.col, p.left, swiglu8(g, u));
}

// A launch has fewer than 2^32 lanes, each of them 8 values of a row (of both halves of
// [g, u]): what SwiGLU keeps of 2^34 columns has twice as many values, and comes in two.
template <typename F>
hipError_t by_parts(int rows, int width, F&& launch) {
    const int64_t padded = (width + kKeptGroup - 1) / kKeptGroup * kKeptGroup;
    const int most = static_cast<int>(std::min<int64_t>(rows, (int64_t{1} << 34) / padded));
    for (int64_t row = 0; row < rows; row += most) {
        const Deal d = deal(static_cast<int>(std::min<int64_t>(most, rows - row)), width);
        const hipError_t e = launch(d, row * width, row * (d.pieces / 4));
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_keep(const uint16_t* x, int rows, int width, int8_t* codes, uint8_t* exponents,
                       hipStream_t st) {
    return by_parts(rows, width, [&](const Deal& d, int64_t at, int64_t group) {
        return launch_kernel(keep_kernel, grid_of(d), dim3(kThreads), st, x + at, d, codes + at,
                             exponents + group);
    });
}

hipError_t launch_restore(const KeptRows& x, int rows, int width, uint16_t* out, hipStream_t st) {
    return by_parts(rows, width, [&](const Deal& d, int64_t at, int64_t group) {
        return launch_kernel(restore_kernel, grid_of(d), dim3(kThreads), st,
                             KeptRows{x.codes + at, x.exponents + group}, d, out + at);
    });
}

hipError_t launch_swiglu(const uint16_t* gu, int rows, int inter, uint16_t* h, int8_t* codes,
                         uint8_t* exponents, hipStream_t st) {
    const Deal d = deal(rows, inter);
    return launch_kernel(codes ? swiglu_kernel<true> : swiglu_kernel<false>, grid_of(d), dim3(kThreads), st,
                         gu, d, h, codes, exponents);
}

hipError_t launch_swiglu_backward(const uint16_t* dh, const uint16_t* gu, const KeptRows& kept, int rows,
                                  int inter, uint16_t* dgu, uint16_t* h, hipStream_t st) {
    const Deal d = deal(rows, inter);
    auto kernel = gu ? (h ? swiglu_backward_kernel<false, true> : swiglu_backward_kernel<false, false>)
                     : (h ? swiglu_backward_kernel<true, true> : swiglu_backward_kernel<true, false>);
    return launch_kernel(kernel, grid_of(d), dim3(kThreads), st, dh, gu, kept, d, dgu, h);
}

}  // namespace trellis
