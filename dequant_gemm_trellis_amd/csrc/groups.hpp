// Shared by the grouped operations: limits, bf16 packing, and the launchers
// of the sort (internal to libtrellis.so; callers have validated arguments).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "launch.hpp"

namespace trellis {

struct KeptRows;  // kept.hpp

constexpr int kMaxGroups = 1024;
constexpr int kMaxSlots = 1 << 21;
constexpr int kMaxKeys = kMaxGroups + 1;  // one more for the slots outside every group
constexpr int kMaxRank = 128;             // of an adapter
constexpr int kTileRows = 64;             // rows of an adapter's tile: four 16-row operands

// Sort of `slots` ids (route.hip). With `tail`, slots outside [0, groups) form
// one more group behind the others (offsets then has groups + 2 entries) and
// every slot has a place; without, they are dropped. `position` may be null.
// `counts` holds route_workspace_bytes(slots, keys) bytes, keys = groups, or
// groups + 1 with `tail`.
size_t route_workspace_bytes(int slots, int keys);
hipError_t launch_route(const int32_t* ids, int slots, int groups, bool tail, int32_t* offsets,
                        int32_t* order, int32_t* position, int32_t* counts, hipStream_t st);

// Rows to their places and back; `vec` where rows are multiples of 8 values
// and every row array is 16-byte aligned.
hipError_t launch_dispatch(const uint16_t* x, const int32_t* position, int tokens, int top_k,
                           int width, uint16_t* out, bool vec, hipStream_t st);
hipError_t launch_combine(const uint16_t* y, const float* weights, const int32_t* position,
                          int tokens, int top_k, int width, uint16_t* out, bool vec,
                          hipStream_t st);
hipError_t launch_combine_backward(const uint16_t* dout, const uint16_t* y, const float* weights,
                                   const int32_t* position, int tokens, int top_k, int width,
                                   uint16_t* dy, float* dweights, bool vec, hipStream_t st);

// Low-rank adapters (adapters.hip): a [count][rank][in], b [count][rank][out].
// `vec_in` (`vec_out`): in (out) is a multiple of 8 and every array with rows
// of that length is 16-byte aligned. `base` may be null (zeros) or y (dx)
// itself; u may be null in launch_adapters.
struct AdapterFactors {
    const uint16_t* a;
    const uint16_t* b;
    const float* scales;
    int in, out, rank, count;
};
size_t adapters_workspace_bytes(int rows, int in, int out, int rank, int count, bool backward);
hipError_t launch_adapters(const uint16_t* x, const int32_t* ids, const AdapterFactors& f, int rows,
                           const uint16_t* base, uint16_t* y, float* u, bool vec_in, bool vec_out,
                           void* ws, hipStream_t st);
// x: bf16, or, where it is null, `kept`.
hipError_t launch_adapters_backward(const uint16_t* dy, const uint16_t* x, const KeptRows& kept,
                                    const float* u, const int32_t* ids, const AdapterFactors& f, int rows,
                                    const uint16_t* base, uint16_t* dx, uint16_t* da, uint16_t* db,
                                    bool vec_in, bool vec_out, void* ws, hipStream_t st);

// The experts' coded products (experts.hip): y[s] = W_e x[s] for the rows s of
// [offsets[e], offsets[e + 1]). Codes [experts] of `lay`, each `words` words.
struct ExpertWeights {
    const uint32_t* codes;
    const float* scales;  // [experts][stored rows]
    const float* lut;
    CodeLayout lay;
    size_t words;
    int axis, k, in, out, experts;
};
size_t experts_workspace_bytes(int axis, int in, int out, int rows, int experts);
hipError_t launch_experts(const uint16_t* x, int rows, const int32_t* offsets,
                          const ExpertWeights& w, uint16_t* y, void* ws, hipStream_t st);

#ifdef __HIP__

// The float32 values of the low and the high bf16 of a word.
__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two floats rounded to bf16 (nearest-even), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    floatx2 p = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
}

// The place of tile t in a list that holds, group by group, ceil(rows of the
// group / per) tiles. Each wave searches for itself, 64 groups at a time.
struct Found {
    int group;  // -1: past the end
    int index;  // tile within its group
    int first;  // the group's first place, and the place after its last
    int end;
};

__device__ __forceinline__ Found find_entry(const int32_t* __restrict__ offsets, int groups, int rows,
                                            int per, int t) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int g0 = 0; g0 < groups; g0 += 64) {
        const int g = g0 + lane;
        int first = 0, end = 0, n = 0;
        if (g < groups) {
            first = min(max(offsets[g], 0), rows);
            end = min(max(offsets[g + 1], first), rows);
            n = (end - first + per - 1) / per;
        }
        int inc = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int a = __shfl_up(inc, d);
            if (lane >= d) inc += a;
        }
        const uint64_t past = __ballot(before + inc > t);
        if (past) {
            const int l = __ffsll(static_cast<unsigned long long>(past)) - 1;
            // the same in every lane: as scalars, so that addresses stay scalar
            auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
            return {g0 + l, t - before - of(inc - n), of(first), of(end)};
        }
        before += __builtin_amdgcn_readlane(inc, 63);
    }
    return {-1, 0, 0, 0};
}

// 16 bytes at a 4-byte boundary (what a global access of any width needs).
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

// 8 values of a row from column `col` on, zeros past `width` and where !live
// (`row` is a row that can be read in any case). VEC: rows are multiples of 8
// values and 16-byte aligned. Otherwise a row starts at any 2-byte boundary, and
// the values come from the five (at a 4-byte boundary four) 4-byte words that
// hold them, whose outer halves are not used; without a branch, so that many
// such loads are in flight together. At the row's end they come one by one.
template <bool VEC>
__device__ __forceinline__ u32x4 load8(const uint16_t* __restrict__ row, int col, int width, bool live) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if constexpr (VEC) {
        if (live && col < width) v = *reinterpret_cast<const u32x4*>(row + col);
        return v;
    }
    const bool whole = col + 8 <= width;
    if (width >= 8) {  // uniform
        const uintptr_t p = reinterpret_cast<uintptr_t>(row + (whole ? col : 0));
        const uint32_t* w = reinterpret_cast<const uint32_t*>(p & ~static_cast<uintptr_t>(3));
        const uint32_t odd = (p >> 1) & 1;
        const u32x4 q = *reinterpret_cast<const u32x4_a4*>(w);
        const uint32_t last = w[3 + odd];
        const bool take = live && whole;
#pragma unroll
        for (int d = 0; d < 4; ++d)
            v[d] = take ? __builtin_amdgcn_alignbit(d < 3 ? q[d < 3 ? d + 1 : 3] : last, q[d], 16 * odd) : 0u;
    }
    if (live && !whole && col < width) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const uint32_t lo = col + 2 * d < width ? row[col + 2 * d] : 0u;
            const uint32_t hi = col + 2 * d + 1 < width ? row[col + 2 * d + 1] : 0u;
            v[d] = lo | (hi << 16);
        }
    }
    return v;
}

#endif  // __HIP__

}  // namespace trellis
