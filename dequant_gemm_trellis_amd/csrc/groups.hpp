// Shared by the grouped operations: limits, bf16 packing, and the launchers
// of the sort (internal to libtrellis.so; callers have validated arguments).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace trellis {

constexpr int kMaxGroups = 1024;
constexpr int kMaxKeys = kMaxGroups + 1;  // one more for the slots outside every group
constexpr int kMaxRank = 128;             // of an adapter

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
hipError_t launch_adapters_backward(const uint16_t* dy, const uint16_t* x, const float* u,
                                    const int32_t* ids, const AdapterFactors& f, int rows,
                                    const uint16_t* base, uint16_t* dx, uint16_t* da, uint16_t* db,
                                    bool vec_in, bool vec_out, void* ws, hipStream_t st);

#ifdef __HIP__

// The float32 values of the low and the high bf16 of a word.
__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two floats rounded to bf16 (nearest-even), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    floatx2 p = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
}

#endif  // __HIP__

}  // namespace trellis
