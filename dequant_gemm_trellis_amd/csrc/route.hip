// Slots sorted by group, token rows moved to the places of their slots and
// back (trellis_route, trellis_dispatch, trellis_combine and its gradient).
//
// Sorting is one stable counting sort: a slot's place is
//   offsets[id] + (slots of the same id before it),
// and the count before it splits into those of earlier chunks of slots (one
// workgroup each), of earlier waves of its chunk, of earlier 64-slot steps of
// its wave, and of lower lanes of its step. Each term is a count, so no
// atomic's order changes the result.
#include "common.hpp"
#include "groups.hpp"
#include "launch.hpp"

namespace trellis {
namespace {

// One workgroup sorts up to kMaxChunkSlots slots in one launch; more slots are
// cut into chunks: a launch counts each chunk's ids, a second one places them.
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kMaxSteps = 8;          // 64-slot steps of a wave: their ids stay in registers
constexpr int kMaxChunkSlots = kMaxSteps * kSortThreads;
// Slots that one workgroup sorts alone: 256 slots of 128 groups 4.5 us, 4096 7.8,
// 8192 11.7, where two launches take 3.4 + 7.1 us (and the host one more launch).
constexpr int kOneChunk = 8192;
constexpr int kChunkSlots = 2048;     // slots per workgroup of several, at least
constexpr int kMaxChunks = kMaxSlots / kMaxChunkSlots;  // each reads all chunks' counts

// Lanes of the wave whose key equals this lane's, among the lanes with `live`.
__device__ __forceinline__ uint64_t same_key(int key, bool live, int bits) {
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
        const bool one = (key >> b) & 1;
        const uint64_t ones = __ballot(one);
        same &= one ? ones : ~ones;
    }
    return same;
}

// Exclusive sum over the workgroup's kSortThreads values (wave sums in
// `part`, kSortWaves + 1 words of LDS); *total gets the sum of all.
__device__ __forceinline__ int scan_workgroup(int v, int* part, int* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(inc, d);
        if (lane >= d) inc += up;
    }
    if (lane == 63) part[wave] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        if (w < wave) before += part[w];
        all += part[w];
    }
    *total = all;
    return before + inc - v;
}

// The group key of slot i: its id, or `groups` (the group behind the others,
// which `tail` keeps) for an id outside them.
__device__ __forceinline__ int slot_key(const int32_t* ids, int i, int groups) {
    const int id = ids[i];
    return static_cast<uint32_t>(id) < static_cast<uint32_t>(groups) ? id : groups;
}

// The keys of a wave's steps of a chunk [s0, s1) (`keys` past its end): each wave
// takes a contiguous part. One memory round trip for all of them.
__device__ __forceinline__ void load_keys(const int32_t* __restrict__ ids, int s0, int s1, int groups,
                                          int keys, int& first, int& steps, int (&key)[kMaxSteps]) {
    steps = (s1 - s0 + kSortThreads - 1) / kSortThreads;
    first = s0 + static_cast<int>(threadIdx.x >> 6) * steps * kWave + (threadIdx.x & 63);
#pragma unroll
    for (int s = 0; s < kMaxSteps; ++s) {
        const int i = first + s * kWave;
        key[s] = s < steps && i < s1 ? slot_key(ids, i, groups) : keys;
    }
}

// Ids per chunk: counts[chunk][keys]. Equal keys of a wave's step are added by
// one lane (runs of one key would queue up at one counter otherwise).
__global__ __launch_bounds__(kSortThreads) void route_count_kernel(
    const int32_t* __restrict__ ids, int slots, int groups, int keys, int chunk,
    int32_t* __restrict__ counts) {
    __shared__ int hist[kMaxKeys];
    const int s0 = blockIdx.x * chunk, s1 = min(slots, s0 + chunk);
    const int lane = threadIdx.x & 63, bits = 32 - __clz(keys);
    int first, steps, key[kMaxSteps];
    load_keys(ids, s0, s1, groups, keys, first, steps, key);
    for (int g = threadIdx.x; g < keys; g += kSortThreads) hist[g] = 0;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kMaxSteps; ++s) {
        if (s >= steps) break;
        const bool live = key[s] < keys;
        const uint64_t same = same_key(key[s], live, bits);
        if (live && (same >> lane) == 1) atomicAdd(&hist[key[s]], __popcll(same));
    }
    __syncthreads();
    for (int g = threadIdx.x; g < keys; g += kSortThreads)
        counts[static_cast<size_t>(blockIdx.x) * keys + g] = hist[g];
}

// Places of one chunk's slots. keys = groups, or groups + 1 where the slots
// outside every group are kept as one more group behind the others (then
// offsets has keys + 1 entries). counts: every chunk's ids (null for one
// chunk, whose counts this kernel takes itself).
__global__ __launch_bounds__(kSortThreads) void route_place_kernel(
    const int32_t* __restrict__ ids, int slots, int groups, int keys, int chunk,
    const int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
    int32_t* __restrict__ order, int32_t* __restrict__ position) {
    // counts of each wave's part, then the first place of each (wave, key)
    __shared__ int next[kSortWaves * kMaxKeys];
    __shared__ int part[kSortWaves + 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int chunks = gridDim.x;
    const int s0 = blockIdx.x * chunk, s1 = min(slots, s0 + chunk);
    const int bits = 32 - __clz(keys);
    int first, steps, key[kMaxSteps], local[kMaxSteps];
    load_keys(ids, s0, s1, groups, keys, first, steps, key);
    for (int g = tid; g < kSortWaves * keys; g += kSortThreads) next[g] = 0;
    __syncthreads();
    // place of each slot among its wave's slots of the same key
#pragma unroll
    for (int s = 0; s < kMaxSteps; ++s) {
        if (s >= steps) break;
        const bool live = key[s] < keys;
        const uint64_t same = same_key(key[s], live, bits);
        int* n = next + wave * keys + key[s];
        local[s] = live ? *n + __popcll(same & ((1ull << lane) - 1)) : 0;
        wave_lds_sync();  // every lane has read its key's count
        if (live && (same >> lane) == 1) *n = local[s] + 1;  // the last lane of its key
        wave_lds_sync();
    }
    __syncthreads();
    // Per key: slots of all chunks, of earlier chunks, and of earlier waves.
    int base = 0;  // first place of these 1024 keys
    for (int g0 = 0; g0 < keys; g0 += kSortThreads) {
        const int g = g0 + tid;
        int mine = 0, earlier = 0, all = 0;
        if (g < keys) {
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                const int n = next[w * keys + g];
                next[w * keys + g] = mine;
                mine += n;
            }
            all = mine;
            if (counts) {
                all = 0;
#pragma unroll 8
                for (int q = 0; q < chunks; ++q) {
                    const int n = counts[static_cast<size_t>(q) * keys + g];
                    if (q < static_cast<int>(blockIdx.x)) earlier += n;
                    all += n;
                }
            }
        }
        int total;
        const int place = base + scan_workgroup(all, part, &total);
        if (g < keys) {
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) next[w * keys + g] += place + earlier;
            if (blockIdx.x == 0) offsets[g] = place;
        }
        base += total;
        __syncthreads();  // `part` is written again, and `next` is read by all waves
    }
    if (blockIdx.x == 0 && tid == 0) offsets[keys] = base;
#pragma unroll
    for (int s = 0; s < kMaxSteps; ++s) {
        const int i = first + s * kWave;
        if (s >= steps || i >= s1) break;
        const int place = key[s] < keys ? next[wave * keys + key[s]] + local[s] : -1;
        if (position) position[i] = place;
        if (place >= 0) order[place] = i;
    }
    for (int p = max(base, s0) + tid; p < s1; p += kSortThreads) order[p] = -1;
}

// ---- rows to their places and back ------------------------------------------
//
// All of these move rows at the memory's rate and do next to nothing to them.
// A thread holds 8 columns (16 bytes; rows of other lengths: one column), and
// a token's positions are uniform over its workgroup. Width 2048, 8 slots per
// token, 128 experts: 8192 tokens out 59 us (302 MB, 5.1 TB/s; a device copy
// reaches 5.5), the gradient of 4097 tokens' way back 59 us (286 MB, 4.8 TB/s),
// 32 tokens back 4 us.
constexpr int kMoveThreads = 256;

template <bool VEC> struct Cols { static constexpr int n = VEC ? 8 : 1; };

template <bool VEC>
__device__ __forceinline__ void load_cols(const uint16_t* p, float (&v)[Cols<VEC>::n]) {
    if constexpr (VEC) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            v[2 * d] = bf16_low(w[d]);
            v[2 * d + 1] = bf16_high(w[d]);
        }
    } else {
        v[0] = bf16_low(*p);
    }
}

template <bool VEC>
__device__ __forceinline__ void store_cols(uint16_t* p, const float (&v)[Cols<VEC>::n]) {
    if constexpr (VEC) {
        u32x4 w;
#pragma unroll
        for (int d = 0; d < 4; ++d) w[d] = pack_bf16(v[2 * d], v[2 * d + 1]);
        *reinterpret_cast<u32x4*>(p) = w;
    } else {
        *p = round_bf16(v[0]);
    }
}

// Grid: (column chunks, tokens): each x row is read once, whatever top_k.
template <bool VEC>
__global__ __launch_bounds__(kMoveThreads) void dispatch_kernel(
    const uint16_t* __restrict__ x, const int32_t* __restrict__ position, int tokens, int top_k,
    int width, uint16_t* __restrict__ out) {
    using Word = std::conditional_t<VEC, u32x4, uint16_t>;
    const int h = (blockIdx.x * kMoveThreads + threadIdx.x) * Cols<VEC>::n;
    const uint32_t slots = static_cast<uint32_t>(tokens) * static_cast<uint32_t>(top_k);
    for (int m = blockIdx.y; m < tokens; m += gridDim.y) {
        if (h >= width) continue;
        const Word v = *reinterpret_cast<const Word*>(x + static_cast<size_t>(m) * width + h);
        const int32_t* pos = position + static_cast<size_t>(m) * top_k;
        for (int j = 0; j < top_k; ++j) {
            const uint32_t p = static_cast<uint32_t>(pos[j]);
            if (p < slots) *reinterpret_cast<Word*>(out + static_cast<size_t>(p) * width + h) = v;
        }
    }
}

// Grid: (column chunks, tokens).
template <bool VEC>
__global__ __launch_bounds__(kMoveThreads) void combine_kernel(
    const uint16_t* __restrict__ y, const float* __restrict__ weights,
    const int32_t* __restrict__ position, int tokens, int top_k, int width,
    uint16_t* __restrict__ out) {
    constexpr int n = Cols<VEC>::n;
    const int h = (blockIdx.x * kMoveThreads + threadIdx.x) * n;
    const uint32_t slots = static_cast<uint32_t>(tokens) * static_cast<uint32_t>(top_k);
    for (int m = blockIdx.y; m < tokens; m += gridDim.y) {
        if (h >= width) continue;
        float sum[n] = {};
        const size_t first = static_cast<size_t>(m) * top_k;
        for (int j = 0; j < top_k; ++j) {
            const uint32_t p = static_cast<uint32_t>(position[first + j]);
            if (p >= slots) continue;
            const float w = weights ? weights[first + j] : 1.f;
            float v[n];
            load_cols<VEC>(y + static_cast<size_t>(p) * width + h, v);
#pragma unroll
            for (int e = 0; e < n; ++e) sum[e] = fmaf(w, v[e], sum[e]);
        }
        store_cols<VEC>(out + static_cast<size_t>(m) * width + h, sum);
    }
}

// One wave per slot: its dy row, and the dot product of its y row with the
// token's dout row (read again for each of the token's slots, from the L1 or
// L2 of the neighbouring waves).
template <bool VEC>
__global__ __launch_bounds__(kMoveThreads) void combine_backward_kernel(
    const uint16_t* __restrict__ dout, const uint16_t* __restrict__ y,
    const float* __restrict__ weights, const int32_t* __restrict__ position, int slots, int top_k,
    int width, uint16_t* __restrict__ dy, float* __restrict__ dweights) {
    constexpr int n = Cols<VEC>::n;
    const int lane = threadIdx.x & 63;
    const int waves = gridDim.x * (kMoveThreads / kWave);
    for (int i = blockIdx.x * (kMoveThreads / kWave) +
                 __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
         i < slots; i += waves) {
        const uint32_t p = static_cast<uint32_t>(position[i]);
        float dot = 0.f;
        if (p < static_cast<uint32_t>(slots)) {
            const float w = weights[i];
            const uint16_t* drow = dout + static_cast<size_t>(i / top_k) * width;
            const uint16_t* yrow = y + static_cast<size_t>(p) * width;
            uint16_t* dyrow = dy + static_cast<size_t>(p) * width;
            for (int h = lane * n; h < width; h += kWave * n) {
                float d[n], v[n];
                load_cols<VEC>(drow + h, d);
                load_cols<VEC>(yrow + h, v);
#pragma unroll
                for (int e = 0; e < n; ++e) {
                    dot = fmaf(d[e], v[e], dot);
                    d[e] *= w;
                }
                store_cols<VEC>(dyrow + h, d);
            }
        }
#pragma unroll
        for (int s = 32; s; s >>= 1) dot += __shfl_xor(dot, s);
        if (lane == 0) dweights[i] = dot;
    }
}

// Slots per workgroup, a multiple of kSortThreads between kChunkSlots and
// kMaxChunkSlots.
int chunk_slots(int slots) {
    const int even = (slots + kMaxChunks - 1) / kMaxChunks;
    return even > kChunkSlots ? (even + kSortThreads - 1) / kSortThreads * kSortThreads
                              : kChunkSlots;
}

dim3 move_grid(int width, int tokens, bool vec) {
    const int cols = kMoveThreads * (vec ? 8 : 1);
    return dim3((width + cols - 1) / cols, tokens < 65535 ? tokens : 65535);
}

}  // namespace

size_t route_workspace_bytes(int slots, int keys) {
    if (slots <= kOneChunk) return 0;
    const int chunk = chunk_slots(slots);
    return static_cast<size_t>((slots + chunk - 1) / chunk) * keys * sizeof(int32_t);
}

hipError_t launch_route(const int32_t* ids, int slots, int groups, bool tail, int32_t* offsets,
                        int32_t* order, int32_t* position, int32_t* counts, hipStream_t st) {
    const int keys = groups + (tail ? 1 : 0);
    if (slots <= kOneChunk)
        return launch_kernel(route_place_kernel, dim3(1), dim3(kSortThreads), st, ids, slots,
                             groups, keys, kOneChunk, nullptr, offsets, order, position);
    const int chunk = chunk_slots(slots), chunks = (slots + chunk - 1) / chunk;
    const hipError_t e = launch_kernel(route_count_kernel, dim3(chunks), dim3(kSortThreads), st, ids,
                                       slots, groups, keys, chunk, counts);
    if (e != hipSuccess) return e;
    return launch_kernel(route_place_kernel, dim3(chunks), dim3(kSortThreads), st, ids, slots,
                         groups, keys, chunk, counts, offsets, order, position);
}

hipError_t launch_dispatch(const uint16_t* x, const int32_t* position, int tokens, int top_k,
                           int width, uint16_t* out, bool vec, hipStream_t st) {
    return launch_kernel(vec ? dispatch_kernel<true> : dispatch_kernel<false>,
                         move_grid(width, tokens, vec), dim3(kMoveThreads), st, x, position, tokens,
                         top_k, width, out);
}

hipError_t launch_combine(const uint16_t* y, const float* weights, const int32_t* position,
                          int tokens, int top_k, int width, uint16_t* out, bool vec,
                          hipStream_t st) {
    return launch_kernel(vec ? combine_kernel<true> : combine_kernel<false>,
                         move_grid(width, tokens, vec), dim3(kMoveThreads), st, y, weights,
                         position, tokens, top_k, width, out);
}

hipError_t launch_combine_backward(const uint16_t* dout, const uint16_t* y, const float* weights,
                                   const int32_t* position, int tokens, int top_k, int width,
                                   uint16_t* dy, float* dweights, bool vec, hipStream_t st) {
    const int slots = tokens * top_k, per = kMoveThreads / kWave;
    return launch_kernel(vec ? combine_backward_kernel<true> : combine_backward_kernel<false>,
                         dim3((slots + per - 1) / per), dim3(kMoveThreads), st, dout, y, weights,
                         position, slots, top_k, width, dy, dweights);
}

}  // namespace trellis
