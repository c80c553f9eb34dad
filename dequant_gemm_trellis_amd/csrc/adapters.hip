// Low-rank adapters of many requests beside one shared projection
// (trellis_adapters, trellis_adapters_backward). With a = ids[m]:
//   u[m] = A[a] x[m],              y[m] = base[m] + s[a] B[a]^T u[m]
//   g[m] = s[a] B[a] dy[m],        dx[m] = base[m] + A[a]^T g[m]
//   dA[a] = sum_m g[m] x[m]^T,     dB[a] = sum_m s[a] u[m] dy[m]^T
// A is [count][rank][in], B [count][rank][out]: stored alike, so three
// products serve both directions: "inner" (a wide row times a factor's rows),
// "expand" (a rank-long row times a factor, added to a wide row) and "outer"
// (the sum over an adapter's rows of a rank-long times a wide row). Each reads
// or writes the wide rows once and does little with them, so the memory bounds
// them all.
//
// Few rows: one or two launches (the gradient: three) that follow each row's own
// adapter, all in float32.
// Many rows: the rows are sorted by adapter and cut into tiles of 64 rows of
// one adapter, which share the factor's values in bf16 matrix instructions.
// There a rank-long float32 value w (u or g) enters as three bf16 parts whose sum
// is w: its mantissa's upper, middle and lower 8 bits, so that every product is
// exact and the sums are float32 as those of few rows. (Two parts, 16 bits of
// mantissa, take up to 7% less time, but then 1.7e-3 to 2.5e-3 of the bf16 results
// of 4096 rows are not the float64 value rounded; with three 1.0e-4 to 3.0e-4.)
// Two parts of 16 ranks fill the 32 contraction slots of one 16x16x32 instruction.
//
// A matrix instruction contracts over 8 consecutive values per lane. Where the
// contraction runs across stored rows (ranks in expand, tokens in outer), a
// lane loads an 8 x 8 patch, 16 bytes from each of 8 rows, and transposes it
// in registers (one byte permute per output word): operand q then holds column
// 8 j + q, and the eight results give a lane 8 adjacent columns to store.
//
// MI355X, 5120 -> 17408: 1 row at rank 16 6.2 us; 4096 rows, 4 adapters, 82 us, 58
// of them y and base at 4.9 TB/s; their gradient at rank 32, 2 adapters, 142 us:
// dy read twice (48 us in the inner product, 3.0 TB/s; 51 with x in both outer
// sums, 3.6 TB/s: the waves, two to a SIMD, wait 42 and 53% of the time for
// data), dx 21, the sort and the tiles' and segments' sums 22.
#include "common.hpp"
#include "groups.hpp"
#include "launch.hpp"

namespace trellis {
namespace {

constexpr int kSubs = kTileRows / 16;
constexpr int kWgThreads = 256;
constexpr int kWgWaves = kWgThreads / kWave;
constexpr int kStrip = 128;            // columns per wave: 16 lanes x 8
constexpr int kMaxSegTiles = 16;       // tiles of one segment of the outer sums: 1024 rows

// 8 values to a row from column `col` on (none past `width`); see load8.
template <bool VEC>
__device__ __forceinline__ void store8(uint16_t* __restrict__ row, int col, int width, u32x4 v) {
    if constexpr (VEC) {
        if (col < width) *reinterpret_cast<u32x4*>(row + col) = v;
    } else if (col + 8 <= width) {
        uint16_t* p = row + col;
        if (reinterpret_cast<uintptr_t>(p) & 2) {
            p[0] = static_cast<uint16_t>(v[0]);
            uint32_t* w = reinterpret_cast<uint32_t*>(p + 1);
#pragma unroll
            for (int d = 0; d < 3; ++d) w[d] = __builtin_amdgcn_alignbit(v[d + 1], v[d], 16);
            p[7] = static_cast<uint16_t>(v[3] >> 16);
        } else {
            *reinterpret_cast<u32x4_a4*>(p) = v;
        }
    } else {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if (col + 2 * d < width) row[col + 2 * d] = static_cast<uint16_t>(v[d]);
            if (col + 2 * d + 1 < width) row[col + 2 * d + 1] = static_cast<uint16_t>(v[d] >> 16);
        }
    }
}

// Column q of an 8 x 8 patch (word d: rows 2d and 2d + 1), q known at compile time.
template <int Q>
__device__ __forceinline__ u32x4 patch_column(const u32x4 (&row)[8]) {
    constexpr uint32_t sel = Q & 1 ? 0x07060302u : 0x05040100u;
    u32x4 r;
#pragma unroll
    for (int d = 0; d < 4; ++d)
        r[d] = __builtin_amdgcn_perm(row[2 * d + 1][Q / 2], row[2 * d][Q / 2], sel);
    return r;
}

// The bf16 parts of a float32 value, the high one first: 8 bits of mantissa each,
// cut off and not rounded, so that none overflows, an integer's are integers, and
// all have its sign: their products with an infinity are the infinity that the
// value's is (a part of 0, of a short mantissa, makes NaN of it). Infinities and
// NaN are in every part.
constexpr int kBf16Parts = 3;
struct Parts3 {
    float p[kBf16Parts];
};
__device__ __forceinline__ Parts3 split3(float w) {
    if (!__builtin_isfinite(w)) return {{w, w, w}};
    auto cut = [](float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); };
    const float hi = cut(w), rest = w - hi, mid = cut(rest);
    return {{hi, mid, rest - mid}};
}

// ---- few rows ----------------------------------------------------------------

constexpr int kDirectCols = 512;  // columns of x per workgroup: 64 lanes x 8

// partial[split][m][r]: the workgroup's columns of u[m][r]; wave w takes ranks
// w, w + 4, ... Grid: (splits, rows).
template <bool VEC>
__global__ __launch_bounds__(kWgThreads) void direct_inner_kernel(
    const uint16_t* __restrict__ x, const int32_t* __restrict__ ids,
    const uint16_t* __restrict__ factor, int width, int rank, int count,
    float* __restrict__ partial) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m = blockIdx.y, col = blockIdx.x * kDirectCols + 8 * lane;
    const int a = ids[m];
    if (static_cast<uint32_t>(a) >= static_cast<uint32_t>(count)) return;
    const u32x4 xv = load8<VEC>(x + static_cast<size_t>(m) * width, col, width, true);
    const uint16_t* f = factor + static_cast<size_t>(a) * rank * width;
    float* out = partial + (static_cast<size_t>(blockIdx.x) * gridDim.y + m) * rank;
#pragma unroll 4
    for (int r = wave; r < rank; r += kWgWaves) {
        const u32x4 w = load8<VEC>(f + static_cast<size_t>(r) * width, col, width, true);
        float s = 0.f;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            s = fmaf(bf16_low(xv[d]), bf16_low(w[d]), s);
            s = fmaf(bf16_high(xv[d]), bf16_high(w[d]), s);
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
        if (lane == 0) out[r] = s;
    }
}

// y[m] = base[m] + s u[m] B over 512 columns: u[m] summed from the splits by 16
// lanes per rank (then a fixed tree), while the first rows of B are on their
// way; wave w multiplies ranks w, w + 4, ..., and the four waves' sums meet in
// LDS in wave order. The first workgroup of a row writes u. Grid: (column
// chunks, rows).
template <bool VEC>
__global__ __launch_bounds__(kWgThreads) void direct_expand_kernel(
    const float* __restrict__ partial, int splits, const int32_t* __restrict__ ids,
    const uint16_t* __restrict__ factor, const float* __restrict__ scales, int width, int rank,
    int count, const uint16_t* base, uint16_t* y, float* __restrict__ u) {
    __shared__ float us[kMaxRank];
    __shared__ float sums[kWgWaves][8][kWave];
    const int m = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, rows = gridDim.y;
    const int a = ids[m];
    const bool has = static_cast<uint32_t>(a) < static_cast<uint32_t>(count);
    const int col = blockIdx.x * kDirectCols + 8 * lane;
    const uint16_t* brow = (base ? base : y) + static_cast<size_t>(m) * width;
    uint16_t* yrow = y + static_cast<size_t>(m) * width;
    if (!has) {
        if (u && blockIdx.x == 0)
            for (int r = threadIdx.x; r < rank; r += kWgThreads) u[static_cast<size_t>(m) * rank + r] = 0.f;
        if (base != y && wave == 0)
            store8<VEC>(yrow, col, width, load8<VEC>(brow, col, width, base != nullptr));
        return;
    }
    const float scale = scales[a];
    const uint16_t* f = factor + static_cast<size_t>(a) * rank * width;
    u32x4 b = {0u, 0u, 0u, 0u};
    if (wave == 0) b = load8<VEC>(brow, col, width, base != nullptr);
    constexpr int kEarly = 4;
    u32x4 early[kEarly];
#pragma unroll
    for (int i = 0; i < kEarly; ++i) {
        const int r = wave + i * kWgWaves;
        early[i] = load8<VEC>(f + static_cast<size_t>(min(r, rank - 1)) * width, col, width, r < rank);
    }
    for (int i = threadIdx.x; i < 16 * rank; i += kWgThreads) {
        const int r = i / 16;
        float s = 0.f;
        for (int k = i % 16; k < splits; k += 16) s += partial[(static_cast<size_t>(k) * rows + m) * rank + r];
#pragma unroll
        for (int d = 8; d; d >>= 1) s += __shfl_xor(s, d);
        if (i % 16 == 0) {
            us[r] = s * scale;
            if (u && blockIdx.x == 0) u[static_cast<size_t>(m) * rank + r] = s;
        }
    }
    __syncthreads();
    float acc[8] = {};
    auto add = [&](int r, const u32x4& w) {
        const float ur = us[r];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            acc[2 * d] = fmaf(ur, bf16_low(w[d]), acc[2 * d]);
            acc[2 * d + 1] = fmaf(ur, bf16_high(w[d]), acc[2 * d + 1]);
        }
    };
#pragma unroll
    for (int i = 0; i < kEarly; ++i)
        if (wave + i * kWgWaves < rank) add(wave + i * kWgWaves, early[i]);
#pragma unroll 4
    for (int r = wave + kEarly * kWgWaves; r < rank; r += kWgWaves)
        add(r, load8<VEC>(f + static_cast<size_t>(r) * width, col, width, true));
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[wave][e][lane] = acc[e];
    __syncthreads();
    if (wave) return;
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        acc[e] = ((sums[0][e][lane] + sums[1][e][lane]) + sums[2][e][lane]) + sums[3][e][lane];
#pragma unroll
    for (int d = 0; d < 4; ++d)
        o[d] = pack_bf16(bf16_low(b[d]) + acc[2 * d], bf16_high(b[d]) + acc[2 * d + 1]);
    store8<VEC>(yrow, col, width, o);
}

// Both products in one launch: every workgroup computes the whole of its row's u
// (its 16 waves take a rank each at a time; the factor comes from the L2 for all
// but the row's first workgroup), then 1024 columns: 128 lanes of 8 columns, the
// ranks in eight parts that meet in LDS in order. The second factor's first
// ranks are on their way during the first product. Grid: (column chunks, rows).
constexpr int kOneThreads = 1024;
constexpr int kOneCols = 1024;
constexpr int kOneParts = kOneThreads / (kOneCols / 8);

template <bool VEC_IN, bool VEC_OUT>
__global__ __launch_bounds__(kOneThreads) void direct_kernel(
    const uint16_t* __restrict__ x, const int32_t* __restrict__ ids, const uint16_t* __restrict__ a,
    const uint16_t* __restrict__ b, const float* __restrict__ scales, int in, int out, int rank,
    int count, const uint16_t* base, uint16_t* y, float* __restrict__ u) {
    __shared__ float us[kMaxRank];
    __shared__ float sums[kOneParts][8][kOneCols / 8];
    const int m = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int id = ids[m];
    const bool has = static_cast<uint32_t>(id) < static_cast<uint32_t>(count);
    const int lc = tid % (kOneCols / 8), part = tid / (kOneCols / 8);
    const int col = blockIdx.x * kOneCols + 8 * lc;
    const uint16_t* brow = (base ? base : y) + static_cast<size_t>(m) * out;
    uint16_t* yrow = y + static_cast<size_t>(m) * out;
    if (!has) {
        if (u && blockIdx.x == 0)
            for (int r = tid; r < rank; r += kOneThreads) u[static_cast<size_t>(m) * rank + r] = 0.f;
        if (base != y && part == 0)
            store8<VEC_OUT>(yrow, col, out, load8<VEC_OUT>(brow, col, out, base != nullptr));
        return;
    }
    const float scale = scales[id];
    const uint16_t* fb = b + static_cast<size_t>(id) * rank * out;
    constexpr int kEarly = 2;
    u32x4 early[kEarly], bv = {0u, 0u, 0u, 0u};
    if (part == 0) bv = load8<VEC_OUT>(brow, col, out, base != nullptr);
#pragma unroll
    for (int i = 0; i < kEarly; ++i) {
        const int r = part + i * kOneParts;
        early[i] = load8<VEC_OUT>(fb + static_cast<size_t>(min(r, rank - 1)) * out, col, out, r < rank);
    }
    const uint16_t* xr = x + static_cast<size_t>(m) * in;
    for (int r = wave; r < rank; r += kOneThreads / kWave) {
        const uint16_t* fa = a + (static_cast<size_t>(id) * rank + r) * in;
        float s = 0.f;
#pragma unroll 8
        for (int k = 8 * lane; k < in; k += 8 * kWave) {
            const u32x4 xv = load8<VEC_IN>(xr, k, in, true), w = load8<VEC_IN>(fa, k, in, true);
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                s = fmaf(bf16_low(xv[d]), bf16_low(w[d]), s);
                s = fmaf(bf16_high(xv[d]), bf16_high(w[d]), s);
            }
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
        if (lane == 0) {
            us[r] = s * scale;
            if (u && blockIdx.x == 0) u[static_cast<size_t>(m) * rank + r] = s;
        }
    }
    __syncthreads();
    float acc[8] = {};
    auto add = [&](int r, const u32x4& w) {
        const float ur = us[r];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            acc[2 * d] = fmaf(ur, bf16_low(w[d]), acc[2 * d]);
            acc[2 * d + 1] = fmaf(ur, bf16_high(w[d]), acc[2 * d + 1]);
        }
    };
#pragma unroll
    for (int i = 0; i < kEarly; ++i)
        if (part + i * kOneParts < rank) add(part + i * kOneParts, early[i]);
#pragma unroll 4
    for (int r = part + kEarly * kOneParts; r < rank; r += kOneParts)
        add(r, load8<VEC_OUT>(fb + static_cast<size_t>(r) * out, col, out, true));
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[part][e][lc] = acc[e];
    __syncthreads();
    if (part) return;
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        acc[e] = sums[0][e][lc];
#pragma unroll
        for (int q = 1; q < kOneParts; ++q) acc[e] += sums[q][e][lc];
    }
#pragma unroll
    for (int d = 0; d < 4; ++d)
        o[d] = pack_bf16(bf16_low(bv[d]) + acc[2 * d], bf16_high(bv[d]) + acc[2 * d + 1]);
    store8<VEC_OUT>(yrow, col, out, o);
}

// The gradients of an adapter's factors over few rows: a workgroup takes 512
// columns and 4 ranks of one adapter, finds its rows (ascending), and its waves
// take them in turn: 4 ranks x 8 columns of float32 sums per lane. Of W waves,
// wave q adds wave q + W / 2's sums to its own, then the halves meet in order.
// `inner` are the float32 rank-long values without the scale. Grid: (column
// chunks of side a then of side b, adapters, 4 ranks each).
// 5120 -> 17408, 4 adapters, us: 16 ranks a workgroup 7.9 (32 rows at rank 16) and
// 19.1 (at rank 64), 8 ranks 6.7 and 15.6, 4 ranks 6.3 and 15.9 (two ranks 7.3 and
// 18.6); with 4 waves instead of 8 5.6 and 10.6. The rows come from the L2 again.
constexpr int kFewRows = 256;  // rows of a call, at most: a thread finds one
constexpr int kFewRanks = 4;

struct FewSide {
    const uint16_t* x;   // the wide rows
    const float* inner;  // [rows][rank]
    uint16_t* grad;
    int width, chunks;
    bool vec;
};

template <int WAVES, bool VEC>
__device__ __forceinline__ void add_rows(const FewSide& p, int col, int n, int wave,
                                         const int* __restrict__ list,
                                         const float (*__restrict__ coef)[kFewRanks],
                                         float (&acc)[kFewRanks][8]) {
#pragma unroll 4
    for (int i = wave; i < n; i += WAVES) {
        const u32x4 v = load8<VEC>(p.x + static_cast<size_t>(list[i]) * p.width, col, p.width, true);
        float e[8];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            e[2 * d] = bf16_low(v[d]);
            e[2 * d + 1] = bf16_high(v[d]);
        }
#pragma unroll
        for (int r = 0; r < kFewRanks; ++r)
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[r][q] = fmaf(coef[i][r], e[q], acc[r][q]);
    }
}

template <int THREADS, bool VEC>
__global__ __launch_bounds__(THREADS) void direct_outer_kernel(
    FewSide a, FewSide b, const int32_t* __restrict__ ids, const float* __restrict__ scales, int rows,
    int rank) {
    constexpr int waves = THREADS / kWave;
    union Shared {
        float coef[kFewRows][kFewRanks];
        float part[waves / 2][kFewRanks][8][kWave];
    };
    __shared__ Shared sh;
    __shared__ int list[kFewRows], found[waves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int id = blockIdx.y, r0 = blockIdx.z * kFewRanks;
    const bool second = static_cast<int>(blockIdx.x) >= a.chunks;
    const FewSide& p = second ? b : a;
    const int chunk = second ? blockIdx.x - a.chunks : blockIdx.x;
    const int col = chunk * kDirectCols + 8 * lane;
    const bool mine = tid < rows && ids[tid] == id;
    const uint64_t votes = __ballot(mine);
    if (lane == 0) found[wave] = __popcll(votes);
    __syncthreads();
    int before = 0, n = 0;
#pragma unroll
    for (int w = 0; w < waves; ++w) {
        if (w < wave) before += found[w];
        n += found[w];
    }
    if (mine) list[before + __popcll(votes & ((1ull << lane) - 1))] = tid;
    __syncthreads();
    const float scale = scales[id];
    for (int i = tid; i < n * kFewRanks; i += THREADS) {
        const int r = r0 + i % kFewRanks;
        sh.coef[i / kFewRanks][i % kFewRanks] =
            r < rank ? p.inner[static_cast<size_t>(list[i / kFewRanks]) * rank + r] * scale : 0.f;
    }
    __syncthreads();
    float acc[kFewRanks][8] = {};
    if (VEC || p.vec)
        add_rows<waves, true>(p, col, n, wave, list, sh.coef, acc);
    else
        add_rows<waves, false>(p, col, n, wave, list, sh.coef, acc);
    __syncthreads();  // the parts take the coefficients' place
    auto each = [&](auto&& f) {
#pragma unroll
        for (int r = 0; r < kFewRanks; ++r)
#pragma unroll
            for (int q = 0; q < 8; ++q) f(sh.part[wave % (waves / 2)][r][q][lane], acc[r][q]);
    };
    if (wave >= waves / 2) each([](float& o, float v) { o = v; });
    __syncthreads();
    if (wave < waves / 2) each([](float& o, float v) { o += v; });
    __syncthreads();
    for (int r = wave; r < kFewRanks && r0 + r < rank; r += waves) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            v[q] = sh.part[0][r][q][lane];
#pragma unroll
            for (int w = 1; w < waves / 2; ++w) v[q] += sh.part[w][r][q][lane];
        }
        u32x4 o;
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] = pack_bf16(v[2 * d], v[2 * d + 1]);
        uint16_t* row = p.grad + (static_cast<size_t>(id) * rank + r0 + r) * p.width;
        if (VEC || p.vec)
            store8<true>(row, col, p.width, o);
        else
            store8<false>(row, col, p.width, o);
    }
}

// ---- many rows ----------------------------------------------------------------

// partial[split][tile][64][16 R]: this split's columns of the tile's inner
// products. The four waves take the split's 64-column steps (a 128-byte line of
// each row) in turn and are summed in wave order. Grid: (splits, tiles).
template <int R, bool VEC>
__global__ __launch_bounds__(kWgThreads) void inner_kernel(
    const uint16_t* __restrict__ x, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ order, const uint16_t* __restrict__ factor, int rows, int width,
    int rank, int count, int split_cols, float* __restrict__ partial) {
    __shared__ float sum[kTileRows * 16 * R];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int j = lane & 15, c = lane >> 4;
    const Found at = find_entry(offsets, count, rows, kTileRows, blockIdx.y);
    if (at.group < 0) return;
    const int p0 = at.first + at.index * kTileRows;
    const uint16_t* xr[kSubs];
#pragma unroll
    for (int s = 0; s < kSubs; ++s)  // rows past the group's last read the last one again
        xr[s] = x + static_cast<size_t>(order[min(p0 + 16 * s + j, at.end - 1)]) * width;
    const uint16_t* f = factor + static_cast<size_t>(at.group) * rank * width;
    const uint16_t* fr[R];
#pragma unroll
    for (int s = 0; s < R; ++s) fr[s] = f + static_cast<size_t>(min(16 * s + j, rank - 1)) * width;
    floatx4 acc[kSubs][R] = {};
    const int k0 = blockIdx.x * split_cols, k1 = min(width, k0 + split_cols);
    struct Step {
        u32x4 x[2][kSubs], f[2][R];
    };
    auto load = [&](Step& q, int k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int s = 0; s < kSubs; ++s) q.x[h][s] = load8<VEC>(xr[s], k + 32 * h + 8 * c, k1, true);
#pragma unroll
            for (int r = 0; r < R; ++r) q.f[h][r] = load8<VEC>(fr[r], k + 32 * h + 8 * c, k1, true);
        }
    };
    auto multiply = [&](const Step& q) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 0; s < kSubs; ++s)
#pragma unroll
                for (int r = 0; r < R; ++r)
                    acc[s][r] = mfma16x16x32(as_bf16x8(q.x[h][s]), as_bf16x8(q.f[h][r]), acc[s][r]);
    };
    // up to two 16-rank operands the next step's loads are in flight while one
    // is multiplied (beyond, the registers hold one step)
    constexpr int step = 64 * kWgWaves;
    const int first = k0 + 64 * wave;
    if constexpr (R <= 2 && VEC) {
        Step q[2];
        if (first < k1) load(q[0], first);
        for (int k = first; k < k1; k += 2 * step) {
            if (k + step < k1) load(q[1], k + step);
            multiply(q[0]);
            if (k + step >= k1) break;
            if (k + 2 * step < k1) load(q[0], k + 2 * step);
            multiply(q[1]);
        }
    } else {
        for (int k = first; k < k1; k += step) {
            Step q;
            load(q, k);
            multiply(q);
        }
    }
    for (int w = 0; w < kWgWaves; ++w) {
        if (wave == w) {
#pragma unroll
            for (int s = 0; s < kSubs; ++s)
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float* o = sum + (16 * s + 4 * c + i) * (16 * R) + 16 * r + j;
                        *o = w ? *o + acc[s][r][i] : acc[s][r][i];
                    }
        }
        __syncthreads();
    }
    floatx4* out = reinterpret_cast<floatx4*>(
        partial + (static_cast<size_t>(blockIdx.x) * gridDim.y + blockIdx.y) * (kTileRows * 16 * R));
    for (int i = tid; i < kTileRows * 16 * R / 4; i += kWgThreads)
        out[i] = reinterpret_cast<const floatx4*>(sum)[i];
}

// What the later launches read of a tile.
struct TileInfo {
    int32_t group;  // its adapter; count: rows without one; -1: no tile
    int32_t rows;
};

// And of a segment of the outer sums: up to kSegRows rows of an adapter, which
// has one at least.
constexpr int kSegRows = kMaxSegTiles * kTileRows;
struct SegInfo {
    int32_t group;  // -1: no segment
    int32_t tile;   // its first
    int32_t rows;
    int32_t slot;   // of its float32 sums where the adapter has several; else -1
};
// And of an adapter of several.
struct SumInfo {
    int32_t group;  // -1: no adapter
    int32_t slot;   // of its first segment
    int32_t n;      // its segments
    int32_t unused;
};

// Segments of adapters of several are counted in the low bits, the adapters above:
// 2^20 rows make 2048 of the one and 1024 of the other at most.
constexpr int kOneSeveral = 1 << 12;

// The lists of `segments` segments and of `several` adapters of several segments
// (the last ones may be none), those of the adapters 64 b, 64 b + 1, ..., by one
// wave: a lane per adapter. Searched for by each
// workgroup of the outer sums it would cost 16 steps of a wave's sums for 1024
// adapters.
__device__ __forceinline__ void list_segments(const int32_t* __restrict__ offsets, int count, int rows,
                                              int b, int segments, SegInfo* __restrict__ segs, int several,
                                              SumInfo* __restrict__ sums) {
    const int lane = threadIdx.x & 63;
    auto group = [&](int g, int& n, int& tiles, int& shared) {
        int size = 0;
        n = tiles = shared = 0;
        if (g < count) {
            const int first = min(max(offsets[g], 0), rows);
            size = min(max(offsets[g + 1], first), rows) - first;
            n = max(1, (size + kSegRows - 1) / kSegRows);
            tiles = (size + kTileRows - 1) / kTileRows;
            shared = n > 1 ? n + kOneSeveral : 0;
        }
        return size;
    };
    int before = 0, tiles = 0, shared = 0;
    for (int c = 0; c < b; ++c) {
        int n, t, s;
        group(64 * c + lane, n, t, s);
        before += n;
        tiles += t;
        shared += s;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        before += __shfl_xor(before, d);
        tiles += __shfl_xor(tiles, d);
        shared += __shfl_xor(shared, d);
    }
    int n, t, s;
    const int g = 64 * b + lane, size = group(g, n, t, s);
    int end = n, tend = t, send = s;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int e = __shfl_up(end, d), te = __shfl_up(tend, d), se = __shfl_up(send, d);
        if (lane >= d) {
            end += e;
            tend += te;
            send += se;
        }
    }
    const int slot = (shared + send - s) % kOneSeveral, index = (shared + send - s) / kOneSeveral;
    for (int i = 0; i < n; ++i) {
        const int at = before + end - n + i;
        if (at < segments)
            segs[at] = {g, tiles + tend - t + i * kMaxSegTiles, min(size - i * kSegRows, kSegRows),
                        s ? slot + i : -1};
    }
    if (s && index < several) sums[index] = {g, slot, n, 0};
    if (64 * b + 64 >= count) {
        const int all = shared + __shfl(send, 63);
        for (int i = before + __shfl(end, 63) + lane; i < segments; i += 64) segs[i] = {-1, 0, 0, -1};
        for (int i = all / kOneSeveral + lane; i < several; i += 64) sums[i] = {-1, 0, 0, 0};
    }
}

// A tile's row numbers and group, its inner products summed from the splits
// (ascending), and their operand forms; a thread per row and rank.
//   by_row [tile][64][R][part][16]    (expand; scaled; half of the last part)
//   by_rank[tile][R][part][16][64]    (outer; scaled)
//   u_rank                            the same of the forward pass's u
// Rows past the tile's last and ranks past the last are zeros there. The first
// workgroups list the segments of the outer sums as well.
// Grid: (tiles, 4 r16): 16 rows x 16 ranks of the tile each, so that the rows of
// a rank are stored side by side.
__global__ __launch_bounds__(kWgThreads) void tile_kernel(
    const float* __restrict__ partial, int splits, int tiles, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ order, const float* __restrict__ scales, int rows, int rank, int r16,
    int count, TileInfo* __restrict__ info, int32_t* __restrict__ tile_rows,
    uint16_t* __restrict__ by_row, uint16_t* __restrict__ by_rank, float* __restrict__ u_out,
    const float* __restrict__ u_in, uint16_t* __restrict__ u_rank, SegInfo* __restrict__ segs,
    int segments, SumInfo* __restrict__ sums, int several) {
    if (segs && blockIdx.y == 0 && threadIdx.x < kWave)
        for (int b = blockIdx.x; 64 * b < count; b += gridDim.x)
            list_segments(offsets, count, rows, b, segments, segs, several, sums);
    const int t = blockIdx.x, ranks = 16 * r16;
    const int s = blockIdx.y / 4, rr = threadIdx.x % 16;
    const int row = 16 * (blockIdx.y % 4) + threadIdx.x / 16, r = 16 * s + rr;
    const Found at = find_entry(offsets, count + 1, rows, kTileRows, t);
    const int p0 = at.first + at.index * kTileRows;
    const int n = at.group < 0 ? 0 : min(kTileRows, at.end - p0);
    if (blockIdx.y == 0 && threadIdx.x == 0) info[t] = {at.group, n};
    if (at.group < 0) return;
    const int orig = row < n ? order[p0 + row] : -1;
    if (r == 0) tile_rows[t * kTileRows + row] = orig;
    const bool live = row < n && r < rank;
    const size_t u_at = static_cast<size_t>(max(orig, 0)) * rank + r;
    if (at.group == count) {
        if (u_out && live) u_out[u_at] = 0.f;
        return;
    }
    const float scale = scales[at.group];
    float v = 0.f;
    if (live) {
        const float* p = partial + static_cast<size_t>(t) * (kTileRows * ranks) + row * ranks + r;
        const size_t step = static_cast<size_t>(tiles) * (kTileRows * ranks);
#pragma unroll 8
        for (int k = 0; k < splits; ++k) v += p[k * step];
        if (u_out) u_out[u_at] = v;
    }
    const Parts3 w = split3(v * scale);
    uint16_t* q = by_row + ((static_cast<size_t>(t) * kTileRows + row) * r16 + s) * (16 * kBf16Parts) + rr;
#pragma unroll
    for (int part = 0; part < kBf16Parts; ++part)
        q[16 * part] = round_bf16(part == 2 ? 0.5f * w.p[part] : w.p[part]);
    if (!by_rank) return;
    const size_t rank_at = ((static_cast<size_t>(t) * r16 + s) * kBf16Parts * 16 + rr) * kTileRows + row;
    const Parts3 uw = split3(live ? u_in[u_at] * scale : 0.f);
#pragma unroll
    for (int part = 0; part < kBf16Parts; ++part) {
        by_rank[rank_at + part * 16 * kTileRows] = round_bf16(w.p[part]);
        u_rank[rank_at + part * 16 * kTileRows] = round_bf16(uw.p[part]);
    }
}

// The eight operands (column 8 j + q each) of 16 ranks of a factor's strip:
// lanes c and c + 2 hold the same ranks, which meet two parts.
template <bool VEC>
__device__ __forceinline__ void factor_operands(const uint16_t* f, int r, int rank, int col, int width,
                                                int c, u32x4 (&op)[8]) {
    u32x4 patch[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int rr = 16 * r + 8 * (c & 1) + i;
        patch[i] = load8<VEC>(f + static_cast<size_t>(min(rr, rank - 1)) * width, col, width, rr < rank);
    }
    static_for<0, 8>([&](auto qc) { op[decltype(qc)::value] = patch_column<decltype(qc)::value>(patch); });
}

// y[row] = base[row] + (scaled rank-long row) * factor. A wave takes 128 columns
// of a tile, 16 rows at a time; with R > 0 (r16 = R) the strip's operands stay
// in registers for all of them, else (R = 0) they are loaded again.
// Grid: (column chunks, tiles).
template <int R, bool VEC>
__global__ __launch_bounds__(kWgThreads) void expand_kernel(
    const TileInfo* __restrict__ info, const int32_t* __restrict__ tile_rows,
    const uint16_t* __restrict__ by_row, const uint16_t* __restrict__ factor, int width, int rank,
    int r16, int count, const uint16_t* base, uint16_t* y) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int j = lane & 15, c = lane >> 4;
    const int t = blockIdx.y;
    const TileInfo ti = info[t];
    const int col = (blockIdx.x * kWgWaves + wave) * kStrip + 8 * j;
    if (ti.group < 0 || col - 8 * j >= width) return;
    const int32_t* trow = tile_rows + t * kTileRows;
    if (ti.group == count) {  // rows without an adapter
        if (base == y) return;
        for (int i = c; i < ti.rows; i += 4) {
            const size_t at = static_cast<size_t>(trow[i]) * width;
            store8<VEC>(y + at, col, width, load8<VEC>((base ? base : y) + at, col, width, base != nullptr));
        }
        return;
    }
    const uint16_t* f = factor + static_cast<size_t>(ti.group) * rank * width;
    const uint16_t* rows_op = by_row + static_cast<size_t>(t) * kTileRows * r16 * (16 * kBf16Parts);
    // a row's number read from memory between the rows' loads would wait for
    // all of them: each lane holds one and passes it on
    const int my_row = trow[lane];
    u32x4 op[R ? R : 1][8];
#pragma unroll
    for (int r = 0; r < R; ++r) factor_operands<VEC>(f, r, rank, col, width, c, op[r]);
    static_for<0, kSubs>([&](auto sub) {
        constexpr int s = decltype(sub)::value;
        if (16 * s >= ti.rows) return;
        int row[4];
        u32x4 bv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) row[i] = __shfl(my_row, 16 * s + 4 * c + i);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            bv[i] = load8<VEC>((base ? base : y) + static_cast<size_t>(max(row[i], 0)) * width, col, width,
                               base && row[i] >= 0);
        const uint16_t* a_at = rows_op + static_cast<size_t>(16 * s + j) * r16 * (16 * kBf16Parts) + 8 * c;
        floatx4 acc[8] = {};
        // the third part fills its 32 slots as two halves, which the lower 32 lanes
        // load and pass to the upper ones
        auto multiply = [&](int r, const u32x4 (&f)[8]) {
            const uint16_t* at = a_at + 16 * kBf16Parts * r;
            const u32x4 two = *reinterpret_cast<const u32x4*>(at);
            u32x4 third = {0u, 0u, 0u, 0u};
            if (c < 2) third = *reinterpret_cast<const u32x4*>(at + 32);
#pragma unroll
            for (int d = 0; d < 4; ++d)
                third[d] = __builtin_amdgcn_permlane32_swap(third[d], third[d], false, false)[0];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                acc[q] = mfma16x16x32(as_bf16x8(two), as_bf16x8(f[q]), acc[q]);
                acc[q] = mfma16x16x32(as_bf16x8(third), as_bf16x8(f[q]), acc[q]);
            }
        };
        if constexpr (R > 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) multiply(r, op[r]);
        } else {
            for (int r = 0; r < r16; ++r) {
                factor_operands<VEC>(f, r, rank, col, width, c, op[0]);
                multiply(r, op[0]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (row[i] < 0) continue;
            u32x4 o;
#pragma unroll
            for (int d = 0; d < 4; ++d)
                o[d] = pack_bf16(bf16_low(bv[i][d]) + acc[2 * d][i], bf16_high(bv[i][d]) + acc[2 * d + 1][i]);
            store8<VEC>(y + static_cast<size_t>(row[i]) * width, col, width, o);
        }
    });
}

// One of the two sums over an adapter's rows of a rank-long column times a wide
// row: dA (g and x) or dB (scaled u and dy).
struct OuterSide {
    const uint16_t* x;        // the wide rows
    const uint16_t* by_rank;  // the rank-long values
    uint16_t* grad;           // [count][rank][width]
    float* sums;              // [shared segment][rank][width]
    int width, strips;
    bool vec;
};

// A segment of an adapter's tiles: its tiles go to the four waves in turn, and the
// sums of the waves that had any are added in wave order. An adapter of one segment (or without rows) is
// written to `grad` in bf16; the float32 sums of the others' segments go to
// `sums`.
template <int R, bool VEC>
__device__ __forceinline__ void outer_segment(const OuterSide& p, const SegInfo& seg, int strip, int r0,
                                              int r16, int rank, const int* seg_rows, float* sum) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int j = lane & 15, c = lane >> 4;
    const int width = p.width, col = strip * kStrip + 8 * j;
    const int n = (seg.rows + kTileRows - 1) / kTileRows, t0 = seg.tile;
    // This wave's 32-row halves of the segment's tiles wave, wave + 4, ...; the
    // next half's rows are loaded while one is multiplied.
    struct Half {
        u32x4 patch[8], a[R][kBf16Parts];
    };
    auto load = [&](Half& q, int step) {
        const int t = wave + kWgWaves * (step >> 1), h = step & 1;
        const int* trow = seg_rows + t * kTileRows + 32 * h + 8 * c;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q.patch[i] = load8<VEC>(p.x + static_cast<size_t>(max(trow[i], 0)) * width, col, width,
                                    trow[i] >= 0);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int part = 0; part < kBf16Parts; ++part)
                q.a[r][part] = *reinterpret_cast<const u32x4*>(
                    p.by_rank +
                    (((static_cast<size_t>(t0 + t) * r16 + r0 + r) * kBf16Parts + part) * 16 + j) * kTileRows +
                    32 * h + 8 * c);
    };
    floatx4 acc[R][8] = {};
    auto multiply = [&](const Half& q) {
        static_for<0, 8>([&](auto qc) {
            constexpr int e = decltype(qc)::value;
            const u32x4 b = patch_column<e>(q.patch);
#pragma unroll
            for (int part = 0; part < kBf16Parts; ++part)
#pragma unroll
                for (int r = 0; r < R; ++r)
                    acc[r][e] = mfma16x16x32(as_bf16x8(q.a[r][part]), as_bf16x8(b), acc[r][e]);
        });
    };
    const int steps = n > wave ? 2 * ((n - wave + kWgWaves - 1) / kWgWaves) : 0;
    Half q[2];
    if (steps) load(q[0], 0);
    for (int step = 0; step < steps; step += 2) {
        load(q[1], step + 1);
        multiply(q[0]);
        if (step + 2 < steps) load(q[0], step + 2);
        multiply(q[1]);
    }
    const int ways = min(n, kWgWaves);  // none: an adapter without rows
    for (int w = 0; w < ways; ++w) {
        if (wave == w) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float* o = sum + (16 * r + 4 * c + i) * kStrip + 8 * j;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = w ? o[e] + acc[r][e][i] : acc[r][e][i];
                }
        }
        __syncthreads();
    }
    // 8 columns per thread at a time
    for (int i = tid; i < 16 * R * kStrip / 8; i += kWgThreads) {
        const int r = 16 * r0 + i / (kStrip / 8), k = strip * kStrip + 8 * (i % (kStrip / 8));
        if (r >= rank || k >= width) continue;
        floatx4 v[2] = {};
        if (ways) {
            v[0] = *reinterpret_cast<const floatx4*>(sum + 8 * i);
            v[1] = *reinterpret_cast<const floatx4*>(sum + 8 * i + 4);
        }
        if (seg.slot >= 0) {
            float* o = p.sums + (static_cast<size_t>(seg.slot) * rank + r) * width + k;
            if constexpr (VEC) {
                *reinterpret_cast<floatx4*>(o) = v[0];
                *reinterpret_cast<floatx4*>(o + 4) = v[1];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (k + e < width) o[e] = v[e / 4][e % 4];
            }
        } else {
            const u32x4 o = {pack_bf16(v[0][0], v[0][1]), pack_bf16(v[0][2], v[0][3]),
                             pack_bf16(v[1][0], v[1][1]), pack_bf16(v[1][2], v[1][3])};
            store8<VEC>(p.grad + (static_cast<size_t>(seg.group) * rank + r) * width, k, width, o);
        }
    }
}

// Both sums in one launch. VEC: both sides' rows are whole 16-byte pieces. Without
// a list (no rows) every adapter is one segment of none.
// Grid: (strips of side a then of side b, segments, rank pairs).
template <int R, bool VEC>
__global__ __launch_bounds__(kWgThreads) void outer_kernel(
    OuterSide a, OuterSide b, const SegInfo* __restrict__ segs, const int32_t* __restrict__ tile_rows,
    int rank, int r16) {
    __shared__ __attribute__((aligned(16))) float sum[16 * R * kStrip];
    __shared__ int seg_rows[kSegRows];
    SegInfo seg = {static_cast<int>(blockIdx.y), 0, 0, -1};
    if (segs) seg = segs[blockIdx.y];
    if (seg.group < 0) return;
    const int n = (seg.rows + kTileRows - 1) / kTileRows * kTileRows;
    for (int i = threadIdx.x; i < n; i += kWgThreads)
        seg_rows[i] = tile_rows[static_cast<size_t>(seg.tile) * kTileRows + i];
    __syncthreads();
    const bool second = static_cast<int>(blockIdx.x) >= a.strips;
    const OuterSide& p = second ? b : a;
    const int strip = second ? blockIdx.x - a.strips : blockIdx.x, r0 = blockIdx.z * R;
    if (VEC || p.vec)
        outer_segment<R, true>(p, seg, strip, r0, r16, rank, seg_rows, sum);
    else
        outer_segment<R, false>(p, seg, strip, r0, r16, rank, seg_rows, sum);
}

// The segments' sums of the adapters of several, ascending, rounded to bf16, of
// both sides. Grid: (column chunks of side a then of side b, ranks, adapters of
// several segments at most).
__global__ __launch_bounds__(kWgThreads) void outer_sum_kernel(OuterSide a, OuterSide b, int chunks_a,
                                                               const SumInfo* __restrict__ sums, int rank) {
    const SumInfo info = sums[blockIdx.z];
    const int r = blockIdx.y;
    const bool second = static_cast<int>(blockIdx.x) >= chunks_a;
    const OuterSide& p = second ? b : a;
    const int k = (second ? blockIdx.x - chunks_a : blockIdx.x) * kWgThreads + threadIdx.x;
    if (info.group < 0 || k >= p.width) return;
    float v = 0.f;
#pragma unroll 4
    for (int q = 0; q < info.n; ++q)
        v += p.sums[(static_cast<size_t>(info.slot + q) * rank + r) * p.width + k];
    p.grad[(static_cast<size_t>(info.group) * rank + r) * p.width + k] = round_bf16(v);
}

// ---- plans and launches ---------------------------------------------------------

// Up to kDirectRanks ranks over all rows each row follows its own adapter: two
// launches, the factors read again by rows that share one. 5120 -> 17408, 32
// adapters, us (direct / tiles): rank 8, 300 rows 22 / 25; rank 16, 32 rows 11 /
// 20, 200 rows 22 / 24, 300 rows 30 / 26; rank 32, 100 rows 25 / 32; rank 64, 32
// rows 26 / 31, 64 rows 38 / 37, 100 rows 46 / 41.
constexpr int kDirectRanks = 4096;
constexpr int kDirectRows = 512;
bool direct_rows(int rows, int rank) {
    return rows <= kDirectRows && rows * rank <= kDirectRanks;
}
constexpr int kTargetGroups = 1024;  // workgroups that fill the compute units a few times

struct Plan {
    int r16, tiles;             // 16-rank operands; tiles at most
    int splits, split_cols;     // column splits of the inner products
    int segments;               // segments of the outer sums, at most
    int several, shared;        // adapters with several, and their segments, at most
    size_t offsets, order, counts, partial, info, tile_rows, segs, sums, by_row, by_rank, u_rank, sums_a, sums_b, bytes;
};

int inner_splits(int tiles, int width) {
    const int most = (width + 255) / 256;
    const int want = tiles ? (kTargetGroups + tiles - 1) / tiles : 1;
    const int n = want < most ? want : most;
    return n < 1 ? 1 : n > 32 ? 32 : n;
}

// Columns of one split: a multiple of 256 (a 64-column step per wave).
int split_columns(int width, int splits) {
    return ((width + splits - 1) / splits + 255) / 256 * 256;
}

Plan make_plan(int rows, int in, int out, int rank, int count, bool backward) {
    Plan p{};
    p.r16 = rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8;
    p.tiles = (rows + kTileRows - 1) / kTileRows + (count + 1 < rows ? count + 1 : rows);
    const int width = backward ? out : in;
    p.split_cols = split_columns(width, inner_splits(p.tiles, width));
    p.splits = (width + p.split_cols - 1) / p.split_cols;
    p.segments = count + rows / kSegRows;  // sum of max(1, ceil(n / kSegRows)), at most
    // n > kSegRows: ceil(n / kSegRows) <= 2 floor(n / kSegRows)
    p.several = rows > kSegRows ? rows / kSegRows : 0;
    p.shared = 2 * p.several;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const size_t tiles = p.tiles, ranks = 16 * static_cast<size_t>(p.r16);
    p.offsets = take((static_cast<size_t>(count) + 2) * 4);
    p.order = take(static_cast<size_t>(rows) * 4);
    p.counts = take(route_workspace_bytes(rows, count + 1));
    p.partial = take(p.splits * tiles * kTileRows * ranks * 4);
    p.info = take(tiles * sizeof(TileInfo));
    p.tile_rows = take(tiles * kTileRows * 4);
    const size_t parts = tiles * kTileRows * ranks * kBf16Parts * sizeof(uint16_t);
    p.by_row = take(parts);
    if (backward) {
        p.segs = take(p.segments * sizeof(SegInfo));
        p.sums = take(p.several * sizeof(SumInfo));
        p.by_rank = take(parts);
        p.u_rank = take(parts);
        p.sums_a = take(static_cast<size_t>(p.shared) * rank * in * 4);
        p.sums_b = take(static_cast<size_t>(p.shared) * rank * out * 4);
    }
    p.bytes = at;
    return p;
}

template <typename T>
T* at(void* ws, size_t offset) {
    return reinterpret_cast<T*>(static_cast<char*>(ws) + offset);
}

template <bool VEC>
hipError_t launch_inner(const Plan& p, const uint16_t* x, const uint16_t* factor, int rows, int width,
                        int rank, int count, void* ws, hipStream_t st) {
    auto kernel = p.r16 == 1   ? inner_kernel<1, VEC>
                  : p.r16 == 2 ? inner_kernel<2, VEC>
                  : p.r16 <= 4 ? inner_kernel<4, VEC>
                               : inner_kernel<8, VEC>;
    return launch_kernel(kernel, dim3(p.splits, p.tiles), dim3(kWgThreads), st, x,
                         at<int32_t>(ws, p.offsets), at<int32_t>(ws, p.order), factor, rows, width,
                         rank, count, p.split_cols, at<float>(ws, p.partial));
}

hipError_t launch_expand(const Plan& p, const uint16_t* factor, int width, int rank, int count,
                         const uint16_t* base, uint16_t* y, bool vec, void* ws, hipStream_t st) {
    const int chunk = kWgWaves * kStrip;
    auto kernel = p.r16 == 1   ? (vec ? expand_kernel<1, true> : expand_kernel<1, false>)
                  : p.r16 == 2 ? (vec ? expand_kernel<2, true> : expand_kernel<2, false>)
                               : (vec ? expand_kernel<0, true> : expand_kernel<0, false>);
    return launch_kernel(kernel,
                         dim3((width + chunk - 1) / chunk, p.tiles), dim3(kWgThreads), st,
                         at<TileInfo>(ws, p.info), at<int32_t>(ws, p.tile_rows),
                         at<uint16_t>(ws, p.by_row), factor, width, rank, p.r16, count, base, y);
}

template <int R>
hipError_t launch_outer_r(const Plan& p, const OuterSide& a, const OuterSide& b, int rows, int rank,
                          void* ws, hipStream_t st) {
    const hipError_t e = launch_kernel(
        a.vec && b.vec ? outer_kernel<R, true> : outer_kernel<R, false>,
        dim3(a.strips + b.strips, p.segments, (p.r16 + R - 1) / R), dim3(kWgThreads), st, a, b,
        rows ? at<SegInfo>(ws, p.segs) : nullptr, at<int32_t>(ws, p.tile_rows), rank, p.r16);
    if (e != hipSuccess || !p.several) return e;
    const int ca = (a.width + kWgThreads - 1) / kWgThreads, cb = (b.width + kWgThreads - 1) / kWgThreads;
    return launch_kernel(outer_sum_kernel, dim3(ca + cb, rank, p.several), dim3(kWgThreads), st, a, b,
                         ca, at<SumInfo>(ws, p.sums), rank);
}

// The gradient of few rows in three launches that follow each row (sorted tiles
// take six); with more adapters up to more ranks over all rows, as the tiles of
// each cost more. 5120 -> 17408, us (this / sorted tiles): 4 adapters, rank 16, 1
// row 13 / 26, 100 rows 21 / 30, 200 rows 29 / 33; rank 32, 100 rows 29 / 36, 200
// rows 44 / 40; one adapter, 200 rows, rank 16 31 / 32, rank 32 45 / 37; 32
// adapters, 250 rows, rank 32 78 / 81; 64, 200 rows, rank 64 185 / 238; 110, 256
// rows, rank 128 543 / 719.
constexpr int kBackwardRows = 256;
constexpr int kBackwardRanks = 4096, kRanksPerAdapter = 256;
static_assert(kBackwardRows <= kFewRows, "a thread finds a row");
bool direct_backward(int rows, int rank, int count) {
    return rows > 0 && rows <= kBackwardRows && rows * rank <= kBackwardRanks + kRanksPerAdapter * count;
}

// The few-row outer products with 4 waves a workgroup, where there are two
// workgroups or more per compute unit; with 8 where there are fewer and the rows
// of an adapter are shared by more waves. Us (4 waves / 8): 512 workgroups 5.3 / 5.9,
// 704 5.6 / 6.3 and 8.1 / 8.6, 2816 10.6 / 15.9; 352 7.5 / 7.0, 160 5.2 / 4.9, 88
// 14.6 / 10.0.
bool many_groups(const dim3& grid) {
    return static_cast<int64_t>(grid.x) * grid.y * grid.z >= 2 * cu_count();
}

// Few rows whose first factor is small enough for every workgroup of a row to
// read: one launch. 5120 -> 17408 at rank 16: 1 row 6.5 us against 8.5 in two
// launches, 8 rows 9.0 / 8.8 (and one launch less for the host to issue), 32
// rows 17.3 / 12.0; 17408 -> 5120, 1 row 12.4 / 8.2.
bool direct_in_one(int rows, int in, int rank) {
    return rows <= 8 && static_cast<int64_t>(in) * rank <= 1 << 17;
}

int direct_splits(int width) { return (width + kDirectCols - 1) / kDirectCols; }

}  // namespace

// The few-row gradient's workspace: the splits' inner products, then their sums.
size_t direct_partial_floats(int rows, int out, int rank) {
    return (static_cast<size_t>(direct_splits(out)) * rows * rank + 3) / 4 * 4;
}

size_t adapters_workspace_bytes(int rows, int in, int out, int rank, int count, bool backward) {
    if (!backward && direct_rows(rows, rank) && direct_in_one(rows, in, rank)) return 0;
    if (!backward && direct_rows(rows, rank))
        return static_cast<size_t>(direct_splits(in)) * rows * rank * sizeof(float);
    if (backward && direct_backward(rows, rank, count))
        return (direct_partial_floats(rows, out, rank) + static_cast<size_t>(rows) * rank) * sizeof(float);
    return make_plan(rows, in, out, rank, count, backward).bytes;
}

hipError_t launch_adapters(const uint16_t* x, const int32_t* ids, const AdapterFactors& f,
                           int rows, const uint16_t* base, uint16_t* y, float* u, bool vec_in,
                           bool vec_out, void* ws, hipStream_t st) {
    hipError_t e;
    if (rows == 0) return hipSuccess;
    if (direct_rows(rows, f.rank) && direct_in_one(rows, f.in, f.rank)) {
        auto kernel = vec_in ? (vec_out ? direct_kernel<true, true> : direct_kernel<true, false>)
                             : (vec_out ? direct_kernel<false, true> : direct_kernel<false, false>);
        return launch_kernel(kernel, dim3((f.out + kOneCols - 1) / kOneCols, rows), dim3(kOneThreads),
                             st, x, ids, f.a, f.b, f.scales, f.in, f.out, f.rank, f.count, base, y, u);
    }
    if (direct_rows(rows, f.rank)) {
        const int splits = direct_splits(f.in);
        e = launch_kernel(vec_in ? direct_inner_kernel<true> : direct_inner_kernel<false>,
                          dim3(splits, rows), dim3(kWgThreads), st, x, ids, f.a, f.in, f.rank,
                          f.count, static_cast<float*>(ws));
        if (e != hipSuccess) return e;
        return launch_kernel(vec_out ? direct_expand_kernel<true> : direct_expand_kernel<false>,
                             dim3(direct_splits(f.out), rows), dim3(kWgThreads), st,
                             static_cast<const float*>(ws), splits, ids, f.b, f.scales, f.out,
                             f.rank, f.count, base, y, u);
    }
    const Plan p = make_plan(rows, f.in, f.out, f.rank, f.count, false);
    if ((e = launch_route(ids, rows, f.count, true, at<int32_t>(ws, p.offsets),
                          at<int32_t>(ws, p.order), nullptr, at<int32_t>(ws, p.counts), st)))
        return e;
    if ((e = vec_in ? launch_inner<true>(p, x, f.a, rows, f.in, f.rank, f.count, ws, st)
                    : launch_inner<false>(p, x, f.a, rows, f.in, f.rank, f.count, ws, st)))
        return e;
    if ((e = launch_kernel(tile_kernel, dim3(p.tiles, 4 * p.r16), dim3(kWgThreads), st,
                           at<float>(ws, p.partial), p.splits, p.tiles, at<int32_t>(ws, p.offsets),
                           at<int32_t>(ws, p.order), f.scales, rows, f.rank, p.r16, f.count,
                           at<TileInfo>(ws, p.info), at<int32_t>(ws, p.tile_rows),
                           at<uint16_t>(ws, p.by_row), nullptr, u, nullptr, nullptr, nullptr, 0, nullptr, 0)))
        return e;
    return launch_expand(p, f.b, f.out, f.rank, f.count, base, y, vec_out, ws, st);
}

hipError_t launch_adapters_backward(const uint16_t* dy, const uint16_t* x, const float* u,
                                    const int32_t* ids, const AdapterFactors& f, int rows,
                                    const uint16_t* base, uint16_t* dx, uint16_t* da, uint16_t* db,
                                    bool vec_in, bool vec_out, void* ws, hipStream_t st) {
    hipError_t e;
    if (direct_backward(rows, f.rank, f.count)) {
        float* partial = static_cast<float*>(ws);
        float* inner = partial + direct_partial_floats(rows, f.out, f.rank);
        const int splits = direct_splits(f.out);
        e = launch_kernel(vec_out ? direct_inner_kernel<true> : direct_inner_kernel<false>,
                          dim3(splits, rows), dim3(kWgThreads), st, dy, ids, f.b, f.out, f.rank,
                          f.count, partial);
        if (e != hipSuccess) return e;
        e = launch_kernel(vec_in ? direct_expand_kernel<true> : direct_expand_kernel<false>,
                          dim3(direct_splits(f.in), rows), dim3(kWgThreads), st, partial, splits, ids,
                          f.a, f.scales, f.in, f.rank, f.count, base, dx, inner);
        if (e != hipSuccess) return e;
        const FewSide side_b{dy, u, db, f.out, direct_splits(f.out), vec_out};
        const FewSide side_a{x, inner, da, f.in, direct_splits(f.in), vec_in};
        const dim3 grid(side_b.chunks + side_a.chunks, f.count, (f.rank + kFewRanks - 1) / kFewRanks);
        const bool vec = vec_in && vec_out;
        if (many_groups(grid))
            return launch_kernel(vec ? direct_outer_kernel<256, true> : direct_outer_kernel<256, false>,
                                 grid, dim3(256), st, side_b, side_a, ids, f.scales, rows, f.rank);
        return launch_kernel(vec ? direct_outer_kernel<512, true> : direct_outer_kernel<512, false>,
                             grid, dim3(512), st, side_b, side_a, ids, f.scales, rows, f.rank);
    }
    const Plan p = make_plan(rows, f.in, f.out, f.rank, f.count, true);
    if ((e = launch_route(ids, rows, f.count, true, at<int32_t>(ws, p.offsets),
                          at<int32_t>(ws, p.order), nullptr, at<int32_t>(ws, p.counts), st)))
        return e;
    // without rows the outer sums write zeros, and nothing else is left to do
    if (rows && (e = vec_out ? launch_inner<true>(p, dy, f.b, rows, f.out, f.rank, f.count, ws, st)
                             : launch_inner<false>(p, dy, f.b, rows, f.out, f.rank, f.count, ws, st)))
        return e;
    if (rows && (e = launch_kernel(tile_kernel, dim3(p.tiles, 4 * p.r16), dim3(kWgThreads), st,
                           at<float>(ws, p.partial), p.splits, p.tiles, at<int32_t>(ws, p.offsets),
                           at<int32_t>(ws, p.order), f.scales, rows, f.rank, p.r16, f.count,
                           at<TileInfo>(ws, p.info), at<int32_t>(ws, p.tile_rows),
                           at<uint16_t>(ws, p.by_row), at<uint16_t>(ws, p.by_rank), nullptr, u,
                           at<uint16_t>(ws, p.u_rank), at<SegInfo>(ws, p.segs), p.segments, at<SumInfo>(ws, p.sums),
                           p.several)))
        return e;
    auto strips = [](int width) { return (width + kStrip - 1) / kStrip; };
    const OuterSide side_b{dy, at<uint16_t>(ws, p.u_rank), db, at<float>(ws, p.sums_b), f.out,
                           strips(f.out), vec_out};
    const OuterSide side_a{x, at<uint16_t>(ws, p.by_rank), da, at<float>(ws, p.sums_a), f.in,
                           strips(f.in), vec_in};
    if ((e = p.r16 == 1 ? launch_outer_r<1>(p, side_b, side_a, rows, f.rank, ws, st)
                        : launch_outer_r<2>(p, side_b, side_a, rows, f.rank, ws, st)))
        return e;
    if (rows == 0) return hipSuccess;
    return launch_expand(p, f.a, f.in, f.rank, f.count, base, dx, vec_in, ws, st);
}

}  // namespace trellis
