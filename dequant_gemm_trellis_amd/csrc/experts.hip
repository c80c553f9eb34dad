// The experts' coded products (trellis_experts): rows sorted by expert, each
// multiplied with its expert's trellis-coded matrix, on either axis.
//
// Every weight is decoded through a random read of the codebook in LDS, as in
// the single projections, and those reads bound a product until a decoded
// weight serves enough rows to keep the matrix cores busy. So a wave decodes
// the operands of a strip of output columns in registers, for a tile of up to
// 16 MT rows of one expert, and multiplies each at once with the tile's MT
// 16-row operands of x.
//   axis 1 (stored row = output column): as the prefill's fragments: lane (j, c)
//     of a wave holds weights [64c, 64c + 64) of a block of stored row j of a
//     16-row group; step S of a block is 8 of them per lane.
//   axis 0 (stored row = input): as the scatter's patches: lane (j, c) decodes 8
//     stored rows x 4 or 8 adjacent columns.
// For tiles of several operands x is first laid out in operand order
// (operands_kernel), so that a wave reads an operand as 1 KB in a row.
// The decode table (pair table for k = 2, else eight bank-partitioned copies of
// the codebook) is staged once per workgroup, which stays for all its work.
// Few rows per expert: a workgroup takes a strip of one tile and its waves
// share the contraction (their sums meet in LDS in wave order). Many: every
// wave takes strips of its own, and no wave waits for another (x through LDS, a
// barrier per step, measured 278 us where this takes 214; one wave per SIMD with
// 128 x 112 accumulators 289).
//
// 64 experts, MI355X: 256 rows of 2048 -> 1536, k = 3: 48 us, 65% of the codebook
// reads' rate; 16384 rows, k = 2: 174 us (34 of it for the order), 580 TFLOP/s,
// 45% of a large library product's rate; 1536 -> 2048 on axis 0, k = 4: 227 us,
// 446 TFLOP/s.
#include "common.hpp"
#include "experts.hpp"
#include "groups.hpp"
#include "launch.hpp"

namespace trellis {
namespace {

constexpr int kStripCols = 128;
constexpr int kXcds = 8;  // accelerator dies, each with its own L2

// Tiles that ascending offsets make at most; the workspace and the unit numbers
// are made for them.
__host__ __device__ __forceinline__ int tiles_at_most(int rows, int experts, int per) {
    return rows / per + (experts < rows ? experts : rows);
}

// Tiles of `per` rows that the experts' rows make (no more than that).
__device__ __forceinline__ int count_tiles(const int32_t* __restrict__ offsets, int experts, int rows,
                                           int per) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int g = lane; g < experts; g += 64) {
        const int first = min(max(offsets[g], 0), rows);
        n += (min(max(offsets[g + 1], first), rows) - first + per - 1) / per;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) n += __shfl_xor(n, d);
    return min(__builtin_amdgcn_readfirstlane(n), tiles_at_most(rows, experts, per));
}

// Where the units of a launch are: `units` of them, this workgroup's (or
// wave's) every `step`-th from `first` on below `end`. Each XCD takes a
// contiguous range, so that strips of one tile share its rows in one L2.
struct Range {
    int first, end, step;
};
__device__ __forceinline__ Range xcd_range(int units, int per_group, int index) {
    const int dies = min(kXcds, static_cast<int>(gridDim.x));
    const int xcd = blockIdx.x % dies, slot = blockIdx.x / dies;
    const int groups = (gridDim.x - xcd + dies - 1) / dies;
    const int u0 = static_cast<int>(static_cast<int64_t>(units) * xcd / dies);
    const int u1 = static_cast<int>(static_cast<int64_t>(units) * (xcd + 1) / dies);
    return {u0 + slot * per_group + index, u1, groups * per_group};
}

struct ExArgs {
    const uint16_t* x;        // rows, or operand order (tiles of several operands)
    const int32_t* offsets;
    const uint32_t* codes;
    const float* scales;
    const float* lut;
    CodeLayout lay;
    uint64_t words;           // code words per expert
    int experts, rows, in, out;
    uint16_t* y;
};

// x of a tile in operand order, [tile][step][MT] operands of 64 lanes x 16 bytes;
// rows past the tile's last are zeros. A wave's load of an operand is then 1 KB
// in a row; taken from the rows it is 16 pieces of 64 bytes on axis 0 (16384 rows
// of 1536 -> 2048, k = 4: 343 us, against 214 with this order and 27 for making
// it) or 64 of 16 bytes on axis 1. Grid: (tiles, 256 contracted values).
template <int MT, int AXIS, bool VEC>
__global__ __launch_bounds__(256) void operands_kernel(const uint16_t* __restrict__ x,
                                                       const int32_t* __restrict__ offsets,
                                                       int experts, int rows, int in,
                                                       u32x4* __restrict__ out) {
    const Found at = find_entry(offsets, experts, rows, 16 * MT, blockIdx.x);
    if (at.group < 0) return;
    const int row0 = at.first + at.index * 16 * MT;
    const int lane = threadIdx.x & 63, j = lane & 15, c = lane >> 4;
    const int steps = (in + 31) / 32, s0 = 8 * blockIdx.y, n = min(8, steps - s0);
    u32x4* o = out + (static_cast<size_t>(blockIdx.x) * steps + s0) * MT * 64 + lane;
    // the reads of a lane (axis 1) or of a lane group (axis 0) come from one line
    for (int m = threadIdx.x >> 6; m < MT; m += 4) {
        const int row = row0 + 16 * m + j;
        const uint16_t* p = x + static_cast<size_t>(min(row, at.end - 1)) * in;
        u32x4 v[8] = {};
        if constexpr (AXIS == 1) {  // step s of a block is weights 64 c + 8 s
            if (row < at.end) {
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    v[s] = *reinterpret_cast<const u32x4*>(p + 256 * blockIdx.y + 64 * c + 8 * s);
            }
        } else {  // 32 rows in a row, the last step's the last 32
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int step = min(s0 + s, steps - 1), first = min(32 * step, in - 32) + 8 * c;
                v[s] = load8<VEC>(p, first, in, row < at.end);
#pragma unroll
                for (int d = 0; d < 4; ++d) {  // values already counted
                    if (first + 2 * d < 32 * step) v[s][d] &= 0xFFFF0000u;
                    if (first + 2 * d + 1 < 32 * step) v[s][d] &= 0x0000FFFFu;
                }
            }
        }
#pragma unroll
        for (int s = 0; s < 8; ++s)
            if (AXIS == 1 || s < n) o[(s * MT + m) * 64] = v[s];
    }
}

constexpr int kWideCols = 64;  // columns of a wave's strip in a tile of several operands

// Axis 1, tiles of MT x 16 rows: a wave takes four 16-column groups of a tile.
template <int K, int MT>
__global__ __launch_bounds__(kExThreads) void experts1_kernel(ExArgs p) {
    constexpr int G = kWideCols / 16;
    constexpr bool pair = ExTable<K>::pair, rep = ExTable<K>::rep;
    __shared__ __attribute__((aligned(16))) float tab[ExTable<K>::Table::floats];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, c = lane >> 4;
    stage_table<K>(tab, p.lut);
    const int nb = p.in / kT, strips = (p.out + kWideCols - 1) / kWideCols;
    const int tiles = count_tiles(p.offsets, p.experts, p.rows, 16 * MT);
    const Range r = xcd_range(tiles * strips, kExWaves, wave);
    for (int u = r.first; u < r.end; u += r.step) {
        const int t = u / strips, n0 = (u - t * strips) * kWideCols;
        const Found at = find_entry(p.offsets, p.experts, p.rows, 16 * MT, t);
        const int row0 = at.first + at.index * 16 * MT;
        const uint32_t* codes = p.codes + at.group * p.words;
        const float* scales = p.scales + static_cast<size_t>(at.group) * p.out;
        int rowc[G];
        float sc[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            rowc[g] = min(n0 + 16 * g + j, p.out - 1);
            sc[g] = scales[rowc[g]];
        }
        const u32x4* xo = reinterpret_cast<const u32x4*>(p.x) + static_cast<size_t>(t) * nb * 8 * MT * 64 + lane;
        floatx4 acc[G][MT] = {};
        for (int b = 0; b < nb; ++b) {
            uint32_t w[G][2 * K + 1];
#pragma unroll
            for (int g = 0; g < G; ++g)
                load_run64<K>(codes + block_word<K>(p.lay, rowc[g], b), 3 - c, w[g]);
            // fragment i is step i / G of group i % G; its values are read one
            // fragment ahead
            u32x4 a[MT];
            Gathered<pair> v[2];
            v[0] = gather_tab<K, 0, pair, rep>(w[0], tab);
            static_for<0, 8 * G>([&](auto ic) {
                constexpr int i = decltype(ic)::value, S = i / G, g = i % G, n = i + 1;
                if constexpr (g == 0) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        a[m] = xo[(static_cast<size_t>(8 * b + S) * MT + m) * 64];
                }
                __builtin_amdgcn_s_setprio(2);
                if constexpr (n < 8 * G) v[n & 1] = gather_tab<K, n / G, pair, rep>(w[n % G], tab);
                __builtin_amdgcn_s_setprio(0);
                const u32x4 f = pack_fragment(v[i & 1], sc[g]);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    acc[g][m] = mfma16x16x32(as_bf16x8(a[m]), as_bf16x8(f), acc[g][m]);
            });
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int n = n0 + 16 * g + j;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = row0 + 16 * m + 4 * c + i;
                    if (row < at.end && n < p.out)
                        p.y[static_cast<size_t>(row) * p.out + n] = round_bf16(acc[g][m][i]);
                }
        }
    }
}

// ---- few rows per expert: a workgroup's waves share a strip's contraction ---------

// Partial sums of up to four waves, [part][16][128]; the columns of a row are
// swizzled by its lane group, so that the 64 lanes of a store hit all banks.
constexpr int kParts = 4;
constexpr int kPartFloats = 16 * kStripCols;
__device__ __forceinline__ int part_at(int row, int col) {
    return row * kStripCols + (col ^ (16 * (row >> 2)));
}

// The sums of a tile's strip from the waves' parts, in a fixed order: wave q
// adds wave q + 4's part to its own, then the four meet, part 0 first. WAYS
// waves (1, 2, 4 or 8) share each column; way `q` of them is this wave's, its
// values given by each(f): f(row, column, value). Every wave of the workgroup
// calls it; a strip of columns [col0, col0 + 128) of rows [row0, end).
template <int WAYS, typename F>
__device__ __forceinline__ void sum_strip(float* parts, int q, F&& each, uint16_t* __restrict__ y,
                                          int row0, int end, int col0, int out) {
    __syncthreads();  // the parts of the strip before are read
    if (WAYS > kParts) {
        if (q >= kParts)
            each([&](int row, int col, float v) { parts[(q - kParts) * kPartFloats + part_at(row, col)] = v; });
        __syncthreads();
        if (q < kParts)
            each([&](int row, int col, float v) { parts[q * kPartFloats + part_at(row, col)] += v; });
    } else {
        each([&](int row, int col, float v) { parts[q * kPartFloats + part_at(row, col)] = v; });
    }
    __syncthreads();
    constexpr int n = WAYS < kParts ? WAYS : kParts;
    const int row = threadIdx.x / (kStripCols / 4), c4 = 4 * (threadIdx.x % (kStripCols / 4));
    if (row0 + row >= end) return;
    floatx4 v = {};
#pragma unroll
    for (int k = 0; k < n; ++k) v += *reinterpret_cast<const floatx4*>(parts + k * kPartFloats + part_at(row, c4));
    uint16_t* o = y + static_cast<size_t>(row0 + row) * out + col0 + c4;
    const uint32_t lo = pack_bf16(v[0], v[1]), hi = pack_bf16(v[2], v[3]);
    if (out % 4 == 0) {
        if (col0 + c4 < out) *reinterpret_cast<uint2*>(o) = uint2{lo, hi};
    } else {
        if (col0 + c4 < out) o[0] = static_cast<uint16_t>(lo);
        if (col0 + c4 + 1 < out) o[1] = static_cast<uint16_t>(lo >> 16);
        if (col0 + c4 + 2 < out) o[2] = static_cast<uint16_t>(hi);
        if (col0 + c4 + 3 < out) o[3] = static_cast<uint16_t>(hi >> 16);
    }
}
static_assert(kExThreads == 16 * kStripCols / 4, "a thread sums four columns of a row");

// A strip of a tile of 16 rows.
struct Unit {
    int group, row0, end, col0;
};
__device__ __forceinline__ Unit unit_at(const ExArgs& p, int u, int strips) {
    const int t = u / strips;
    const Found at = find_entry(p.offsets, p.experts, p.rows, 16, t);
    return {at.group, at.first + 16 * at.index, at.end, (u - t * strips) * kStripCols};
}

// A wave's work over its strips: pieces (a block or a 32-row step) from `first`
// on, every `stride`-th below `pieces` of every strip of `r`. load(work, unit,
// piece) of the next piece is in flight while multiply(work) runs;
// finish(unit) follows a strip's last piece.
template <typename Work, typename Load, typename Between, typename Multiply, typename Finish>
__device__ __forceinline__ void run_units(const ExArgs& p, const Range& r, int strips, int first,
                                          int stride, int pieces, Load&& load, Between&& between,
                                          Multiply&& multiply, Finish&& finish) {
    int u = r.first, piece = first;
    Unit unit = {};
    Work q[2];
    if (u < r.end) {
        unit = unit_at(p, u, strips);
        if (piece < pieces) load(q[0], unit, piece);
    }
    between();
    auto one = [&](Work& now, Work& next) {
        int nu = u, np = piece + stride;
        Unit nunit = unit;
        if (np >= pieces) {
            np = first;
            nu = u + r.step;
            if (nu < r.end) nunit = unit_at(p, nu, strips);
        }
        if (nu < r.end && np < pieces) load(next, nunit, np);
        if (piece < pieces) multiply(now);
        if (nu != u) finish(unit);
        u = nu;
        piece = np;
        unit = nunit;
    };
    while (u < r.end) {
        one(q[0], q[1]);
        if (u < r.end) one(q[1], q[0]);
    }
}

// Axis 1: the waves are G ways along the contraction (a block each at a time)
// and 8 / G along the columns, G 16-column groups each.
template <int K, int G>
__global__ __launch_bounds__(kExThreads) void experts1_few_kernel(ExArgs p) {
    constexpr bool pair = ExTable<K>::pair, rep = ExTable<K>::rep;
    __shared__ __attribute__((aligned(16))) float tab[ExTable<K>::Table::floats];
    __shared__ __attribute__((aligned(16))) float parts[kParts * kPartFloats];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, c = lane >> 4;
    const int kw = wave % G, first = (wave / G) * 16 * G;  // this wave's way and its columns
    const int nb = p.in / kT, strips = (p.out + kStripCols - 1) / kStripCols;
    const int tiles = count_tiles(p.offsets, p.experts, p.rows, 16);
    struct Work {
        uint32_t w[G][2 * K + 1];
        float sc[G];
        u32x4 a[8];
    };
    floatx4 acc[G] = {};
    run_units<Work>(
        p, xcd_range(tiles * strips, 1, 0), strips, kw, G, nb,
        [&](Work& q, const Unit& un, int b) {
            const uint32_t* codes = p.codes + un.group * p.words;
            const float* scales = p.scales + static_cast<size_t>(un.group) * p.out;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int row = min(un.col0 + first + 16 * g + j, p.out - 1);
                load_run64<K>(codes + block_word<K>(p.lay, row, b), 3 - c, q.w[g]);
                q.sc[g] = scales[row];
            }
            const uint16_t* x = p.x + static_cast<size_t>(min(un.row0 + j, un.end - 1)) * p.in +
                                static_cast<size_t>(b) * kT + 64 * c;
#pragma unroll
            for (int s = 0; s < 8; ++s) q.a[s] = *reinterpret_cast<const u32x4*>(x + 8 * s);
        },
        [&] { stage_table<K>(tab, p.lut); },
        [&](const Work& q) {
            // fragment i is step i / G of group i % G; its values are read one
            // fragment ahead
            Gathered<pair> v[2];
            v[0] = gather_tab<K, 0, pair, rep>(q.w[0], tab);
            static_for<0, 8 * G>([&](auto ic) {
                constexpr int i = decltype(ic)::value, S = i / G, g = i % G, n = i + 1;
                __builtin_amdgcn_s_setprio(2);
                if constexpr (n < 8 * G) v[n & 1] = gather_tab<K, n / G, pair, rep>(q.w[n % G], tab);
                __builtin_amdgcn_s_setprio(0);
                acc[g] = mfma16x16x32(as_bf16x8(q.a[S]), as_bf16x8(pack_fragment(v[i & 1], q.sc[g])),
                                      acc[g]);
            });
        },
        [&](const Unit& un) {
            sum_strip<G>(parts, kw, [&](auto&& f) {
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) f(4 * c + i, first + 16 * g + j, acc[g][i]);
            }, p.y, un.row0, un.end, un.col0, p.out);
#pragma unroll
            for (int g = 0; g < G; ++g) acc[g] = floatx4{};
        });
}

// ---- axis 0 ---------------------------------------------------------------------

template <int K, int CL>
__device__ __forceinline__ Strip0 expert_strip(const ExArgs& p, int expert, int col0, int j, int c) {
    return strip0<K, CL>(p.codes + expert * p.words, p.scales + static_cast<size_t>(expert) * p.in, p.lay,
                         col0, j, c);
}

// x operand of 16 rows from row0 on (rows past `end` read the last), step `step`.
template <bool VEC>
__device__ __forceinline__ u32x4 x_operand(const ExArgs& p, int row0, int end, int step, int j, int c) {
    const int row = min(row0 + j, end - 1);
    return load8<VEC>(p.x + static_cast<size_t>(row) * p.in, 32 * step + 8 * c, p.in, true);
}

// Tiles of MT x 16 rows: a wave takes 64 columns of a tile, 4 per lane. A last
// step of fewer than 32 rows takes the last 32 stored rows again, with zeros in
// the x operands (operands_kernel) and scales of zero for those already counted:
// an infinite weight times a zero would be NaN; in >= 32. TAIL: in is no multiple
// of 32 (an instance of its own: the step's code behind the loop costs whole steps
// 7% at k = 2 and 128 rows).
template <int K, int MT, bool TAIL>
__global__ __launch_bounds__(kExThreads) void experts0_kernel(ExArgs p) {
    constexpr int CL = 4;
    using Ps = Pieces<K, CL>;
    __shared__ __attribute__((aligned(16))) float tab[ExTable<K>::Table::floats];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, c = lane >> 4;
    stage_table<K>(tab, p.lut);
    const int steps = (p.in + 31) / 32, strips = p.out / kWideCols;
    const int tiles = count_tiles(p.offsets, p.experts, p.rows, 16 * MT);
    const Range r = xcd_range(tiles * strips, kExWaves, wave);
    for (int u = r.first; u < r.end; u += r.step) {
        const int t = u / strips, col0 = (u - t * strips) * kWideCols;
        const Found at = find_entry(p.offsets, p.experts, p.rows, 16 * MT, t);
        const int row0 = at.first + at.index * 16 * MT;
        const Strip0 s = expert_strip<K, CL>(p, at.group, col0, j, c);
        auto first_row = [&](int step) { return min(32 * step, p.in - 32); };
        const u32x4* xo = reinterpret_cast<const u32x4*>(p.x) + static_cast<size_t>(t) * steps * MT * kWave;
        auto load_x = [&](int step, int m) {
            return load_at<u32x4>(xo + (static_cast<size_t>(min(step, steps - 1)) * MT + m) * kWave, 16 * lane);
        };
        auto load_sc = [&](float (&q)[8], int step) {
            const float* at_row = s.scales + first_row(step);
            const floatx4 lo = load_at<floatx4_a4>(at_row, 32 * c), hi = load_at<floatx4_a4>(at_row + 4, 32 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                q[i] = lo[i];
                q[4 + i] = hi[i];
            }
        };
        Words q;
        float sc[8], next_sc[8];
        u32x4 x[MT];
        load_sc(sc, 0);
        load_words(q, s, 0);
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = load_x(0, m);
        floatx4 acc[CL][MT] = {};
        auto one = [&](int step) {
            Ps ps;
            ps.set(q, s.sh);
            // the scales first: they are moved at the step's end, and a move
            // waits for everything loaded before
            load_sc(next_sc, step + 1);
            load_words(q, s, first_row(step + 1));
            ps.each(sc, tab, [&](auto ec, const u32x4& f) {
                constexpr int e = decltype(ec)::value;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    acc[e][m] = mfma16x16x32(as_bf16x8(x[m]), as_bf16x8(f), acc[e][m]);
                    if constexpr (e == CL - 1) x[m] = load_x(step + 1, m);
                }
            });
#pragma unroll
            for (int i = 0; i < 8; ++i) sc[i] = next_sc[i];
        };
        const int whole = TAIL ? p.in / 32 : steps;
        for (int step = 0; step < whole; ++step) one(step);
        if constexpr (TAIL) {  // none for the rows already counted
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (p.in - 32 + 8 * c + i < 32 * whole) sc[i] = 0.f;
            one(whole);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = row0 + 16 * m + 4 * c + i;
                if (row >= at.end) continue;
                *reinterpret_cast<uint2*>(p.y + static_cast<size_t>(row) * p.out + col0 + CL * j) =
                    uint2{pack_bf16(acc[0][m][i], acc[1][m][i]), pack_bf16(acc[2][m][i], acc[3][m][i])};
            }
    }
}

template <int K, bool VEC>
__global__ __launch_bounds__(kExThreads) void experts0_few_kernel(ExArgs p) {
    constexpr int CL = 8;
    __shared__ __attribute__((aligned(16))) float tab[ExTable<K>::Table::floats];
    __shared__ __attribute__((aligned(16))) float parts[kParts * kPartFloats];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, c = lane >> 4;
    const int steps = (p.in + 31) / 32, strips = p.out / kStripCols;
    const int tiles = count_tiles(p.offsets, p.experts, p.rows, 16);
    struct Work {
        Words q;
        float sc[8];
        u32x4 x;
        int sh;
    };
    floatx4 acc[CL] = {};
    run_units<Work>(
        p, xcd_range(tiles * strips, 1, 0), strips, wave, kExWaves, steps,
        [&](Work& q, const Unit& un, int step) {
            const Strip0 s = expert_strip<K, CL>(p, un.group, un.col0, j, c);
            q.x = x_operand<VEC>(p, un.row0, un.end, step, j, c);
            q.sh = s.sh;
            if (32 * step + 32 <= p.in) {
                load_words(q.q, s, 32 * step);
                const floatx4 lo = load_at<floatx4_a4>(s.scales + 32 * step, 32 * c);
                const floatx4 hi = load_at<floatx4_a4>(s.scales + 32 * step + 4, 32 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    q.sc[i] = lo[i];
                    q.sc[4 + i] = hi[i];
                }
                return;
            }
            // the last rows, one by one; past the end x is zero, and so is the
            // scale: an infinite weight times a zero would be NaN
            const uint32_t row = static_cast<uint32_t>(32 * c * s.row_words);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int past = 32 * step + 8 * c + i, r = min(past, p.in - 1);
                const uint32_t* w = s.codes + static_cast<uint64_t>(r) * s.row_words;
                q.q.a[i] = w[(s.at_a - row) / 4];
                q.q.b[i] = w[(s.at_b - row) / 4];
                q.sc[i] = past < p.in ? s.scales[r] : 0.f;
            }
        },
        [&] { stage_table<K>(tab, p.lut); },
        [&](const Work& q) {
            Pieces<K, CL> ps;
            ps.set(q.q, q.sh);
            ps.each(q.sc, tab, [&](auto ec, const u32x4& f) {
                constexpr int e = decltype(ec)::value;
                acc[e] = mfma16x16x32(as_bf16x8(q.x), as_bf16x8(f), acc[e]);
            });
        },
        [&](const Unit& un) {
            sum_strip<kExWaves>(parts, wave, [&](auto&& f) {
#pragma unroll
                for (int e = 0; e < CL; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) f(4 * c + i, CL * j + e, acc[e][i]);
            }, p.y, un.row0, un.end, un.col0, p.out);
#pragma unroll
            for (int e = 0; e < CL; ++e) acc[e] = floatx4{};
        });
}

// ---- launches ---------------------------------------------------------------------

// The tiles of a call: strips of 16 rows shared by a workgroup's waves, or tiles
// of 2, 4 or 8 operands of which every wave takes strips of its own.
enum class Tile { few, two, four, eight };
constexpr int kOperands[] = {1, 2, 4, 8};

// The tile with the least estimated time. The host does not know how the rows
// fall: it takes rows / (rows of a tile) tiles plus 0.6 of an expert's last, at
// least one per expert. All units of a launch of about one size, the time goes
// by the rounds that the compute units (few) or their eight waves take, times a
// round's. Measured for 64 experts of 2048 -> 1536 (axis 1; axis 0 alike per
// contracted value, its few-row strips a third slower) at k = 3, 512 to 8192
// rows, us: a round of few-row strips 16, of two operands 68, of four 75, of
// eight 100; at 512 rows 54 / 68 / 71 / 93, at 1024 83 / 71 / 77 / 97, at 2048
// 129 / 132 / 82 / 106, at 4096 218 / 146 / 150 / 110, at 8192 377 / 261 / 167 /
// 200 (two operands at 4096 rows took fewer rounds than estimated).
Tile tile_for(int axis, int in, int out, int rows, int experts) {
    if (axis == 0 && in < 32) return Tile::few;  // a tile's step is 32 whole rows
    const int64_t used = experts < rows ? experts : rows;
    const int64_t cus = cu_count();
    auto cost = [&](int t, int64_t round) {
        const int64_t per = 16 * kOperands[t];
        int64_t tiles = rows / per + used * 6 / 10;
        tiles = tiles > used ? tiles : used;
        const int cols = t ? kWideCols : kStripCols;
        const int64_t units = tiles * ((out + cols - 1) / cols), slots = t ? cus * kExWaves : cus;
        return (units + slots - 1) / slots * round;
    };
    const int64_t round[] = {axis == 1 ? 16 : 21, 68, 75, 100};
    int best = 0;
    for (int t = 1; t < 4; ++t)
        if (cost(t, round[t]) < cost(best, round[best])) best = t;
    return static_cast<Tile>(best);
}

// x in operand order into the workspace, then the products.
template <int K, int MT>
hipError_t launch_wide(const ExpertWeights& w, ExArgs p, void* ws, hipStream_t st) {
    const dim3 grid(tiles_at_most(p.rows, p.experts, 16 * MT), (w.in + 255) / 256);
    u32x4* operands = static_cast<u32x4*>(ws);
    auto order = w.axis == 1      ? operands_kernel<MT, 1, true>
                 : w.in % 8 == 0 ? operands_kernel<MT, 0, true>
                                 : operands_kernel<MT, 0, false>;
    const hipError_t e = launch_kernel(order, grid, dim3(256), st, p.x, p.offsets, p.experts, p.rows,
                                       p.in, operands);
    if (e != hipSuccess) return e;
    p.x = static_cast<const uint16_t*>(ws);
    return launch_kernel(w.axis == 1      ? experts1_kernel<K, MT>
                         : w.in % 32 == 0 ? experts0_kernel<K, MT, false>
                                          : experts0_kernel<K, MT, true>,
                         dim3(cu_count()), dim3(kExThreads), st, p);
}

template <int K>
hipError_t launch_k(const ExpertWeights& w, const ExArgs& p, void* ws, hipStream_t st) {
    switch (tile_for(w.axis, w.in, w.out, p.rows, p.experts)) {
    case Tile::two: return launch_wide<K, 2>(w, p, ws, st);
    case Tile::four: return launch_wide<K, 4>(w, p, ws, st);
    case Tile::eight: return launch_wide<K, 8>(w, p, ws, st);
    case Tile::few: break;
    }
    const int nb = w.in / kT;
    auto kernel = w.axis == 1 ? (nb >= 4   ? experts1_few_kernel<K, 4>
                                 : nb >= 2 ? experts1_few_kernel<K, 2>
                                           : experts1_few_kernel<K, 1>)
                              : (w.in % 8 == 0 ? experts0_few_kernel<K, true> : experts0_few_kernel<K, false>);
    return launch_kernel(kernel, dim3(cu_count()), dim3(kExThreads), st, p);
}

}  // namespace

size_t experts_workspace_bytes(int axis, int in, int out, int rows, int experts) {
    const Tile tile = tile_for(axis, in, out, rows, experts);
    if (tile == Tile::few) return 0;
    const int per = 16 * kOperands[static_cast<int>(tile)];
    const size_t values = static_cast<size_t>((in + 31) / 32) * 32;
    return static_cast<size_t>(tiles_at_most(rows, experts, per)) * per * values * sizeof(uint16_t);
}

hipError_t launch_experts(const uint16_t* x, int rows, const int32_t* offsets,
                          const ExpertWeights& w, uint16_t* y, void* ws, hipStream_t st) {
    const ExArgs p{x, offsets, w.codes, w.scales, w.lut, w.lay, w.words, w.experts, rows, w.in, w.out, y};
    return w.k == 2 ? launch_k<2>(w, p, ws, st) : w.k == 3 ? launch_k<3>(w, p, ws, st)
                                                           : launch_k<4>(w, p, ws, st);
}

}  // namespace trellis
