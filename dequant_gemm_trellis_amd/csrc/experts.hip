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
//     16-row group; step S of a block is 8 of them per lane. The matching x
//     operand is 16 bytes from 64 cache lines, so for tiles of several operands
//     x is first laid out in operand order (operands_kernel).
//   axis 0 (stored row = input): as the scatter's patches: lane (j, c) decodes 8
//     stored rows x 8 adjacent columns; x operands are read as they are.
// The decode table (pair table for k = 2, else eight bank-partitioned copies of
// the codebook) is staged once per workgroup, which stays for all its work.
// Few rows per expert: a workgroup takes a strip of one tile and its waves
// share the contraction (their sums meet in LDS in wave order). Many: every
// wave takes strips of its own, and no wave waits for another.
#include "common.hpp"
#include "groups.hpp"
#include "launch.hpp"

namespace trellis {
namespace {

constexpr int kExThreads = 512;
constexpr int kExWaves = kExThreads / kWave;
constexpr int kStripCols = 128;
constexpr int kXcds = 8;  // accelerator dies, each with its own L2

template <int K>
struct ExTable {
    static constexpr bool pair = K == 2, rep = !pair;
    using Table = DecodeTable<kExThreads, pair, rep>;
};

template <int K>
__device__ __forceinline__ void stage_table(float* tab, const float* lut) {
    typename ExTable<K>::Table::Src src;
    ExTable<K>::Table::fetch(src, lut);
    ExTable<K>::Table::store(src, tab);
    __syncthreads();
}

// Tiles of `per` rows that the experts' rows make.
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
    return __builtin_amdgcn_readfirstlane(n);
}

// Where the units of a launch are: `units` of them, this workgroup's (or
// wave's) every `step`-th from `first` on below `end`. Each XCD takes a
// contiguous range, so that strips of one tile share its rows in one L2.
struct Range {
    int first, end, step;
};
__device__ __forceinline__ Range xcd_range(int units, int per_group, int index) {
    const int xcd = blockIdx.x % kXcds, slot = blockIdx.x / kXcds;
    const int groups = (gridDim.x - xcd + kXcds - 1) / kXcds;
    const int u0 = static_cast<int>(static_cast<int64_t>(units) * xcd / kXcds);
    const int u1 = static_cast<int>(static_cast<int64_t>(units) * (xcd + 1) / kXcds);
    return {u0 + slot * per_group + index, u1, groups * per_group};
}

struct ExArgs {
    const uint16_t* x;        // rows, or operand order (axis 1 with MT > 1)
    const int32_t* offsets;
    const uint32_t* codes;
    const float* scales;
    const float* lut;
    CodeLayout lay;
    uint64_t words;           // code words per expert
    int experts, rows, in, out;
    uint16_t* y;
};

// x of a tile in operand order: [tile][block][S][MT] operands of 64 lanes x 16
// bytes; rows past the tile's last are zeros. Grid: (tiles, blocks).
template <int MT>
__global__ __launch_bounds__(256) void operands_kernel(const uint16_t* __restrict__ x,
                                                       const int32_t* __restrict__ offsets,
                                                       int experts, int rows, int in,
                                                       u32x4* __restrict__ out) {
    const Found at = find_entry(offsets, experts, rows, 16 * MT, false, blockIdx.x);
    if (at.group < 0) return;
    const int row0 = at.first + at.index * 16 * MT;
    const int lane = threadIdx.x & 63, j = lane & 15, c = lane >> 4;
    const size_t base = (static_cast<size_t>(blockIdx.x) * gridDim.y + blockIdx.y) * 8 * MT;
    // S fastest within a wave: the eight reads of a lane come from one line
    for (int o = threadIdx.x >> 6; o < MT; o += 4) {
        const int row = row0 + 16 * o + j;
        const uint16_t* p = x + static_cast<size_t>(row) * in + 256 * blockIdx.y + 64 * c;
        u32x4 v[8] = {};
        if (row < at.end) {
#pragma unroll
            for (int s = 0; s < 8; ++s) v[s] = *reinterpret_cast<const u32x4*>(p + 8 * s);
        }
#pragma unroll
        for (int s = 0; s < 8; ++s) out[(base + s * MT + o) * 64 + lane] = v[s];
    }
}

// Axis 1, tiles of MT x 16 rows: a wave takes 16 G output columns of a tile.
template <int K, int MT, int G>
__global__ __launch_bounds__(kExThreads) void experts1_kernel(ExArgs p) {
    constexpr bool pair = ExTable<K>::pair, rep = ExTable<K>::rep;
    __shared__ __attribute__((aligned(16))) float tab[ExTable<K>::Table::floats];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, c = lane >> 4;
    stage_table<K>(tab, p.lut);
    const int nb = p.in / kT, strips = (p.out + 16 * G - 1) / (16 * G);
    const int tiles = count_tiles(p.offsets, p.experts, p.rows, 16 * MT);
    const Range r = xcd_range(tiles * strips, kExWaves, wave);
    for (int u = r.first; u < r.end; u += r.step) {
        const int t = u / strips, n0 = (u - t * strips) * 16 * G;
        const Found at = find_entry(p.offsets, p.experts, p.rows, 16 * MT, false, t);
        const int row0 = at.first + at.index * 16 * MT;
        const int live = __builtin_amdgcn_readfirstlane(min(MT, (at.end - row0 + 15) / 16));
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
            static_for<0, 8>([&](auto sc_) {
                constexpr int S = decltype(sc_)::value;
                u32x4 a[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) a[m] = xo[(static_cast<size_t>(8 * b + S) * MT + m) * 64];
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const u32x4 f = pack_fragment(gather_tab<K, S, pair, rep>(w[g], tab), sc[g]);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        if (m < live)
                            acc[g][m] = mfma16x16x32(as_bf16x8(a[m]), as_bf16x8(f), acc[g][m]);
                }
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

// Sum of the waves' [16][128] parts in wave order (parts of wave groups that
// own other columns are kept apart by the caller's columns).
__device__ __forceinline__ void add_part(float* sum, int col, int c, const floatx4& v, bool first) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float* o = sum + (4 * c + i) * kStripCols + col;
        *o = first ? v[i] : *o + v[i];
    }
}

// Axis 1, tiles of 16 rows: a workgroup takes 128 output columns of a tile; its
// waves are G ways along the contraction (8 blocks at a time) and 8 / G along
// the columns, G 16-column groups each.
template <int K, int G>
__global__ __launch_bounds__(kExThreads) void experts1_few_kernel(ExArgs p) {
    constexpr bool pair = ExTable<K>::pair, rep = ExTable<K>::rep;
    __shared__ __attribute__((aligned(16))) float tab[ExTable<K>::Table::floats];
    __shared__ float sum[16 * kStripCols];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, c = lane >> 4;
    const int kw = wave % G, nw = wave / G;
    stage_table<K>(tab, p.lut);
    const int nb = p.in / kT, strips = (p.out + kStripCols - 1) / kStripCols;
    const int tiles = count_tiles(p.offsets, p.experts, p.rows, 16);
    const Range r = xcd_range(tiles * strips, 1, 0);
    for (int u = r.first; u < r.end; u += r.step) {
        const int t = u / strips, n0 = (u - t * strips) * kStripCols + nw * 16 * G;
        const Found at = find_entry(p.offsets, p.experts, p.rows, 16, false, t);
        const int row0 = at.first + at.index * 16;
        const uint32_t* codes = p.codes + at.group * p.words;
        const float* scales = p.scales + static_cast<size_t>(at.group) * p.out;
        int rowc[G];
        float sc[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            rowc[g] = min(n0 + 16 * g + j, p.out - 1);
            sc[g] = scales[rowc[g]];
        }
        const uint16_t* xr = p.x + static_cast<size_t>(min(row0 + j, at.end - 1)) * p.in + 64 * c;
        floatx4 acc[G] = {};
        for (int b = kw; b < nb; b += G) {
            uint32_t w[G][2 * K + 1];
            u32x4 a[8];
#pragma unroll
            for (int g = 0; g < G; ++g)
                load_run64<K>(codes + block_word<K>(p.lay, rowc[g], b), 3 - c, w[g]);
#pragma unroll
            for (int s = 0; s < 8; ++s)
                a[s] = *reinterpret_cast<const u32x4*>(xr + static_cast<size_t>(b) * kT + 8 * s);
            static_for<0, 8>([&](auto sc_) {
                constexpr int S = decltype(sc_)::value;
#pragma unroll
                for (int g = 0; g < G; ++g)
                    acc[g] = mfma16x16x32(
                        as_bf16x8(a[S]),
                        as_bf16x8(pack_fragment(gather_tab<K, S, pair, rep>(w[g], tab), sc[g])),
                        acc[g]);
            });
        }
        for (int q = 0; q < G; ++q) {
            if (kw == q) {
#pragma unroll
                for (int g = 0; g < G; ++g)
                    add_part(sum, nw * 16 * G + 16 * g + j, c, acc[g], q == 0);
            }
            __syncthreads();
        }
        const int first = (u - t * strips) * kStripCols;
        for (int i = tid; i < 16 * kStripCols; i += kExThreads) {
            const int row = row0 + i / kStripCols, n = first + i % kStripCols;
            if (row < at.end && n < p.out)
                p.y[static_cast<size_t>(row) * p.out + n] = round_bf16(sum[i]);
        }
        __syncthreads();  // `sum` is written again by the next unit
    }
}

// ---- axis 0 ---------------------------------------------------------------------

// One 32-row step of a wave's strip: the two words that hold the windows of a
// lane's 8 columns in each of its 8 stored rows, and the rows' scales.
struct Patch {
    uint32_t a[8], b[8];
    float sc[8];
};

struct Strip0 {
    const uint32_t* codes;  // the strip's block in stored row 0
    const float* scales;
    uint64_t row_words;
    int w0, w1, sh, in, c;
};

template <int K>
__device__ __forceinline__ Strip0 strip0(const ExArgs& p, int expert, int col0, int j, int c) {
    constexpr int wpb = Bits<K>::wpb;
    const int t0 = (col0 % kT) + 8 * j;  // first weight of this lane's 8 columns
    const int lo = (kT - 8 - t0) * K;    // bit of weight t0 + 7
    Strip0 s;
    s.codes = p.codes + expert * p.words + block_word<K>(p.lay, 0, col0 / kT);
    s.scales = p.scales + static_cast<size_t>(expert) * p.in;
    s.row_words = p.lay.row_words;
    s.w0 = lo >> 5;
    s.sh = lo & 31;
    s.w1 = s.w0 + 1 == wpb ? 0 : s.w0 + 1;  // tail-biting wrap
    s.in = p.in;
    s.c = c;
    return s;
}

__device__ __forceinline__ void load_patch(Patch& q, const Strip0& s, int step) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = min(32 * step + 8 * s.c + i, s.in - 1);  // past the end: x is zero there
        const uint32_t* w = s.codes + row * s.row_words;
        q.a[i] = w[s.w0];
        q.b[i] = w[s.w1];
        q.sc[i] = s.scales[row];
    }
}

// The eight operands of a patch, column by column (k = 2: by pairs), each
// multiplied with the tile's x operands.
template <int K, int MT>
__device__ __forceinline__ void mul_patch(const Patch& q, const Strip0& s, const float* tab,
                                          const u32x4 (&x)[MT], int live, floatx4 (&acc)[8][MT]) {
    uint32_t g[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        g[i][0] = __builtin_amdgcn_alignbit(q.b[i], q.a[i], s.sh);
        g[i][1] = q.b[i] >> s.sh;
    }
    auto mul = [&](auto ec, const u32x4& f) {
        constexpr int e = decltype(ec)::value;
#pragma unroll
        for (int m = 0; m < MT; ++m)
            if (MT == 1 || m < live)
                acc[e][m] = mfma16x16x32(as_bf16x8(x[m]), as_bf16x8(f), acc[e][m]);
    };
    if constexpr (ExTable<K>::pair) {
        static_for<0, 4>([&](auto pc) {
            constexpr int P = decltype(pc)::value, O = (6 - 2 * P) * K;
            floatx2 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = lds_pair(tab, field_offset<O, 14, 3>(g[i]));
            u32x4 f0, f1;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                f0[d] = pack_bf16(v[2 * d].x * q.sc[2 * d], v[2 * d + 1].x * q.sc[2 * d + 1]);
                f1[d] = pack_bf16(v[2 * d].y * q.sc[2 * d], v[2 * d + 1].y * q.sc[2 * d + 1]);
            }
            mul(std::integral_constant<int, 2 * P>{}, f0);
            mul(std::integral_constant<int, 2 * P + 1>{}, f1);
        });
    } else {
        const uint32_t copy = rep_lane_offset();
        static_for<0, 8>([&](auto ec) {
            constexpr int e = decltype(ec)::value, o = (7 - e) * K;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = lds_lut(tab, field_offset<o, kL, 5>(g[i]) | copy);
            u32x4 f;
#pragma unroll
            for (int d = 0; d < 4; ++d)
                f[d] = pack_bf16(v[2 * d] * q.sc[2 * d], v[2 * d + 1] * q.sc[2 * d + 1]);
            mul(ec, f);
        });
    }
}

// x operand of 16 rows from row0 on (rows past `end` read the last), step `step`.
template <bool VEC>
__device__ __forceinline__ u32x4 x_operand(const ExArgs& p, int row0, int end, int step, int j, int c) {
    const int row = min(row0 + j, end - 1);
    return load8<VEC>(p.x + static_cast<size_t>(row) * p.in, 32 * step + 8 * c, p.in, true);
}

template <int K, int MT, bool VEC>
__global__ __launch_bounds__(kExThreads) void experts0_kernel(ExArgs p) {
    __shared__ __attribute__((aligned(16))) float tab[ExTable<K>::Table::floats];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, c = lane >> 4;
    stage_table<K>(tab, p.lut);
    const int steps = (p.in + 31) / 32, strips = p.out / kStripCols;
    const int tiles = count_tiles(p.offsets, p.experts, p.rows, 16 * MT);
    const Range r = xcd_range(tiles * strips, kExWaves, wave);
    for (int u = r.first; u < r.end; u += r.step) {
        const int t = u / strips, col0 = (u - t * strips) * kStripCols;
        const Found at = find_entry(p.offsets, p.experts, p.rows, 16 * MT, false, t);
        const int row0 = at.first + at.index * 16 * MT;
        const int live = __builtin_amdgcn_readfirstlane(min(MT, (at.end - row0 + 15) / 16));
        const Strip0 s = strip0<K>(p, at.group, col0, j, c);
        floatx4 acc[8][MT] = {};
        Patch q[2];
        load_patch(q[0], s, 0);
        auto one = [&](Patch& now, Patch& next, int step) {
            u32x4 x[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m)
                x[m] = x_operand<VEC>(p, min(row0 + 16 * m, at.end - 1), at.end, step, j, c);
            if (step + 1 < steps) load_patch(next, s, step + 1);
            mul_patch<K, MT>(now, s, tab, x, live, acc);
        };
        for (int step = 0; step < steps; step += 2) {
            one(q[0], q[1], step);
            if (step + 1 < steps) one(q[1], q[0], step + 1);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = row0 + 16 * m + 4 * c + i;
                if (row >= at.end) continue;
                u32x4 o;
#pragma unroll
                for (int d = 0; d < 4; ++d) o[d] = pack_bf16(acc[2 * d][m][i], acc[2 * d + 1][m][i]);
                *reinterpret_cast<u32x4*>(p.y + static_cast<size_t>(row) * p.out + col0 + 8 * j) = o;
            }
    }
}

template <int K, bool VEC>
__global__ __launch_bounds__(kExThreads) void experts0_few_kernel(ExArgs p) {
    __shared__ __attribute__((aligned(16))) float tab[ExTable<K>::Table::floats];
    __shared__ float sum[16 * kStripCols];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, c = lane >> 4;
    stage_table<K>(tab, p.lut);
    const int steps = (p.in + 31) / 32, strips = p.out / kStripCols;
    const int tiles = count_tiles(p.offsets, p.experts, p.rows, 16);
    const Range r = xcd_range(tiles * strips, 1, 0);
    for (int u = r.first; u < r.end; u += r.step) {
        const int t = u / strips, col0 = (u - t * strips) * kStripCols;
        const Found at = find_entry(p.offsets, p.experts, p.rows, 16, false, t);
        const int row0 = at.first + at.index * 16;
        const Strip0 s = strip0<K>(p, at.group, col0, j, c);
        floatx4 acc[8][1] = {};
        for (int step = wave; step < steps; step += kExWaves) {
            Patch q;
            load_patch(q, s, step);
            const u32x4 x[1] = {x_operand<VEC>(p, row0, at.end, step, j, c)};
            mul_patch<K, 1>(q, s, tab, x, 1, acc);
        }
        for (int w = 0; w < kExWaves; ++w) {
            if (wave == w) {
#pragma unroll
                for (int e = 0; e < 8; ++e) add_part(sum, 8 * j + e, c, acc[e][0], w == 0);
            }
            __syncthreads();
        }
        for (int i = tid; i < 16 * kStripCols / 2; i += kExThreads) {
            const int row = row0 + i / (kStripCols / 2), at2 = 2 * (i % (kStripCols / 2));
            if (row < at.end)
                *reinterpret_cast<uint32_t*>(p.y + static_cast<size_t>(row) * p.out + col0 + at2) =
                    pack_bf16(sum[2 * i], sum[2 * i + 1]);
        }
        __syncthreads();
    }
}

// ---- launches ---------------------------------------------------------------------

// Rows of a tile by the average of an expert's: up to 16 the products are
// decode-bound and a workgroup shares one tile; beyond, taller tiles decode
// each weight for more rows.
enum class Tile { few, some, many };
Tile tile_for(int rows, int experts) {
    const int mean = (rows + experts - 1) / experts;
    return mean <= 16 ? Tile::few : mean <= 64 ? Tile::some : Tile::many;
}

int tiles_at_most(int rows, int experts, int per) {
    return rows / per + (experts < rows ? experts : rows);
}

// Rows per tile on axis 1 and axis 0.
constexpr int kSome1 = 4, kMany1 = 8, kSome0 = 2, kMany0 = 4;

template <int K, int MT>
hipError_t launch1(const ExpertWeights& w, ExArgs p, void* ws, hipStream_t st) {
    const int tiles = tiles_at_most(p.rows, p.experts, 16 * MT);
    u32x4* operands = static_cast<u32x4*>(ws);
    const hipError_t e = launch_kernel(operands_kernel<MT>, dim3(tiles, w.in / kT), dim3(256), st, p.x,
                                       p.offsets, p.experts, p.rows, p.in, operands);
    if (e != hipSuccess) return e;
    p.x = static_cast<const uint16_t*>(ws);
    return launch_kernel(experts1_kernel<K, MT, 4>, dim3(cu_count()), dim3(kExThreads), st, p);
}

template <int K>
hipError_t launch_k(const ExpertWeights& w, const ExArgs& p, void* ws, hipStream_t st) {
    const Tile tile = tile_for(p.rows, p.experts);
    const dim3 grid(cu_count()), block(kExThreads);
    if (w.axis == 1) {
        if (tile == Tile::some) return launch1<K, kSome1>(w, p, ws, st);
        if (tile == Tile::many) return launch1<K, kMany1>(w, p, ws, st);
        const int nb = w.in / kT;
        auto kernel = nb >= 8   ? experts1_few_kernel<K, 8>
                      : nb >= 4 ? experts1_few_kernel<K, 4>
                      : nb >= 2 ? experts1_few_kernel<K, 2>
                                : experts1_few_kernel<K, 1>;
        return launch_kernel(kernel, grid, block, st, p);
    }
    const bool vec = w.in % 8 == 0;
    auto kernel = tile == Tile::few    ? (vec ? experts0_few_kernel<K, true> : experts0_few_kernel<K, false>)
                  : tile == Tile::some ? (vec ? experts0_kernel<K, kSome0, true> : experts0_kernel<K, kSome0, false>)
                                       : (vec ? experts0_kernel<K, kMany0, true> : experts0_kernel<K, kMany0, false>);
    return launch_kernel(kernel, grid, block, st, p);
}

}  // namespace

size_t experts_workspace_bytes(int axis, int in, int rows, int experts) {
    const Tile tile = tile_for(rows, experts);
    if (axis != 1 || tile == Tile::few) return 0;
    const int per = 16 * (tile == Tile::some ? kSome1 : kMany1);
    return static_cast<size_t>(tiles_at_most(rows, experts, per)) * per * in * sizeof(uint16_t);
}

hipError_t launch_experts(const uint16_t* x, int rows, const int32_t* offsets,
                          const ExpertWeights& w, uint16_t* y, void* ws, hipStream_t st) {
    const ExArgs p{x, offsets, w.codes, w.scales, w.lut, w.lay, w.words, w.experts, rows, w.in, w.out, y};
    return w.k == 2 ? launch_k<2>(w, p, ws, st) : w.k == 3 ? launch_k<3>(w, p, ws, st)
                                                           : launch_k<4>(w, p, ws, st);
}

}  // namespace trellis
