// Decoding of the experts' coded matrices in registers, shared by the products
// over sorted rows (experts.hip) and the layer for few tokens (layer.hip): the
// decode table of a workgroup, and the operands of axis 0.
#pragma once

#include "common.hpp"
#include "groups.hpp"

namespace trellis {

constexpr int kExThreads = 512;
constexpr int kExWaves = kExThreads / kWave;

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

// A load from a uniform address plus an offset per lane. The offset is opaque, or
// the compiler adds it to a loop's invariant base and keeps 64-bit addresses in
// vector registers.
template <typename T>
__device__ __forceinline__ T load_at(const void* uniform, uint32_t lane_bytes) {
    asm volatile("" : "+v"(lane_bytes));
    return *reinterpret_cast<const T*>(static_cast<const char*>(uniform) + lane_bytes);
}

// Words of one 32-row step of a wave's strip, CL adjacent columns per lane: the
// two that hold a lane's windows in each of its 8 stored rows.
struct Words {
    uint32_t a[8], b[8];
};

struct Strip0 {
    const uint32_t* codes;   // the strip's block in stored row 0
    const float* scales;
    uint64_t row_words;
    uint32_t at_a, at_b;     // bytes from a step's first row to the words of the lane's first row
    int sh;                  // where the windows start in the first word
};

// The strip of columns from col0 on of the coded matrix at `codes`.
template <int K, int CL>
__device__ __forceinline__ Strip0 strip0(const uint32_t* codes, const float* scales, const CodeLayout& lay,
                                         int col0, int j, int c) {
    constexpr int wpb = Bits<K>::wpb;
    const int t0 = (col0 % kT) + CL * j;  // first weight of this lane's columns
    const int lo = (kT - CL - t0) * K;    // bit of its last weight
    const int w0 = lo >> 5, w1 = w0 + 1 == wpb ? 0 : w0 + 1;  // tail-biting wrap
    const uint32_t row = static_cast<uint32_t>(8 * c * lay.row_words);
    return {codes + block_word<K>(lay, 0, col0 / kT), scales, lay.row_words, 4 * (row + w0),
            4 * (row + w1), lo & 31};
}

typedef floatx4 floatx4_a4 __attribute__((aligned(4)));

// Loads of 32 whole rows from row0 on: a uniform row plus an offset per lane.
__device__ __forceinline__ void load_words(Words& q, const Strip0& s, int row0) {
    const uint32_t* row = s.codes + static_cast<uint64_t>(row0) * s.row_words;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q.a[i] = load_at<uint32_t>(row + i * s.row_words, s.at_a);
        q.b[i] = load_at<uint32_t>(row + i * s.row_words, s.at_b);
    }
}

// A step's operands come in pieces: a column, or for k = 2 a pair of columns.
// Their codebook values are read a piece ahead of their use.
template <int K, int CL>
struct Pieces {
    static constexpr bool pair = ExTable<K>::pair;
    static constexpr int cols = pair ? 2 : 1, n = CL / cols;
    static constexpr int words = (CL - 1) * K + kL <= 32 ? 1 : 2;  // of a row's windows
    struct Values {
        float v[8][cols];
    };
    uint32_t g[8][words];

    __device__ __forceinline__ void set(const Words& q, int sh) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[i][0] = __builtin_amdgcn_alignbit(q.b[i], q.a[i], sh);
            if constexpr (words == 2) g[i][1] = q.b[i] >> sh;
        }
    }
    template <int P>
    __device__ __forceinline__ void gather(Values& o, const float* tab) const {
        const uint32_t copy = rep_lane_offset();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (pair) {
                const floatx2 v = lds_pair(tab, field_offset<(CL - 2 - 2 * P) * K, 14, 3>(g[i]));
                o.v[i][0] = v.x;
                o.v[i][1] = v.y;
            } else {
                o.v[i][0] = lds_lut(tab, field_offset<(CL - 1 - P) * K, kL, 5>(g[i]) | copy);
            }
        }
    }
    // Column C of a piece, scaled by the rows' scales.
    template <int C>
    static __device__ __forceinline__ u32x4 pack(const Values& o, const float (&sc)[8]) {
        u32x4 f;
#pragma unroll
        for (int d = 0; d < 4; ++d)
            f[d] = pack_bf16(o.v[2 * d][C] * sc[2 * d], o.v[2 * d + 1][C] * sc[2 * d + 1]);
        return f;
    }
    // Every column's operand to mul(column, operand).
    template <typename F>
    __device__ __forceinline__ void each(const float (&sc)[8], const float* tab, F&& mul) const {
        Values v[2];
        gather<0>(v[0], tab);
        static_for<0, n>([&](auto pc) {
            constexpr int P = decltype(pc)::value;
            if constexpr (P + 1 < n) gather<P + 1>(v[(P + 1) & 1], tab);
            static_for<0, cols>([&](auto cc) {
                constexpr int C = decltype(cc)::value;
                mul(std::integral_constant<int, cols * P + C>{}, pack<C>(v[P & 1], sc));
            });
        });
    }
};

}  // namespace trellis
