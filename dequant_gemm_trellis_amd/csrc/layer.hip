// A whole layer of experts for few tokens (trellis_experts_mlp):
//   h_e[m] = bf16( w_e[m] silu(Wg_e x[m]) (Wu_e x[m]) ),
//   out[m] = bf16( sum over the experts e that m chose of Wd_e h_e[m] ).
//
// With few tokens nearly all work is decoding, and a decoded operand meets 16
// rows in one matrix instruction at no cost. So no token is sorted or moved: every
// expert that anyone chose is decoded once and multiplied with all tokens, and
// what a token did not choose is left out of its sums (not multiplied by zero: an
// infinite weight of another's expert must not reach it). The second product is
// one long contraction over all chosen experts.
//   up: units of 8 gate and 8 up rows of an expert, dealt evenly to the workgroups;
//     a unit's blocks go to the eight waves in turn, whose sums meet in LDS, where h
//     is formed. h is stored in the second product's operand order.
//   down: a workgroup takes a strip of output columns and a part of the contraction;
//     its waves take steps in turn.
//   sum: adds the parts.
#include "common.hpp"
#include "experts.hpp"
#include "groups.hpp"
#include "kept.hpp"
#include "launch.hpp"
#include "layer.hpp"

namespace trellis {
namespace {

constexpr int kUnitCols = 8;  // columns of h per unit: 8 gate and 8 up rows
constexpr int kPartFloats = 5 * 1024;

// ---- the chosen experts -------------------------------------------------------

struct Chosen {
    uint32_t mask[kMaxGroups];   // by expert: the tokens that chose it
    uint16_t expert[kMaxGroups]; // ascending
    int first[kMaxGroups / kWave + 1];
};

// Fills `s` from the tokens' ids; every thread of the workgroup calls it. Returns
// the number of chosen experts. An id outside [0, experts) chooses none.
__device__ __forceinline__ int find_chosen(Chosen& s, const int32_t* __restrict__ ids, int tokens,
                                           int top_k, int experts) {
    const int tid = threadIdx.x, lane = tid & 63;
    for (int e = tid; e < experts; e += kExThreads) s.mask[e] = 0;
    __syncthreads();
    for (int i = tid; i < tokens * top_k; i += kExThreads) {
        const int e = ids[i];
        if (static_cast<uint32_t>(e) < static_cast<uint32_t>(experts)) atomicOr(&s.mask[e], 1u << (i / top_k));
    }
    __syncthreads();
    for (int e0 = tid - lane; e0 < experts; e0 += kExThreads) {
        const uint64_t live = __ballot(e0 + lane < experts && s.mask[e0 + lane] != 0);
        if (lane == 0) s.first[e0 / kWave + 1] = __popcll(live);
    }
    if (tid == 0) s.first[0] = 0;
    __syncthreads();
    const int chunks = (experts + kWave - 1) / kWave;
    if (tid == 0)
        for (int i = 0; i < chunks; ++i) s.first[i + 1] += s.first[i];
    __syncthreads();
    for (int e0 = tid - lane; e0 < experts; e0 += kExThreads) {
        const bool mine = e0 + lane < experts && s.mask[e0 + lane] != 0;
        const uint64_t live = __ballot(mine);
        if (mine) s.expert[s.first[e0 / kWave] + __popcll(live & ((1ull << lane) - 1))] = static_cast<uint16_t>(e0 + lane);
    }
    __syncthreads();
    return s.first[chunks];
}

// ---- operand order of h ---------------------------------------------------------

// h of the chosen expert number `at` in the order that the down product reads:
// [chosen][piece of 32 contracted values][operand][64 lanes][8].
// Axis 0: piece s is values 32 s + 8 c ...; axis 1: piece (b, s) is values
// 256 b + 64 c + 8 s ... (c = lane / 16).
__host__ __device__ __forceinline__ int h_pieces(int inter) { return (inter + 31) / 32; }

template <int MT>
__device__ __forceinline__ size_t h_at(int at, int pieces, int axis, int col, int token) {
    const int piece = axis == 1 ? col / 256 * 8 + col % 64 / 8 : col / 32;
    const int c = axis == 1 ? col % 256 / 64 : col % 32 / 8;
    return (((static_cast<size_t>(at) * pieces + piece) * MT + token / 16) * kWave + 16 * c + token % 16) * 8 +
           col % 8;
}

// ---- up -------------------------------------------------------------------------

struct UpArgs {
    const uint16_t* x;
    const int32_t* ids;
    const float* weights;
    int tokens, top_k, experts, hidden, inter, axis_down;
    const uint32_t* codes;
    const float* scales;
    const float* lut;
    CodeLayout lay;
    uint64_t words;
    uint16_t* h;
};

template <int K, int MT>
__global__ __launch_bounds__(kExThreads) void layer_up_kernel(UpArgs p) {
    constexpr bool pair = ExTable<K>::pair, rep = ExTable<K>::rep;
    __shared__ __attribute__((aligned(16))) float tab[ExTable<K>::Table::floats];
    __shared__ float parts[kPartFloats];
    __shared__ Chosen chosen;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, c = lane >> 4;
    typename ExTable<K>::Table::Src src;
    ExTable<K>::Table::fetch(src, p.lut);
    const int live = __builtin_amdgcn_readfirstlane(find_chosen(chosen, p.ids, p.tokens, p.top_k, p.experts));
    const int nb = p.hidden / kT, per = (p.inter + kUnitCols - 1) / kUnitCols;
    const int64_t units = static_cast<int64_t>(live) * per;
    const int u0 = static_cast<int>(units * blockIdx.x / gridDim.x);
    const int u1 = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
    ExTable<K>::Table::store(src, tab);
    __syncthreads();

    // Units of a phase: their sums of all waves, [unit][wave][token][16], fill `parts`.
    const int unit_floats = 16 * p.tokens, phase_units = kPartFloats / (kExWaves * unit_floats);
    const int tasks = (u1 - u0) * nb, phase_tasks = phase_units * nb;
    struct Work {
        uint32_t w[2 * K + 1];
        float sc;
        u32x4 a[MT][8];
    };
    auto load = [&](Work& q, int t) {
        const int u = u0 + t / nb, b = t % nb;
        const int at = u / per, col0 = (u - at * per) * kUnitCols;
        const int e = __builtin_amdgcn_readfirstlane(chosen.expert[at]);
        const int row = min(col0 + (j & 7), p.inter - 1) + (j < 8 ? 0 : p.inter);
        load_run64<K>(p.codes + e * p.words + block_word<K>(p.lay, row, b), 3 - c, q.w);
        q.sc = p.scales[static_cast<size_t>(e) * (2 * p.inter) + row];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint16_t* x = p.x + static_cast<size_t>(min(16 * m + j, p.tokens - 1)) * p.hidden +
                                static_cast<size_t>(b) * kT + 64 * c;
#pragma unroll
            for (int s = 0; s < 8; ++s) q.a[m][s] = *reinterpret_cast<const u32x4*>(x + 8 * s);
        }
    };
    floatx4 acc[MT] = {};
    int phase = 0, unit = -1;  // unit: whose sums `acc` holds
    auto put = [&] {
        if (unit < 0) return;
        float* o = parts + ((unit - phase * phase_units) * kExWaves + wave) * unit_floats + j;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (16 * m + 4 * c + i < p.tokens) o[16 * (16 * m + 4 * c + i)] = acc[m][i];
            acc[m] = floatx4{};
        }
        unit = -1;
    };
    // Sums of a phase's units, the waves in the order of their first blocks, and h.
    auto finish = [&] {
        put();
        __syncthreads();
        const int n = min(phase_units, u1 - u0 - phase * phase_units);
        for (int i = tid; i < n * p.tokens * kUnitCols; i += kExThreads) {
            const int col = i % kUnitCols, m = i / kUnitCols % p.tokens, v = i / kUnitCols / p.tokens;
            const int lu = phase * phase_units + v, at = (u0 + lu) / per;
            const int out = (u0 + lu - at * per) * kUnitCols + col, e = chosen.expert[at];
            if (!((chosen.mask[e] >> m) & 1)) continue;
            float g = 0.f, u = 0.f;
            for (int k = 0; k < min(nb, kExWaves); ++k) {
                const float* o = parts + (v * kExWaves + (lu * nb + k) % kExWaves) * unit_floats + 16 * m + col;
                g += o[0];
                u += o[8];
            }
            float w = 0.f;
            for (int k = 0; k < p.top_k; ++k)
                if (p.ids[m * p.top_k + k] == e) w += p.weights ? p.weights[m * p.top_k + k] : 1.f;
            const float hv = w * (g / (1.f + expf(-g)) * u);
            p.h[h_at<MT>(at, h_pieces(p.inter), p.axis_down, out, m)] = out < p.inter ? round_bf16(hv) : uint16_t{0};
        }
        __syncthreads();
        ++phase;
    };
    auto multiply = [&](const Work& q) {
        Gathered<pair> v[2];
        v[0] = gather_tab<K, 0, pair, rep>(q.w, tab);
        static_for<0, 8>([&](auto sc) {
            constexpr int S = decltype(sc)::value;
            __builtin_amdgcn_s_setprio(2);
            if constexpr (S + 1 < 8) v[(S + 1) & 1] = gather_tab<K, S + 1, pair, rep>(q.w, tab);
            __builtin_amdgcn_s_setprio(0);
            const u32x4 f = pack_fragment(v[S & 1], q.sc);
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[m] = mfma16x16x32(as_bf16x8(q.a[m][S]), as_bf16x8(f), acc[m]);
        });
    };
    const int phases = (u1 - u0 + phase_units - 1) / phase_units;
    auto one = [&](Work& now, Work& next, int t) {
        while (phase < t / phase_tasks) finish();
        if (t / nb != unit) {
            put();
            unit = t / nb;
        }
        if (t + kExWaves < tasks) load(next, t + kExWaves);
        multiply(now);
    };
    Work q[2];
    int t = wave;
    if (t < tasks) load(q[0], t);
    while (t < tasks) {
        one(q[0], q[1], t);
        t += kExWaves;
        if (t >= tasks) break;
        one(q[1], q[0], t);
        t += kExWaves;
    }
    while (phase < phases) finish();
}

// ---- down -----------------------------------------------------------------------

struct DownArgs {
    const uint16_t* h;
    const int32_t* ids;
    int tokens, top_k, experts, hidden, inter;
    const uint32_t* codes;
    const float* scales;
    const float* lut;
    CodeLayout lay;
    uint64_t words;
    int strips, ways;  // strips of columns, parts of the contraction
    float* partial;    // [way][tokens][hidden]
};

// A wave's sums over its tasks (an expert's and piece's, `steps` pieces each), the
// experts kept apart: a token takes what it chose.
template <int N, int MT>
struct Sums {
    floatx4 now[N][MT] = {}, total[N][MT] = {};

    __device__ __forceinline__ void close(uint32_t mask, int c) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool mine = (mask >> (16 * m + 4 * c + i)) & 1;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    total[n][m][i] = mine ? total[n][m][i] + now[n][m][i] : total[n][m][i];
                    now[n][m][i] = 0.f;
                }
            }
    }
};

// The waves' sums of a strip of COLS columns, in wave order, to the workgroup's
// part: each(f) gives f(token, column, value). `sums` takes the table's place.
template <int COLS, typename F>
__device__ __forceinline__ void put_part(float* sums, const DownArgs& p, int strip, int way, F&& each) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    __syncthreads();  // the table is read
    each([&](int token, int col, float v) {
        if (token < p.tokens) sums[(wave * p.tokens + token) * COLS + col] = v;
    });
    __syncthreads();
    for (int i = threadIdx.x; i < p.tokens * COLS; i += kExThreads) {
        const int token = i / COLS, col = strip * COLS + i % COLS;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kExWaves; ++w) v += sums[w * p.tokens * COLS + i];
        if (col < p.hidden) p.partial[(static_cast<size_t>(way) * p.tokens + token) * p.hidden + col] = v;
    }
}

// The tasks of this workgroup, wave by wave: load(work, at, piece) of the next one
// is in flight while multiply(work) runs; `at` numbers the chosen experts.
template <typename Work, typename Load, typename Multiply, typename Close>
__device__ __forceinline__ void run_tasks(int first, int end, int pieces, int wave, Load&& load,
                                          Multiply&& multiply, Close&& close) {
    Work q[2];
    int t = first + wave, at = t / pieces;
    if (t < end) load(q[0], at, t - at * pieces);
    auto one = [&](Work& now, Work& next) {
        const int nt = t + kExWaves, nat = nt / pieces;
        if (nt < end) load(next, nat, nt - nat * pieces);
        multiply(now);
        if (nt >= end || nat != at) close(at);
        t = nt;
        at = nat;
    };
    while (t < end) {
        one(q[0], q[1]);
        if (t < end) one(q[1], q[0]);
    }
}

constexpr int kDownGroups = 2;  // axis 1: 16-row groups of a strip
constexpr int kDownCols1 = 16 * kDownGroups;
constexpr int kDownCols0 = 128;

template <int K, int MT>
__global__ __launch_bounds__(kExThreads) void layer_down1_kernel(DownArgs p) {
    constexpr bool pair = ExTable<K>::pair, rep = ExTable<K>::rep;
    constexpr int G = kDownGroups;
    __shared__ __attribute__((aligned(16))) float tab[ExTable<K>::Table::floats];
    __shared__ Chosen chosen;
    const int lane = threadIdx.x & 63, j = lane & 15, c = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    typename ExTable<K>::Table::Src src;
    ExTable<K>::Table::fetch(src, p.lut);
    const int live = __builtin_amdgcn_readfirstlane(find_chosen(chosen, p.ids, p.tokens, p.top_k, p.experts));
    ExTable<K>::Table::store(src, tab);
    __syncthreads();
    const int strip = blockIdx.x / p.ways, way = blockIdx.x % p.ways, nb = p.inter / kT;
    const int64_t tasks = static_cast<int64_t>(live) * nb;
    struct Work {
        uint32_t w[G][2 * K + 1];
        float sc[G];
        u32x4 a[MT][8];
    };
    Sums<G, MT> sums;
    int rows[G];
#pragma unroll
    for (int g = 0; g < G; ++g) rows[g] = min(strip * kDownCols1 + 16 * g + j, p.hidden - 1);
    const u32x4* h = reinterpret_cast<const u32x4*>(p.h) + lane;
    run_tasks<Work>(
        static_cast<int>(tasks * way / p.ways), static_cast<int>(tasks * (way + 1) / p.ways), nb, wave,
        [&](Work& q, int at, int b) {
            const int e = __builtin_amdgcn_readfirstlane(chosen.expert[at]);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                load_run64<K>(p.codes + e * p.words + block_word<K>(p.lay, rows[g], b), 3 - c, q.w[g]);
                q.sc[g] = p.scales[static_cast<size_t>(e) * p.hidden + rows[g]];
            }
            const u32x4* ha = h + (static_cast<size_t>(at) * nb + b) * 8 * MT * kWave;
#pragma unroll
            for (int s = 0; s < 8; ++s)
#pragma unroll
                for (int m = 0; m < MT; ++m) q.a[m][s] = ha[(s * MT + m) * kWave];
        },
        [&](const Work& q) {
            Gathered<pair> v[2];
            v[0] = gather_tab<K, 0, pair, rep>(q.w[0], tab);
            static_for<0, 8 * G>([&](auto ic) {
                constexpr int i = decltype(ic)::value, S = i / G, g = i % G, n = i + 1;
                __builtin_amdgcn_s_setprio(2);
                if constexpr (n < 8 * G) v[n & 1] = gather_tab<K, n / G, pair, rep>(q.w[n % G], tab);
                __builtin_amdgcn_s_setprio(0);
                const u32x4 f = pack_fragment(v[i & 1], q.sc[g]);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    sums.now[g][m] = mfma16x16x32(as_bf16x8(q.a[m][S]), as_bf16x8(f), sums.now[g][m]);
            });
        },
        [&](int at) { sums.close(chosen.mask[chosen.expert[at]], c); });
    put_part<kDownCols1>(tab, p, strip, way, [&](auto&& f) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i) f(16 * m + 4 * c + i, 16 * g + j, sums.total[g][m][i]);
    });
}

template <int K, int MT>
__global__ __launch_bounds__(kExThreads) void layer_down0_kernel(DownArgs p) {
    constexpr int CL = 8;
    __shared__ __attribute__((aligned(16))) float tab[ExTable<K>::Table::floats];
    __shared__ Chosen chosen;
    const int lane = threadIdx.x & 63, j = lane & 15, c = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    typename ExTable<K>::Table::Src src;
    ExTable<K>::Table::fetch(src, p.lut);
    const int live = __builtin_amdgcn_readfirstlane(find_chosen(chosen, p.ids, p.tokens, p.top_k, p.experts));
    ExTable<K>::Table::store(src, tab);
    __syncthreads();
    const int strip = blockIdx.x / p.ways, way = blockIdx.x % p.ways, steps = h_pieces(p.inter);
    const int64_t tasks = static_cast<int64_t>(live) * steps;
    struct Work {
        Words q;
        float sc[8];
        u32x4 a[MT];
        int rows;  // stored rows of the step
    };
    Sums<CL, MT> sums;
    const Strip0 first = strip0<K, CL>(p.codes, p.scales, p.lay, strip * kDownCols0, j, c);
    const u32x4* h = reinterpret_cast<const u32x4*>(p.h) + lane;
    run_tasks<Work>(
        static_cast<int>(tasks * way / p.ways), static_cast<int>(tasks * (way + 1) / p.ways), steps, wave,
        [&](Work& q, int at, int step) {
            const int e = __builtin_amdgcn_readfirstlane(chosen.expert[at]);
            Strip0 s = first;
            s.codes += e * p.words;
            s.scales += static_cast<size_t>(e) * p.inter;
            q.rows = p.inter - 32 * step;
            const u32x4* ha = h + (static_cast<size_t>(at) * steps + step) * MT * kWave;
            // 8 values of a token that lie behind the last are no values at all
#pragma unroll
            for (int m = 0; m < MT; ++m) q.a[m] = 8 * c < q.rows ? ha[m * kWave] : u32x4{0u, 0u, 0u, 0u};
            if (q.rows >= 32) {
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
            const uint32_t row = static_cast<uint32_t>(32 * c * s.row_words);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = min(32 * step + 8 * c + i, p.inter - 1);
                const uint32_t* w = s.codes + static_cast<uint64_t>(r) * s.row_words;
                q.q.a[i] = w[(s.at_a - row) / 4];
                q.q.b[i] = w[(s.at_b - row) / 4];
                q.sc[i] = s.scales[r];
            }
        },
        [&](const Work& q) {
            Pieces<K, CL> ps;
            ps.set(q.q, first.sh);
            const int left = q.rows - 8 * c;  // of this lane's 8 rows
            ps.each(q.sc, tab, [&](auto ec, u32x4 f) {
                constexpr int e = decltype(ec)::value;
                if (q.rows < 32) {  // rows behind the last have no weights: theirs may be infinite
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        f[d] &= (2 * d < left ? 0xFFFFu : 0u) | (2 * d + 1 < left ? 0xFFFF0000u : 0u);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    sums.now[e][m] = mfma16x16x32(as_bf16x8(q.a[m]), as_bf16x8(f), sums.now[e][m]);
            });
        },
        [&](int at) { sums.close(chosen.mask[chosen.expert[at]], c); });
    put_part<kDownCols0>(tab, p, strip, way, [&](auto&& f) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < CL; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) f(16 * m + 4 * c + i, CL * j + e, sums.total[e][m][i]);
    });
}

// out = the parts' sum, ascending.
__global__ __launch_bounds__(256) void layer_sum_kernel(const float* __restrict__ partial, int ways, int n,
                                                        uint16_t* __restrict__ out) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float v = 0.f;
#pragma unroll 8
    for (int w = 0; w < ways; ++w) v += partial[static_cast<size_t>(w) * n + i];
    out[i] = round_bf16(v);
}

// ---- launches ---------------------------------------------------------------------

struct LayerPlan {
    int strips, ways;
    size_t partial, bytes;
};

LayerPlan layer_plan(int tokens, int top_k, int experts, int hidden, int inter, int axis_down) {
    LayerPlan p;
    const int cols = axis_down == 1 ? kDownCols1 : kDownCols0;
    p.strips = (hidden + cols - 1) / cols;
    p.ways = cu_count() / p.strips;
    if (p.ways < 1) p.ways = 1;
    const size_t chosen = tokens * top_k < experts ? tokens * top_k : experts;
    const size_t operands = tokens > 16 ? 2 : 1;
    p.partial = chosen * h_pieces(inter) * operands * kWave * 16;
    p.bytes = p.partial + static_cast<size_t>(p.ways) * tokens * hidden * sizeof(float);
    return p;
}

template <int K>
hipError_t launch_up(const UpArgs& p, hipStream_t st) {
    return launch_kernel(p.tokens > 16 ? layer_up_kernel<K, 2> : layer_up_kernel<K, 1>, dim3(cu_count()),
                         dim3(kExThreads), st, p);
}

template <int K>
hipError_t launch_down(const DownArgs& p, int axis, hipStream_t st) {
    auto kernel = axis == 1 ? (p.tokens > 16 ? layer_down1_kernel<K, 2> : layer_down1_kernel<K, 1>)
                            : (p.tokens > 16 ? layer_down0_kernel<K, 2> : layer_down0_kernel<K, 1>);
    return launch_kernel(kernel, dim3(p.strips * p.ways), dim3(kExThreads), st, p);
}

}  // namespace

size_t layer_workspace_bytes(int tokens, int top_k, int experts, int hidden, int inter, int axis_down) {
    return layer_plan(tokens, top_k, experts, hidden, inter, axis_down).bytes;
}

hipError_t launch_layer(const LayerArgs& a, void* ws, hipStream_t st) {
    const ExpertWeights &u = a.up, &d = a.down;
    const int hidden = u.in, inter = d.in;
    const LayerPlan plan = layer_plan(a.tokens, a.top_k, u.experts, hidden, inter, d.axis);
    uint16_t* h = static_cast<uint16_t*>(ws);
    float* partial = reinterpret_cast<float*>(static_cast<char*>(ws) + plan.partial);
    const UpArgs up{a.x,    a.ids,   a.weights, a.tokens, a.top_k, u.experts, hidden, inter,
                    d.axis, u.codes, u.scales,  u.lut,    u.lay,   u.words,   h};
    hipError_t e = u.k == 2 ? launch_up<2>(up, st) : u.k == 3 ? launch_up<3>(up, st) : launch_up<4>(up, st);
    if (e != hipSuccess) return e;
    const DownArgs down{h,       a.ids,    a.tokens, a.top_k, d.experts, hidden,      inter,     d.codes,
                        d.scales, d.lut,   d.lay,    d.words, plan.strips, plan.ways, partial};
    e = d.k == 2   ? launch_down<2>(down, d.axis, st)
        : d.k == 3 ? launch_down<3>(down, d.axis, st)
                   : launch_down<4>(down, d.axis, st);
    if (e != hipSuccess) return e;
    const int n = a.tokens * hidden;
    return launch_kernel(layer_sum_kernel, dim3((n + 255) / 256), dim3(256), st, partial, plan.ways, n, a.out);
}

}  // namespace trellis
