// A whole layer of experts for few tokens (trellis_experts_mlp):
//   h_e[m] = w_e[m] silu(Wg_e x[m]) (Wu_e x[m]),
//   out[m] = bf16( sum over the experts e that m chose of Wd_e h_e[m] ).
//
// With few tokens nearly all work is decoding, through random reads of a codebook table
// in LDS, its floor; a decoded operand meets 16 rows in one matrix instruction at no
// cost. So up to 16 tokens none is sorted or moved: every expert that anyone chose is
// decoded once and multiplied with all tokens, and what a token did not choose is left
// out of its sums (not multiplied by zero: an infinite weight of another's expert must
// not reach it). The second product is one long contraction over all chosen experts.
//   up: units of 8 gate and 8 up rows of an expert, dealt evenly to the workgroups,
//     whose waves share units or a unit's blocks, as takes fewer rounds; several waves'
//     sums meet in LDS. h is stored in the second product's operand order. More than 16
//     tokens go as tiles of an expert's own, if there is work for them.
//   down: a workgroup takes a strip of output columns and a part of the contraction;
//     its waves take steps in turn. The last workgroup of a strip to arrive adds the parts.
//
// MI355X, 64 experts 2048 -> 768 -> 2048, 8 choices a token, us in the two kernels: one
// token at k = 3 11.9 + 10.7 (37.7 M weights, 5.9 us at the codebook reads' rate; about
// 4.5 us of each kernel is the choice of experts, the table and the first loads), 32
// tokens at k = 2, 3 31 + 27 (49 experts chosen, 231 M weights). 15 experts 5120 -> 1280,
// 13 tokens, k = 4: 46 + 28 (255 M weights). LDS is active 36 to 47% of the time in the
// larger ones: the table leaves room for two waves per SIMD, which do not cover the
// latency of the reads and of the loads.
#include "common.hpp"
#include "experts.hpp"
#include "groups.hpp"
#include "kept.hpp"
#include "launch.hpp"
#include "layer.hpp"

namespace trellis {
namespace {

constexpr int kUnitCols = 8;  // columns of h per unit: 8 gate and 8 up rows
constexpr int kChunk = 4;     // units of a wave at a time
constexpr int kUpPartFloats = 4096;  // 16 columns of 32 tokens of 8 waves
constexpr int kAhead = 2;     // operands whose codebook values are read ahead
constexpr int kHalvedTokens = 8;  // up to which both parts of h fit one operand
constexpr int kMeet = 2;      // what a meeting of units costs, in quarter rounds of blocks

// ---- the chosen experts -------------------------------------------------------

constexpr int kMaxSlots = kLayerTokens * kLayerChoices;
constexpr int kSlotsPerThread = (kMaxSlots + kExThreads - 1) / kExThreads;

struct Chosen {
    uint32_t mask[kMaxGroups];    // by expert: the tokens that chose it
    uint16_t expert[kMaxGroups];  // the chosen, ascending
};

// A thread's share of the tokens' choices, on their way from memory.
struct Slots {
    int id[kSlotsPerThread];  // -1 behind the last
};
__device__ __forceinline__ Slots load_slots(const int32_t* __restrict__ ids, int n) {
    Slots s;
#pragma unroll
    for (int i = 0; i < kSlotsPerThread; ++i) s.id[i] = ids[min(static_cast<int>(threadIdx.x) + i * kExThreads, n - 1)];
#pragma unroll
    for (int i = 0; i < kSlotsPerThread; ++i)
        if (static_cast<int>(threadIdx.x) + i * kExThreads >= n) s.id[i] = -1;
    return s;
}

// Fills `s`; every thread of the workgroup calls it. Returns the number of chosen
// experts. An id outside [0, experts) chooses none. Every wave writes the whole list
// (the same values), so that it can read it without a barrier.
// A slot's token is its number times `inverse` = ceil(2^32 / top_k), upper half (exact
// for so few; 0 stands for top_k = 1).
__device__ __forceinline__ int find_chosen(Chosen& s, const Slots& slots, uint32_t inverse, int experts) {
    const int tid = threadIdx.x, lane = tid & 63;
    for (int e = tid; e < experts; e += kExThreads) s.mask[e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSlotsPerThread; ++i)
        if (static_cast<uint32_t>(slots.id[i]) < static_cast<uint32_t>(experts))
            atomicOr(&s.mask[slots.id[i]],
                     1u << (inverse ? __umulhi(tid + i * kExThreads, inverse) : tid + i * kExThreads));
    __syncthreads();
    int n = 0;
    for (int e0 = 0; e0 < experts; e0 += kWave) {
        const bool mine = e0 + lane < experts && s.mask[e0 + lane] != 0;
        const uint64_t live = __ballot(mine);
        if (mine) s.expert[n + __popcll(live & ((1ull << lane) - 1))] = static_cast<uint16_t>(e0 + lane);
        n += __popcll(live);
    }
    wave_lds_sync();
    return n;
}

// The tokens' choices with their weights.
struct Choice {
    int id;
    float weight;
};

// A token's weight of expert e: the sum over its choices of it, ascending. Eight
// choices are read at a time, without a wait between.
__device__ __forceinline__ float weight_of(const Choice* given, int token, int top_k, int e) {
    float sum = 0.f;
    for (int k0 = 0; k0 < top_k; k0 += 8) {
        Choice v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = given[token * top_k + min(k0 + k, top_k - 1)];
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += k0 + k < top_k && v[k].id == e ? v[k].weight : 0.f;
    }
    return sum;
}

// The decode table of ExTable (the same bytes), staged by 16-byte pieces in a row:
// lanes that write both pieces of an entry, 32 bytes apart, take twice the banks' time,
// which a call of few tokens feels. Piece q is half q % 2 of codebook entry q / 2 in
// eight copies, or for k = 2 two entries of the pair table: (LUT[q / 2], LUT[2 q']) and
// (LUT[q / 2], LUT[2 q' + 1]), q' = q % 2048.
template <int K>
struct LayerTable {
    static constexpr int floats = ExTable<K>::Table::floats, n = floats / 4 / kExThreads;
    static_assert(n * 4 * kExThreads == floats && floats == 8 * kLutEntries, "whole pieces per thread");
    float a[n];
    floatx2 b[K == 2 ? 4 : 1];

    __device__ __forceinline__ void fetch(const float* lut) {
        using gf32 = const __attribute__((address_space(1))) float*;
        using gf32x2 = const __attribute__((address_space(1))) floatx2*;
        gf32 l = (gf32)lut;  // opaque, or the loads sink to their use
        asm volatile("" : "+s"(l));
#pragma unroll
        for (int i = 0; i < n; ++i) a[i] = l[threadIdx.x / 2 + kExThreads / 2 * i];
        if constexpr (K == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = reinterpret_cast<gf32x2>(l)[threadIdx.x + kExThreads * i];
        }
    }
    __device__ __forceinline__ void store(float* __restrict__ tab) const {
        floatx4* dst = reinterpret_cast<floatx4*>(tab) + threadIdx.x;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float v = a[i];
            if constexpr (K == 2) dst[kExThreads * i] = floatx4{v, b[i % 4].x, v, b[i % 4].y};
            else dst[kExThreads * i] = floatx4{v, v, v, v};
        }
    }
};

// ---- operand order of h ---------------------------------------------------------

// h of the chosen expert number `at` in the order that the down product reads:
// [chosen][piece of 32 contracted values][operand][64 lanes][8].
// Axis 0: piece s is values 32 s + 8 c ...; axis 1: piece (b, s) is values
// 256 b + 64 c + 8 s ... (c = lane / 16).
// A value is two bf16 parts. Up to kHalvedTokens tokens both are in one operand, token
// m's in rows m and m + 8; with more each 16 tokens have an operand of upper parts and
// behind it one of lower parts.
__host__ __device__ __forceinline__ int h_pieces(int inter) { return (inter + 31) / 32; }
__host__ __device__ __forceinline__ int h_operands(int tokens) {
    return tokens <= kHalvedTokens ? 1 : tokens <= 16 ? 2 : 4;
}
// From a value's upper part to its lower one.
__device__ __forceinline__ int h_lower(int tokens) { return 8 * (tokens <= kHalvedTokens ? kHalvedTokens : kWave); }

__device__ __forceinline__ size_t h_at(uint32_t at, uint32_t pieces, int operands, int axis, uint32_t col,
                                       uint32_t token) {
    const uint32_t piece = axis == 1 ? col / 256 * 8 + col % 64 / 8 : col / 32;
    const uint32_t c = axis == 1 ? col % 256 / 64 : col % 32 / 8;
    return ((static_cast<size_t>(at) * pieces + piece) * operands + token / 16 * 2) * (kWave * 8) +
           (16 * c + token % 16) * 8 + col % 8;
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
    uint32_t inverse; // ceil(2^32 / top_k)
    int per;          // units of an expert
    int strips;       // of the down product, whose arrivals start at zero
    uint32_t* arrived;
    int round, meet;  // units that meet in LDS at once, and what a chunk's meetings cost
};

__device__ __forceinline__ float h_value(float weight, float g, float u) {
    return weight * (g / (1.f + expf(-g)) * u);
}

// h enters the second product as two bf16 parts, the upper 8 bits of its mantissa (cut
// off) and the rest rounded, for any number of tokens: rounded to bf16 as a whole, it
// moved the result by about as much as the result's own rounding does (a relative error
// of 2.3e-3 for 1.7e-3), and a token's precision went by the size of its batch.
// The parts of an h that is not zero have its sign and are not zero either (2^-133 at
// least, the smallest bf16), so that an infinite weight gives the infinity that it gives h.
struct Halves {
    uint16_t upper, lower;
};
__device__ __forceinline__ Halves halves_of(float h) {
    const uint32_t bits = __float_as_uint(h);
    const float upper = __uint_as_float(bits & 0xFFFF0000u), rest = h - upper;
    const uint32_t least = (bits >> 16 & 0x8000u) | ((bits & 0x7FFFFFFFu) != 0);
    const uint32_t hi = bits >> 16, lo = __builtin_isfinite(h) ? round_bf16(rest) : hi;
    return {static_cast<uint16_t>(hi & 0x7FFFu ? hi : least), static_cast<uint16_t>(lo & 0x7FFFu ? lo : least)};
}

// How the eight waves share a workgroup's units: 2^w of them a unit's blocks, in
// teams that share the units. The fewest rounds of blocks win, in which every wave reads
// the tokens' operands of its blocks once a chunk: in quarter rounds 1, of two operands,
// which do not stay ahead, 4. us of the whole layer without and with them: 32 tokens of 3
// experts 5120 -> 5120 at k = 4 134 / 89, of one 5120 -> 17408 at k = 2 117 / 88, 16 tokens
// of 3 experts 78 / 73; 2 for two operands left one expert 5120 -> 5120 at 50 (45), 2 for
// one took 16 tokens of 64 experts from 63 to 64. Several waves to a unit pay for meeting
// in LDS (`meet` a chunk: without, the first product of 32 tokens of 64 experts 2048 ->
// 768 at k = 2 in two operands took 63 us for 54).
template <int MT>
__device__ __forceinline__ int log_ways_for(int units, int nb, int meet) {
    constexpr int reads = MT == 1 ? 1 : 4;
    int best = 0, least = INT32_MAX;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int each = (units + (kExWaves >> w) - 1) >> (3 - w);
        const int chunks = (each + kChunk - 1) / kChunk;
        const int cost = ((nb + (1 << w) - 1) >> w) * (4 * each + reads * chunks) + (w ? chunks * meet : 0);
        if (cost < least) {
            least = cost;
            best = w;
        }
    }
    return best;
}

// h of a token in a column of the chosen expert number `at`; columns behind the last are
// zeros there.
__device__ __forceinline__ void put_h(const UpArgs& p, int at, int col, int token, float v) {
    if (col >= p.inter) v = 0.f;
    uint16_t* o = p.h + h_at(at, h_pieces(p.inter), h_operands(p.tokens), p.axis_down, col, token);
    const Halves parts = halves_of(v);
    o[0] = parts.upper;
    o[h_lower(p.tokens)] = parts.lower;
}

// The choices with their weights into LDS (a barrier follows before they are read).
__device__ __forceinline__ void stage_choices(Choice* given, const Slots& slots, const UpArgs& p) {
#pragma unroll
    for (int i = 0; i < kSlotsPerThread; ++i) {
        const int s = threadIdx.x + i * kExThreads;
        if (s >= p.tokens * p.top_k) continue;
        given[s] = {slots.id[i], p.weights ? p.weights[s] : 1.f};
    }
}

// The sums of n units over a block of 256 inputs: their words and scales in registers,
// the tokens' operands in `a`. during(unit) is called when a unit's words are there and
// its first operand is multiplied, after(unit) when they are done with, and the operands
// behind the last.
template <int K, int MT, typename During, typename After>
__device__ __forceinline__ void decode_units(uint32_t (&w)[kChunk][2 * K + 1], const float (&sc)[kChunk],
                                             const u32x4 (&a)[MT][8], floatx4 (&acc)[kChunk][MT], int n,
                                             const float* tab, During&& during, After&& after) {
    constexpr bool pair = ExTable<K>::pair, rep = ExTable<K>::rep;
    constexpr int D = kAhead;
    Gathered<pair> v[D + 1];
    // operands 7 to 0: the word behind a run, its neighbour's first, is in the last
    static_for<0, D>([&](auto ic) {
        constexpr int A = decltype(ic)::value;
        v[A] = gather_tab<K, 7 - A, pair, rep>(w[0], tab);
    });
    static_for<0, kChunk>([&](auto gc) {
        constexpr int g = decltype(gc)::value;
        if (g >= n) return;
        w[g][2 * K] = next_run_word(w[g][0]);
        static_for<0, 8>([&](auto ic) {
            constexpr int I = decltype(ic)::value, S = 7 - I, A = I + D, i = 8 * g + I;
            if constexpr (A < 8) {
                v[(i + D) % (D + 1)] = gather_tab<K, 7 - A, pair, rep>(w[g], tab);
            } else if constexpr (g + 1 < kChunk) {
                if (g + 1 < n) v[(i + D) % (D + 1)] = gather_tab<K, 15 - A, pair, rep>(w[g + 1], tab);
            }
            const u32x4 f = pack_fragment(v[i % (D + 1)], sc[g]);
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[g][m] = mfma16x16x32(as_bf16x8(a[m][S]), as_bf16x8(f), acc[g][m]);
            if constexpr (I == 0) during(gc);
        });
        after(gc);
    });
}

// A unit's words of block b and its scales: its rows are a uniform address for gate and
// up plus a lane's offset.
template <int K>
__device__ __forceinline__ void load_unit(const UpArgs& p, int e, int col0, int b, uint32_t (&words)[2 * K + 1],
                                          float& scale, bool other) {  // another unit than the words' last
    const int lane = threadIdx.x & 63, j = lane & 15, c = lane >> 4;
    const uint32_t* gate = p.codes + e * p.words + block_word<K>(p.lay, col0, b);
    const uint32_t* up = gate + static_cast<uint64_t>(p.inter) * p.lay.row_words;
    const float* sg = p.scales + static_cast<size_t>(e) * (2 * p.inter) + col0;
    const int row = min(j & 7, p.inter - 1 - col0);
    load_run64_words<K>((j < 8 ? gate : up) + static_cast<uint32_t>(row) * static_cast<uint32_t>(p.lay.row_words),
                        3 - c, words);
    if (other) scale = sg[j < 8 ? row : row + p.inter];
}

// This workgroup's units. A wave takes `kChunk` units of its team at a time through
// its blocks: the tokens' operands of a block serve all of them. A unit's next words
// are loaded as soon as its last ones are decoded.
template <int K, int MT>
__global__ __launch_bounds__(kExThreads) void layer_up_kernel(UpArgs p) {
    __shared__ __attribute__((aligned(16))) float tab[LayerTable<K>::floats];
    __shared__ float parts[kUpPartFloats];
    __shared__ Chosen chosen;
    __shared__ Choice given[kMaxSlots];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, c = lane >> 4;
    const Slots slots = load_slots(p.ids, p.tokens * p.top_k);
    stage_choices(given, slots, p);
    if (blockIdx.x == 0)
        for (int i = tid; i < p.strips; i += kExThreads) p.arrived[i] = 0;
    LayerTable<K> table;
    table.fetch(p.lut);
    const int live = find_chosen(chosen, slots, p.inverse, p.experts);
    const int nb = p.hidden / kT, per = p.per, all = live * per;
    const int share = all / static_cast<int>(gridDim.x), rest = all - share * static_cast<int>(gridDim.x);
    const int u0 = static_cast<int>(blockIdx.x) * share + min(static_cast<int>(blockIdx.x), rest);
    const int units = share + (static_cast<int>(blockIdx.x) < rest);
    if (units == 0) return;
    const int round = min(kChunk, p.round);  // units that meet at once
    const int lw = log_ways_for<MT>(units, nb, p.meet), ways = 1 << lw, lt = 3 - lw;
    const int way = wave & (ways - 1), team = wave >> lw;
    auto team_first = [&](int t) { return u0 + ((units * t) >> lt); };
    const int first = team_first(team), end = team_first(team + 1);
    const int chunks = (((units + (1 << lt) - 1) >> lt) + kChunk - 1) / kChunk;

    uint32_t w[kChunk][2 * K + 1];
    float sc[kChunk];
    u32x4 a[MT][8];
    const uint16_t* x[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        x[m] = p.x + static_cast<size_t>(min(16 * m + j, p.tokens - 1)) * p.hidden + 64 * c;
    auto load_x = [&](int b, u32x4 (&o)[8], int m = 0) {
#pragma unroll
        for (int s = 0; s < 8; ++s) o[s] = *reinterpret_cast<const u32x4*>(x[m] + static_cast<size_t>(b) * kT + 8 * s);
    };
    floatx4 acc[kChunk][MT] = {};
    // the wave's place in its team's units and blocks, and unit u's expert and columns (a
    // team without a unit loads the workgroup's last, and does not use it)
    int u = first, b = min(way, nb - 1), at = first / per, in = first - at * per;
    {
        int v = min(first, u0 + units - 1), va = at, vi = in, e[kChunk], col0[kChunk];
        if (v != first) va = v / per, vi = v - va * per;
#pragma unroll
        for (int g = 0; g < kChunk; ++g) {
            e[g] = chosen.expert[va];
            col0[g] = vi * kUnitCols;
            const bool more = v + 1 < u0 + units;
            v += more;
            vi += more;
            if (vi == per) {
                vi = 0;
                ++va;
            }
        }
#pragma unroll
        for (int g = 0; g < kChunk; ++g)
            if (g == 0 || first + g < end)
                load_unit<K>(p, __builtin_amdgcn_readfirstlane(e[g]), col0[g], b, w[g], sc[g], true);
    }
    table.store(tab);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m) load_x(b, a[m], m);
    auto one = [&] {
        int nu = u, next = b + ways;
        if (next >= nb) {
            next = way;
            nu = u + kChunk;
        }
        const int n = min(kChunk, end - u);
        const bool reload = nu < end && next != b;
        int na = at, ni = in + (nu - u);
        while (ni >= per) {
            ni -= per;
            ++na;
        }
        const int next_at = na, next_in = ni;
        decode_units<K>(
            w, sc, a, acc, n, tab, [](auto) {},
            [&](auto gc) {
                constexpr int g = decltype(gc)::value;
                // the next block's operands before the last unit's words: they are waited
                // for first, and a wait is for all loads before
                if (reload && g + 1 == n) {
#pragma unroll
                    for (int m = 0; m < MT; ++m) load_x(next, a[m], m);
                }
                if (nu + g < end)
                    load_unit<K>(p, __builtin_amdgcn_readfirstlane(chosen.expert[na]), ni * kUnitCols, next, w[g],
                                 sc[g], nu != u);
                if (++ni == per) {
                    ni = 0;
                    ++na;
                }
            });
        u = nu;
        b = next;
        at = next_at;
        in = next_in;
    };
    // h of the chunk from `from` on: of a whole unit per wave from registers (lanes j
    // and j + 8 hold its gate and up; lane l the weight of token l) ...
    auto finish_alone = [&](int from) {
        int fa = from / per, fi = from - fa * per, known = -1;
        float mine = 0.f;
        uint32_t mask = 0;
#pragma unroll
        for (int g = 0; g < kChunk; ++g) {
            if (from + g >= end) break;
            if (fa != known) {
                const int e = chosen.expert[fa];
                mask = chosen.mask[e];
                mine = weight_of(given, min(lane, p.tokens - 1), p.top_k, e);
                known = fa;
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int token = 16 * m + 4 * c + i;
                    const float up = __shfl_xor(acc[g][m][i], 8), weight = __shfl(mine, token);
                    if (j < 8 && ((mask >> token) & 1))
                        put_h(p, fa, fi * kUnitCols + j, token, h_value(weight, acc[g][m][i], up));
                }
            if (++fi == per) {
                fi = 0;
                ++fa;
            }
        }
    };
    // ... or from the ways' sums in LDS, in their order.
    auto finish_together = [&](int chunk) {
        for (int r0 = 0; r0 < kChunk; r0 += round) {
#pragma unroll
            for (int g = 0; g < kChunk; ++g) {
                if (g < r0 || g >= r0 + round) continue;
                float* o = parts + ((g - r0) * kExWaves + wave) * 16 * p.tokens + j;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int token = 16 * m + 4 * c + i;
                        if (token < p.tokens) o[16 * token] = acc[g][m][i];
                    }
            }
            __syncthreads();
            const uint32_t col = tid % kUnitCols, tokens = p.tokens;
            for (uint32_t i = tid / kUnitCols; i < (round * tokens) << lt; i += kExThreads / kUnitCols) {
                const uint32_t t = i & ((1 << lt) - 1), q = (i >> lt) / tokens, token = (i >> lt) - q * tokens;
                const int unit = team_first(t) + kChunk * chunk + r0 + static_cast<int>(q);
                if (r0 + static_cast<int>(q) >= kChunk || unit >= team_first(t + 1)) continue;
                const uint32_t expert = static_cast<uint32_t>(unit) / static_cast<uint32_t>(per);
                const int e = chosen.expert[expert];
                const float* o = parts + ((q * kExWaves + (t << lw)) * tokens + token) * 16 + col;
                float gate[kExWaves], up[kExWaves];
#pragma unroll
                for (int k = 0; k < kExWaves; ++k) {
                    const uint32_t at_k = 16 * tokens * min(k, ways - 1);
                    gate[k] = o[at_k];
                    up[k] = o[at_k + 8];
                }
                const float weight = weight_of(given, token, p.top_k, e);
#pragma unroll
                for (int k = 1; k < kExWaves; ++k) {
                    gate[0] += k < ways ? gate[k] : 0.f;
                    up[0] += k < ways ? up[k] : 0.f;
                }
                if ((chosen.mask[e] >> token) & 1)
                    put_h(p, expert, (unit - expert * per) * kUnitCols + col, token, h_value(weight, gate[0], up[0]));
            }
            if (chunk + 1 < chunks || r0 + round < kChunk) __syncthreads();
        }
    };
    for (int chunk = 0; chunk < chunks; ++chunk) {
        const int from = first + kChunk * chunk;
        for (int s = way; s < nb && from < end; s += ways) one();
        if (ways == 1) finish_alone(from);
        else finish_together(chunk);
#pragma unroll
        for (int g = 0; g < kChunk; ++g)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[g][m] = floatx4{};
    }
}

// More than 16 tokens of which each expert has few: a tile is up to 16 tokens of one
// expert, one operand where all tokens would take two. A wave takes units of its own;
// none waits for another. h is stored by tokens, as the other kernel does.
struct Tiles {
    uint16_t tile[kMaxGroups + kMaxSlots / 17];  // 2 (number of the chosen expert) + (tokens 16 ...)
};

// Every wave writes the whole list, as find_chosen does.
__device__ __forceinline__ int find_tiles(Tiles& s, const Chosen& chosen, int live) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int at0 = 0; at0 < live; at0 += kWave) {
        const int at = at0 + lane, tokens = at < live ? __popc(chosen.mask[chosen.expert[at]]) : 0;
        const uint64_t one = __ballot(tokens > 0), two = __ballot(tokens > 16), below = (1ull << lane) - 1;
        const int first = n + __popcll(one & below) + __popcll(two & below);
        if (tokens > 0) s.tile[first] = static_cast<uint16_t>(2 * at);
        if (tokens > 16) s.tile[first + 1] = static_cast<uint16_t>(2 * at + 1);
        n += __popcll(one) + __popcll(two);
    }
    wave_lds_sync();
    return n;
}

// The place of the set bit number n (from 0) of a mask that has it.
__device__ __forceinline__ int set_bit(uint32_t mask, int n) {
    int at = 0;
#pragma unroll
    for (int w = 16; w; w >>= 1) {
        const int below = __popc((mask >> at) & ((1u << w) - 1u));
        if (n >= below) {
            n -= below;
            at += w;
        }
    }
    return at;
}

template <int K>
__global__ __launch_bounds__(kExThreads) void layer_up_listed_kernel(UpArgs p) {
    __shared__ __attribute__((aligned(16))) float tab[LayerTable<K>::floats];
    __shared__ Chosen chosen;
    __shared__ Tiles tiles;
    __shared__ Choice given[kMaxSlots];
    const int tid = threadIdx.x, lane = tid & 63, j = lane & 15, c = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Slots slots = load_slots(p.ids, p.tokens * p.top_k);
    stage_choices(given, slots, p);
    if (blockIdx.x == 0)
        for (int i = tid; i < p.strips; i += kExThreads) p.arrived[i] = 0;
    LayerTable<K> table;
    table.fetch(p.lut);
    const int live = find_tiles(tiles, chosen, find_chosen(chosen, slots, p.inverse, p.experts));
    table.store(tab);
    __syncthreads();
    const int nb = p.hidden / kT, per = p.per, waves = static_cast<int>(gridDim.x) * kExWaves;
    // a workgroup's waves take units far apart, so that all workgroups have as many
    const int64_t units = static_cast<int64_t>(live) * per;
    const int turn = wave * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    int u = static_cast<int>(units * turn / waves);
    const int end = static_cast<int>(units * (turn + 1) / waves);
    if (u == end) return;

    uint32_t w[kChunk][2 * K + 1];
    float sc[kChunk];
    u32x4 a[1][8];
    int at = u / per, in = u - at * per, n, e, token, rows;
    const uint16_t* x;
    // the tile of the chunk at u: its expert, rows and (lane j) the row's token
    auto enter = [&] {
        n = min(min(kChunk, end - u), per - in);
        const int tile = tiles.tile[at];
        e = __builtin_amdgcn_readfirstlane(chosen.expert[tile >> 1]);
        const uint32_t mask = chosen.mask[e];
        const int skip = 16 * (tile & 1);
        rows = min(16, __popc(mask) - skip);
        token = set_bit(mask, skip + min(j, rows - 1));
        x = p.x + static_cast<size_t>(token) * p.hidden + 64 * c;
    };
    auto load_x = [&](int b, u32x4 (&o)[8]) {
#pragma unroll
        for (int s = 0; s < 8; ++s) o[s] = *reinterpret_cast<const u32x4*>(x + static_cast<size_t>(b) * kT + 8 * s);
    };
    auto load_words = [&](auto gc, int b) {
        constexpr int g = decltype(gc)::value;
        load_unit<K>(p, e, (in + g) * kUnitCols, b, w[g], sc[g], false);
    };
    auto load_first = [&] {  // block 0 of the chunk's units
        load_x(0, a[0]);
        static_for<0, kChunk>([&](auto gc) {
            constexpr int g = decltype(gc)::value;
            if (g < n) load_unit<K>(p, e, (in + g) * kUnitCols, 0, w[g], sc[g], true);
        });
    };
    enter();
    load_first();
    // The next block's words of a unit are loaded during the unit behind it, the last one's
    // during the next block's first, and the operands ahead of both: a wait for words is
    // for every load before, as some are under conditions, and none of them is younger
    // than a unit's decoding then (the first product of 32 tokens of 64 experts 33.5 us; with
    // the loads right behind a unit, as in the kernel for fewer tokens, 37.8; that one
    // lost by this order, 49 to 56 us for 13 tokens of 15 experts 5120 -> 1280).
    for (;;) {
        floatx4 acc[kChunk][1] = {};
        for (int b = 0; b < nb; ++b) {
            const bool more = b + 1 < nb;
            u32x4 ahead[8];
            decode_units<K>(
                w, sc, a, acc, n, tab,
                [&](auto gc) {
                    constexpr int g = decltype(gc)::value;
                    if constexpr (g == 0) {
                        if (more) load_x(b + 1, ahead);
                        static_for<1, kChunk>([&](auto lc) {
                            if (b && decltype(lc)::value + 1 == n) load_words(lc, b);
                        });
                    } else if (more) {
                        load_words(std::integral_constant<int, g - 1>{}, b + 1);
                    }
                },
                [&](auto gc) {
                    if (!more || decltype(gc)::value + 1 != n) return;
#pragma unroll
                    for (int s = 0; s < 8; ++s) a[0][s] = ahead[s];
                    if (n == 1) load_words(gc, b + 1);
                });
        }
        const int done_at = tiles.tile[at] >> 1, done_in = in, done = n, done_rows = rows, done_token = token;
        const float mine = weight_of(given, token, p.top_k, e);
        u += n;
        if (u < end) {
            in += n;
            if (in == per) {
                in = 0;
                ++at;
            }
            enter();
            load_first();
        }
#pragma unroll
        for (int g = 0; g < kChunk; ++g) {
            if (g >= done) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 4 * c + i, t = __shfl(done_token, row), col = (done_in + g) * kUnitCols + j;
                const float up = __shfl_xor(acc[g][0][i], 8), weight = __shfl(mine, row);
                if (j < 8 && row < done_rows)
                    put_h(p, done_at, col, t, h_value(weight, acc[g][0][i], up));
            }
        }
        if (u == end) return;
    }
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
    uint32_t inverse;   // ceil(2^32 / top_k)
    int strips, ways;   // strips of columns, parts of the contraction
    float* partial;     // [strip][way][token][columns of a strip]
    uint32_t* arrived;  // [strip] workgroups whose part is there
    uint16_t* out;
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

// The rows of the operands that hold the tokens of a mask.
template <int P>
__device__ __forceinline__ uint32_t rows_of(uint32_t mask) {
    return P == 1 ? mask | mask << kHalvedTokens : mask;
}

// The waves' sums of a strip of COLS columns, in wave order, are the workgroup's part; a
// lane's column n is at(n). `sums` takes the table's place. The last workgroup of a strip
// to arrive adds the parts, in their order, whichever it is. Parts and arrivals are
// device-scope accesses, which no die's L2 keeps to itself, and a wave waits until its
// parts are in memory before its workgroup arrives. That order is the hardware's, not the
// language's, which has none between relaxed accesses: a device-scope store of gfx950
// writes through, vmcnt counts it until it has, and the loads behind the count pass by the
// L2. With fences instead, which write a whole L2 back, the kernel took 44 and 88 us for 1
// and 32 tokens of 64 experts where it then took 11.5 and 27; a kernel of its own for the
// sums took 2.4 to 5.3 us and the host's launch.
template <int COLS, bool HALVED, int N, int MT, typename F>
__device__ __forceinline__ void put_part(float* sums, const DownArgs& p, int strip, int way,
                                         const floatx4 (&total)[N][MT], F&& at) {
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = (tid & 63) >> 4;
    __syncthreads();  // the table is read
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (16 * m + i >= p.tokens) continue;  // nor any lane's
            const int token = 16 * m + 4 * c + i;
            float v[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                v[n] = total[n][m][i];
                if constexpr (HALVED) {  // row token + 8 is 32 lanes on
                    const uint32_t bits = __float_as_uint(v[n]);
                    v[n] += __uint_as_float(__builtin_amdgcn_permlane32_swap(bits, bits, false, false)[1]);
                }
            }
            if (token < p.tokens) {
                float* o = sums + (wave * p.tokens + token) * COLS;
#pragma unroll
                for (int n = 0; n < N; ++n) o[at(n)] = v[n];
            }
        }
    __syncthreads();
    const int n = p.tokens * COLS;
    auto sum_of = [&](int i) {
        float v[kExWaves];
#pragma unroll
        for (int w = 0; w < kExWaves; ++w) v[w] = sums[w * n + i];
#pragma unroll
        for (int w = 1; w < kExWaves; ++w) v[0] += v[w];
        return v[0];
    };
    const int col0 = strip * COLS;
    if (p.ways == 1) {
        for (int i = tid; i < n; i += kExThreads) {
            const int col = col0 + i % COLS;
            if (col < p.hidden) p.out[(i / COLS) * p.hidden + col] = round_bf16(sum_of(i));
        }
        return;
    }
    // parts in strips, two columns a word: [strip][way][token][COLS]
    uint64_t* parts = reinterpret_cast<uint64_t*>(p.partial + static_cast<size_t>(strip) * p.ways * n);
    auto pair_of = [](float a, float b) {
        return static_cast<uint64_t>(__float_as_uint(a)) | static_cast<uint64_t>(__float_as_uint(b)) << 32;
    };
    for (int i = tid; i < n / 2; i += kExThreads)
        __hip_atomic_store(parts + way * (n / 2) + i, pair_of(sum_of(2 * i), sum_of(2 * i + 1)), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    __shared__ uint32_t before;
    if (tid == 0)
        before = __hip_atomic_fetch_add(p.arrived + strip, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (before != static_cast<uint32_t>(p.ways) - 1) return;
    constexpr int kAtOnce = 16;  // a strip of 128 columns of 2048 has 16 parts
    for (int i = tid; i < n / 2; i += kExThreads) {
        float v0 = 0.f, v1 = 0.f;
        for (int w0 = 0; w0 < p.ways; w0 += kAtOnce) {
            uint64_t q[kAtOnce];
#pragma unroll
            for (int w = 0; w < kAtOnce; ++w)
                q[w] = __hip_atomic_load(parts + min(w0 + w, p.ways - 1) * (n / 2) + i, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int w = 0; w < kAtOnce; ++w) {
                const bool there = w0 + w < p.ways;
                v0 += there ? __uint_as_float(static_cast<uint32_t>(q[w])) : 0.f;
                v1 += there ? __uint_as_float(static_cast<uint32_t>(q[w] >> 32)) : 0.f;
            }
        }
        // hidden is a multiple of 256: both columns are there
        const int col = col0 + 2 * i % COLS;
        if (col < p.hidden)
            *reinterpret_cast<uint32_t*>(p.out + (2 * i / COLS) * p.hidden + col) = pack_bf16(v0, v1);
    }
}

// The tasks of this workgroup, wave by wave: load(work, at, piece, first) of the next one
// is in flight while multiply(work, next, ahead) runs, which calls ahead() for it;
// `at` numbers the chosen experts.
template <typename Work, typename Load, typename Between, typename Multiply, typename Close>
__device__ __forceinline__ void run_tasks(int first, int end, int pieces, int wave, Load&& load,
                                          Between&& between, Multiply&& multiply, Close&& close) {
    Work q[2];
    int t = first + wave, at = t / pieces;
    if (t < end) load(q[0], at, t - at * pieces, true);
    between();
    auto one = [&](Work& now, Work& next) {
        const int nt = t + kExWaves, nat = nt / pieces;
        multiply(now, next, [&] {
            if (nt < end) load(next, nat, nt - nat * pieces, false);
        });
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

// MT operands of 16 tokens, of each P: one that holds both parts of h, or one of each.
template <int K, int MT, int P>
__global__ __launch_bounds__(kExThreads) void layer_down1_kernel(DownArgs p) {
    constexpr bool pair = ExTable<K>::pair, rep = ExTable<K>::rep;
    constexpr int G = kDownGroups, N = MT * P;
    // A task's operands, four a step, are half of the registers: the next task's of a step
    // come into those that this task's leave. Fewer are held for both tasks.
    constexpr bool rolled = N == 4;
    __shared__ __attribute__((aligned(16))) float tab[LayerTable<K>::floats];
    __shared__ Chosen chosen;
    const int lane = threadIdx.x & 63, j = lane & 15, c = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Slots slots = load_slots(p.ids, p.tokens * p.top_k);
    LayerTable<K> table;
    table.fetch(p.lut);
    const int live = find_chosen(chosen, slots, p.inverse, p.experts);
    const int strip = blockIdx.x / p.ways, way = blockIdx.x % p.ways, nb = p.inter / kT;
    const int64_t tasks = static_cast<int64_t>(live) * nb;
    struct Work {
        uint32_t w[G][2 * K + 1];
        float sc[G];
        u32x4 a[rolled ? 1 : 8][N];
        const u32x4* h;
    };
    u32x4 roll[8][N];  // by steps, the last first
    auto load_step = [&](u32x4 (&a)[N], const u32x4* from, int s) {
#pragma unroll
        for (int o = 0; o < N; ++o) a[o] = from[(s * N + o) * kWave];
    };
    Sums<G, MT> sums;
    int rows[G];
#pragma unroll
    for (int g = 0; g < G; ++g) rows[g] = min(strip * kDownCols1 + 16 * g + j, p.hidden - 1);
    const u32x4* h = reinterpret_cast<const u32x4*>(p.h) + lane;
    run_tasks<Work>(
        static_cast<int>(tasks * way / p.ways), static_cast<int>(tasks * (way + 1) / p.ways), nb, wave,
        [&](Work& q, int at, int b, bool first) {
            const int e = __builtin_amdgcn_readfirstlane(chosen.expert[at]);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                load_run64_words<K>(p.codes + e * p.words + block_word<K>(p.lay, rows[g], b), 3 - c, q.w[g]);
                q.sc[g] = p.scales[static_cast<size_t>(e) * p.hidden + rows[g]];
            }
            q.h = h + (static_cast<size_t>(at) * nb + b) * 8 * N * kWave;
            if constexpr (!rolled)
                static_for<0, 8>([&](auto ic) { load_step(q.a[decltype(ic)::value], q.h, 7 - decltype(ic)::value); });
            else if (first)
                static_for<0, 8>([&](auto ic) { load_step(roll[decltype(ic)::value], q.h, 7 - decltype(ic)::value); });
        },
        [&] {
            table.store(tab);
            __syncthreads();
        },
        [&](Work& q, Work& next, auto&& ahead) {
            next.h = q.h;
            ahead();
            Gathered<pair> v[2];
            v[0] = gather_tab<K, 7, pair, rep>(q.w[0], tab);
#pragma unroll
            for (int g = 0; g < G; ++g) q.w[g][2 * K] = next_run_word(q.w[g][0]);
            static_for<0, 8 * G>([&](auto ic) {
                constexpr int i = decltype(ic)::value, S = 7 - i / G, g = i % G, n = i + 1;
                __builtin_amdgcn_s_setprio(2);
                if constexpr (n < 8 * G) v[n & 1] = gather_tab<K, 7 - n / G, pair, rep>(q.w[n % G], tab);
                __builtin_amdgcn_s_setprio(0);
                const u32x4 f = pack_fragment(v[i & 1], q.sc[g]);
                u32x4(&a)[N] = rolled ? roll[7 - S] : q.a[rolled ? 0 : 7 - S];
#pragma unroll
                for (int o = 0; o < N; ++o)
                    sums.now[g][o / P] = mfma16x16x32(as_bf16x8(a[o]), as_bf16x8(f), sums.now[g][o / P]);
                if constexpr (rolled && g + 1 == G) load_step(a, next.h, S);
            });
        },
        [&](int at) { sums.close(rows_of<P>(chosen.mask[chosen.expert[at]]), c); });
    put_part<kDownCols1, P == 1>(tab, p, strip, way, sums.total, [&](int n) { return 16 * n + j; });
}

template <int K, int MT, int P>
__global__ __launch_bounds__(kExThreads) void layer_down0_kernel(DownArgs p) {
    constexpr int CL = 8, N = MT * P;
    // With two operands of tokens the sums are half of the registers, and at k < 4 the next
    // task's operands and scales come into those that this task's leave, behind its last
    // column, its words once this task's are taken (32 tokens x 8 of 64 experts 768 -> 2048:
    // k = 2 31.6 us, but 49.6 with both tasks' held, which spills 37 registers; k = 3 34.5 /
    // 39.3 and 6; k = 4 34.6 / 33.4, where both fit).
    constexpr bool rolled = MT == 2 && K < 4;
    __shared__ __attribute__((aligned(16))) float tab[LayerTable<K>::floats];
    __shared__ Chosen chosen;
    const int lane = threadIdx.x & 63, j = lane & 15, c = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Slots slots = load_slots(p.ids, p.tokens * p.top_k);
    LayerTable<K> table;
    table.fetch(p.lut);
    const int live = find_chosen(chosen, slots, p.inverse, p.experts);
    const int strip = blockIdx.x / p.ways, way = blockIdx.x % p.ways, steps = h_pieces(p.inter);
    const int64_t tasks = static_cast<int64_t>(live) * steps;
    struct Inputs {
        float sc[8];
        u32x4 a[N];
    };
    struct None {};
    struct Work {
        Words q;
        std::conditional_t<rolled, None, Inputs> in;
        const uint16_t* h;
        const float* scales;
        int rows;  // stored rows of the step
    };
    Inputs roll;
    auto load_inputs = [&](Inputs& in, const Work& q) {
        // 8 values of a token that lie behind the last are no values at all
#pragma unroll
        for (int o = 0; o < N; ++o) in.a[o] = 8 * c < q.rows ? load_at<u32x4>(q.h + o * kWave * 8, 16 * lane) : u32x4{0u, 0u, 0u, 0u};
        if (q.rows >= 32) {
            const floatx4 lo = load_at<floatx4_a4>(q.scales, 32 * c);
            const floatx4 hi = load_at<floatx4_a4>(q.scales + 4, 32 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                in.sc[i] = lo[i];
                in.sc[4 + i] = hi[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) in.sc[i] = q.scales[min(8 * c + i, q.rows - 1)];
        }
    };
    Sums<CL, MT> sums;
    const Strip0 strip_at = strip0<K, CL>(p.codes, p.scales, p.lay, strip * kDownCols0, j, c);
    run_tasks<Work>(
        static_cast<int>(tasks * way / p.ways), static_cast<int>(tasks * (way + 1) / p.ways), steps, wave,
        [&](Work& q, int at, int step, bool first) {
            const int e = __builtin_amdgcn_readfirstlane(chosen.expert[at]);
            Strip0 s = strip_at;
            s.codes += e * p.words;
            q.scales = s.scales + static_cast<size_t>(e) * p.inter + 32 * step;
            q.rows = p.inter - 32 * step;
            q.h = p.h + (static_cast<size_t>(at) * steps + step) * (N * kWave * 8);
            if constexpr (!rolled) load_inputs(q.in, q);
            else if (first) load_inputs(roll, q);
            if (q.rows >= 32) {
                load_words(q.q, s, 32 * step);
            } else {
                const uint32_t row = static_cast<uint32_t>(32 * c * s.row_words);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = min(32 * step + 8 * c + i, p.inter - 1);
                    const uint32_t* w = s.codes + static_cast<uint64_t>(r) * s.row_words;
                    q.q.a[i] = w[(s.at_a - row) / 4];
                    q.q.b[i] = w[(s.at_b - row) / 4];
                }
            }
        },
        [&] {
            table.store(tab);
            __syncthreads();
        },
        [&](Work& q, Work& next, auto&& ahead) {
            Pieces<K, CL> ps;
            next.rows = 0;
            if constexpr (!rolled) ahead();
            ps.set(q.q, strip_at.sh);
            if constexpr (rolled) ahead();
            const int left = q.rows - 8 * c;  // of this lane's 8 rows
            auto multiply = [&](const Inputs& in) {
                ps.each(in.sc, tab, [&](auto ec, u32x4 f) {
                    constexpr int e = decltype(ec)::value;
                    if (q.rows < 32) {  // rows behind the last have no weights: theirs may be infinite
#pragma unroll
                        for (int d = 0; d < 4; ++d)
                            f[d] &= (2 * d < left ? 0xFFFFu : 0u) | (2 * d + 1 < left ? 0xFFFF0000u : 0u);
                    }
#pragma unroll
                    for (int o = 0; o < N; ++o)
                        sums.now[e][o / P] = mfma16x16x32(as_bf16x8(in.a[o]), as_bf16x8(f), sums.now[e][o / P]);
                });
            };
            if constexpr (!rolled) {
                multiply(q.in);
            } else {
                multiply(roll);
                if (next.rows) load_inputs(roll, next);
            }
        },
        [&](int at) { sums.close(rows_of<P>(chosen.mask[chosen.expert[at]]), c); });
    put_part<kDownCols0, P == 1>(tab, p, strip, way, sums.total, [&](int n) { return CL * j + n; });
}

// ---- launches ---------------------------------------------------------------------

struct LayerPlan {
    int strips, cols, ways;
    size_t arrived, partial, bytes;
};

LayerPlan layer_plan(int tokens, int top_k, int experts, int hidden, int inter, int axis_down) {
    LayerPlan p;
    p.cols = axis_down == 1 ? kDownCols1 : kDownCols0;
    p.strips = (hidden + p.cols - 1) / p.cols;
    p.ways = cu_count() / p.strips;
    if (p.ways < 1) p.ways = 1;
    const size_t chosen = tokens * top_k < experts ? tokens * top_k : experts;
    p.arrived = chosen * h_pieces(inter) * h_operands(tokens) * kWave * 16;
    p.partial = p.arrived + (static_cast<size_t>(p.strips) * sizeof(uint32_t) + 255) / 256 * 256;
    p.bytes = p.partial;
    if (p.ways > 1) p.bytes += static_cast<size_t>(p.strips) * p.ways * tokens * p.cols * sizeof(float);
    return p;
}

// More than 16 tokens as tiles where an expert has kListedTokens of them or fewer on
// average (with more it has two tiles, and is decoded twice) and the experts have more
// units than there are waves, else all tokens in two operands. The whole layer, us (tiles
// / all tokens), 32 tokens with 8 choices, 2048 -> 768 at k = 3: 64 experts (4 tokens
// each) 84 / 99, 24 experts (11 each, 2304 units) 57 / 60, 20 experts (13 each, 1920
// units) 55 / 49, 12 experts 48 / 41; 2048 -> 1024, 4 of 16 experts (8 each, 2048 units) 55 / 49;
// 5120 -> 5120, 4 experts (16 each, 2560 units) 117 / 123; one expert 5120 -> 17408 and 18
// tokens 127 / 97; but 15 experts 5120 -> 1280 (17 each, 2400 units) 116 / 122 and (13
// each) 117 / 114. Up to 16 tokens all are one operand anyway: 62 / 63 for 16 tokens of 64
// experts, but 66 / 64 for 8 tokens and 77 / 74 for 13 of 15 experts 5120 -> 1280, where
// waves that share units have more even work.
// The host does not know how many experts are chosen, so the average is over all. Where
// tokens choose alike it is wrong: 32 that all choose the same 8 of 64 experts 2048 -> 768
// have two tiles of each, and the layer takes 42 where all tokens in two operands take 34.
constexpr int kListedTokens = 16;

template <int K>
hipError_t launch_up(const UpArgs& p, hipStream_t st) {
    const int slots = p.tokens * p.top_k;
    const int64_t units = static_cast<int64_t>(slots < p.experts ? slots : p.experts) * p.per;
    const bool listed = slots <= kListedTokens * p.experts && units > cu_count() * kExWaves;
    auto kernel = p.tokens <= 16 ? layer_up_kernel<K, 1>
                  : listed       ? layer_up_listed_kernel<K>
                                 : layer_up_kernel<K, 2>;
    return launch_kernel(kernel, dim3(cu_count()), dim3(kExThreads), st, p);
}

template <int K>
hipError_t launch_down(const DownArgs& p, int axis, hipStream_t st) {
    auto kernel = axis == 1 ? layer_down1_kernel<K, 1, 1> : layer_down0_kernel<K, 1, 1>;
    if (p.tokens > 16) kernel = axis == 1 ? layer_down1_kernel<K, 2, 2> : layer_down0_kernel<K, 2, 2>;
    else if (p.tokens > kHalvedTokens) kernel = axis == 1 ? layer_down1_kernel<K, 1, 2> : layer_down0_kernel<K, 1, 2>;
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
    uint32_t* arrived = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + plan.arrived);
    float* partial = reinterpret_cast<float*>(static_cast<char*>(ws) + plan.partial);
    const uint32_t inverse = a.top_k == 1 ? 0 : static_cast<uint32_t>(((uint64_t{1} << 32) + a.top_k - 1) / a.top_k);
    // a unit's sums of eight waves: 16 columns of every token
    int round = kUpPartFloats / (kExWaves * 16 * a.tokens);
    if (round > kChunk) round = kChunk;
    const UpArgs up{a.x,     a.ids,   a.weights, a.tokens, a.top_k, u.experts, hidden,  inter,
                    d.axis,  u.codes, u.scales,  u.lut,    u.lay,   u.words,   h,       inverse,
                    (inter + kUnitCols - 1) / kUnitCols,   plan.strips,        arrived, round,
                    kMeet * ((kChunk + round - 1) / round)};
    const hipError_t e = u.k == 2   ? launch_up<2>(up, st)
                         : u.k == 3 ? launch_up<3>(up, st)
                                    : launch_up<4>(up, st);
    if (e != hipSuccess) return e;
    const DownArgs down{h,     a.ids,   a.tokens, a.top_k, d.experts,   hidden,    inter,   d.codes, d.scales,
                        d.lut, d.lay,   d.words,  inverse, plan.strips, plan.ways, partial, arrived, a.out};
    return d.k == 2   ? launch_down<2>(down, d.axis, st)
           : d.k == 3 ? launch_down<3>(down, d.axis, st)
                      : launch_down<4>(down, d.axis, st);
}

}  // namespace trellis
