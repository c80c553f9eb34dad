// C-ABI entry points around an MLP or a layer of experts (trellis_mlp.h): argument
// validation on the host, then launches on the caller's stream.
#include <stdint.h>

#include "checks.hpp"
#include "kept.hpp"
#include "launch.hpp"
#include "layer.hpp"
#include "trellis_mlp.h"

using trellis::aligned;
using trellis::status_of;

static_assert(trellis::kLayerTokens == TRELLIS_MAX_MLP_TOKENS, "the header's limit");
static_assert(trellis::kLayerChoices == TRELLIS_MAX_MLP_CHOICES, "the header's limit");

namespace {

struct LayerDims {
    trellis::Dims up, down;
    int hidden, inter;
};

int check_layer(int32_t tokens, int32_t top_k, int32_t experts, const trellis_expert_set* up,
                const trellis_expert_set* down, LayerDims* d) {
    if (!up || !down) return TRELLIS_ERR_NULL;
    int st;
    if ((st = trellis::check_geometry(&up->g, &d->up)) || (st = trellis::check_geometry(&down->g, &d->down)))
        return st;
    d->hidden = up->g.in_features;
    d->inter = down->g.in_features;
    if (up->g.axis != 1 || up->g.out_features != 2 * d->inter || down->g.out_features != d->hidden ||
        tokens < 0 || tokens > TRELLIS_MAX_MLP_TOKENS || top_k < 1 || top_k > TRELLIS_MAX_MLP_CHOICES ||
        experts < 1 || experts > TRELLIS_MAX_GROUPS)
        return TRELLIS_ERR_GEOMETRY;
    return TRELLIS_OK;
}

trellis::ExpertWeights weights_of(const trellis_expert_set* s, const trellis::Dims& d, int32_t experts) {
    const size_t words = static_cast<size_t>(d.rows) * d.nb * 8 * s->g.k;
    return {s->codes, s->scales, s->lut, d.lay, words, s->g.axis, s->g.k, s->g.in_features,
            s->g.out_features, experts};
}

int check_rows(int32_t rows, int32_t most, int32_t width) {
    if (rows < 0 || rows > most || width < 1 || width > trellis::kMaxFeatures) return TRELLIS_ERR_GEOMETRY;
    const int64_t padded = (static_cast<int64_t>(width) + 31) / 32 * 32;
    return rows * padded > TRELLIS_MAX_KEPT_VALUES ? TRELLIS_ERR_GEOMETRY : TRELLIS_OK;
}

// Rows [g, u] and what is kept of them, [2 rows][inter].
int check_halves(int32_t rows, int32_t inter) {
    if (rows < 0 || rows > TRELLIS_MAX_SLOTS || inter > trellis::kMaxFeatures / 2) return TRELLIS_ERR_GEOMETRY;
    return check_rows(2 * rows, 2 * TRELLIS_MAX_SLOTS, inter);
}

int check_kept(const trellis_kept* k) {
    return !k || !k->codes || !k->exponents ? TRELLIS_ERR_NULL : TRELLIS_OK;
}

trellis::KeptRows rows_of(const trellis_kept* k) { return {k->codes, k->exponents}; }

}  // namespace

extern "C" {

size_t trellis_experts_mlp_workspace_bytes(int32_t tokens, int32_t top_k, int32_t experts,
                                           const trellis_expert_set* up,
                                           const trellis_expert_set* down) {
    LayerDims d;
    if (check_layer(tokens, top_k, experts, up, down, &d)) return static_cast<size_t>(-1);
    return tokens ? trellis::layer_workspace_bytes(tokens, top_k, experts, d.hidden, d.inter, down->g.axis) : 0;
}

int trellis_experts_mlp(const uint16_t* x, const int32_t* ids, const float* weights, int32_t tokens,
                        int32_t top_k, int32_t experts, const trellis_expert_set* up,
                        const trellis_expert_set* down, uint16_t* out, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
    LayerDims d;
    int st = check_layer(tokens, top_k, experts, up, down, &d);
    if (st) return st;
    if (tokens == 0) return TRELLIS_OK;
    if (!ids) return TRELLIS_ERR_NULL;
    if ((st = trellis::check_operands(up->codes, up->scales, up->lut)) ||
        (st = trellis::check_operands(down->codes, down->scales, down->lut)) ||
        (st = trellis::check_io(x, out)))
        return st;
    if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(workspace, 16)) return TRELLIS_ERR_ALIGN;
    if (!workspace ||
        workspace_bytes < trellis_experts_mlp_workspace_bytes(tokens, top_k, experts, up, down))
        return TRELLIS_ERR_WORKSPACE;
    const trellis::LayerArgs a{x,
                               ids,
                               weights,
                               tokens,
                               top_k,
                               weights_of(up, d.up, experts),
                               weights_of(down, d.down, experts),
                               out};
    return status_of(trellis::launch_layer(a, workspace, stream));
}

int trellis_keep(const uint16_t* x, int32_t rows, int32_t width, const trellis_kept* kept,
                 hipStream_t stream) {
    int st = check_rows(rows, TRELLIS_MAX_KEPT_ROWS, width);
    if (st) return st;
    if (rows == 0) return TRELLIS_OK;
    if (!x || check_kept(kept)) return TRELLIS_ERR_NULL;
    if (!aligned(x, 2)) return TRELLIS_ERR_ALIGN;
    return status_of(trellis::launch_keep(x, rows, width, kept->codes, kept->exponents, stream));
}

int trellis_restore(const trellis_kept* kept, int32_t rows, int32_t width, uint16_t* out,
                    hipStream_t stream) {
    int st = check_rows(rows, TRELLIS_MAX_KEPT_ROWS, width);
    if (st) return st;
    if (rows == 0) return TRELLIS_OK;
    if (!out || check_kept(kept)) return TRELLIS_ERR_NULL;
    if (!aligned(out, 2)) return TRELLIS_ERR_ALIGN;
    return status_of(trellis::launch_restore(rows_of(kept), rows, width, out, stream));
}

int trellis_swiglu(const uint16_t* gu, int32_t rows, int32_t inter, uint16_t* h,
                   const trellis_kept* kept, hipStream_t stream) {
    int st = check_halves(rows, inter);
    if (st) return st;
    if (rows == 0) return TRELLIS_OK;
    if (!gu || !h || (kept && check_kept(kept))) return TRELLIS_ERR_NULL;
    if (!aligned(gu, 2) || !aligned(h, 2)) return TRELLIS_ERR_ALIGN;
    return status_of(trellis::launch_swiglu(gu, rows, inter, h, kept ? kept->codes : nullptr,
                                            kept ? kept->exponents : nullptr, stream));
}

int trellis_swiglu_backward(const uint16_t* dh, const uint16_t* gu, const trellis_kept* kept,
                            int32_t rows, int32_t inter, uint16_t* dgu, uint16_t* h,
                            hipStream_t stream) {
    int st = check_halves(rows, inter);
    if (st) return st;
    if (gu && kept) return TRELLIS_ERR_GEOMETRY;
    if (rows == 0) return TRELLIS_OK;
    if (!dh || !dgu || (!gu && check_kept(kept))) return TRELLIS_ERR_NULL;
    if (!aligned(dh, 2) || !aligned(gu, 2) || !aligned(dgu, 2) || !aligned(h, 2)) return TRELLIS_ERR_ALIGN;
    return status_of(trellis::launch_swiglu_backward(
        dh, gu, kept ? rows_of(kept) : trellis::KeptRows{nullptr, nullptr}, rows, inter, dgu, h, stream));
}

}  // extern "C"
