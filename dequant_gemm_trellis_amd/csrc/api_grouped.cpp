// C-ABI entry points of the grouped operations (trellis_grouped.h): argument
// validation on the host, then launches on the caller's stream.
#include <stdint.h>

#include "checks.hpp"
#include "groups.hpp"
#include "launch.hpp"
#include "trellis_grouped.h"

using trellis::aligned;
using trellis::status_of;

static_assert(trellis::kMaxGroups == TRELLIS_MAX_GROUPS, "the header's limit");
static_assert(trellis::kMaxSlots == TRELLIS_MAX_SLOTS, "the header's limit");
static_assert(trellis::kMaxRank == TRELLIS_MAX_RANK, "the header's limit");

namespace {

constexpr int32_t kMaxWidth = 1 << 19;

// tokens x top_k slots of rows of `width` values.
int check_slots(int32_t tokens, int32_t top_k) {
    if (tokens < 0 || top_k < 1) return TRELLIS_ERR_GEOMETRY;
    if (static_cast<int64_t>(tokens) * top_k > TRELLIS_MAX_SLOTS) return TRELLIS_ERR_GEOMETRY;
    return TRELLIS_OK;
}

int check_moves(int32_t tokens, int32_t top_k, int32_t width) {
    if (width < 1 || width > kMaxWidth) return TRELLIS_ERR_GEOMETRY;
    return check_slots(tokens, top_k);
}

int check_groups(int32_t groups) {
    return groups < 1 || groups > trellis::kMaxGroups ? TRELLIS_ERR_GEOMETRY : TRELLIS_OK;
}

// The sizes of an adapter set and of the rows it is applied to.
int check_adapters(const trellis_adapter_set* f, int32_t rows) {
    if (!f) return TRELLIS_ERR_NULL;
    if (check_groups(f->count) || f->rank < 1 || f->rank > TRELLIS_MAX_RANK ||
        f->in_features < 1 || f->in_features > kMaxWidth || f->out_features < 1 ||
        f->out_features > kMaxWidth || rows < 0 || rows > TRELLIS_MAX_ADAPTER_ROWS)
        return TRELLIS_ERR_GEOMETRY;
    return TRELLIS_OK;
}

int check_factors(const trellis_adapter_set* f) {
    if (!f->a || !f->b || !f->scales) return TRELLIS_ERR_NULL;
    if (!aligned(f->a, 2) || !aligned(f->b, 2) || !aligned(f->scales, 4)) return TRELLIS_ERR_ALIGN;
    return TRELLIS_OK;
}

trellis::AdapterFactors factors(const trellis_adapter_set* f) {
    return {f->a, f->b, f->scales, f->in_features, f->out_features, f->rank, f->count};
}

bool all16(const void* p, const void* q, const void* r) {
    return aligned(p, 16) && aligned(q, 16) && aligned(r, 16);
}

int check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (!aligned(workspace, 16)) return TRELLIS_ERR_ALIGN;
    return need && (!workspace || bytes < need) ? TRELLIS_ERR_WORKSPACE : TRELLIS_OK;
}

}  // namespace

extern "C" {

size_t trellis_route_workspace_bytes(int32_t tokens, int32_t top_k, int32_t groups) {
    if (check_slots(tokens, top_k) || check_groups(groups)) return static_cast<size_t>(-1);
    return trellis::route_workspace_bytes(tokens * top_k, groups);
}

int trellis_route(const int32_t* ids, int32_t tokens, int32_t top_k, int32_t groups,
                  int32_t* offsets, int32_t* order, int32_t* position, void* workspace,
                  size_t workspace_bytes, hipStream_t stream) {
    int st = check_slots(tokens, top_k);
    if (st || (st = check_groups(groups))) return st;
    const int slots = tokens * top_k;
    if (!offsets || (slots && (!ids || !order || !position))) return TRELLIS_ERR_NULL;
    if (!aligned(offsets, 4) || !aligned(ids, 4) || !aligned(order, 4) || !aligned(position, 4))
        return TRELLIS_ERR_ALIGN;
    if ((st = check_workspace(workspace, workspace_bytes,
                              trellis::route_workspace_bytes(slots, groups))))
        return st;
    return status_of(trellis::launch_route(ids, slots, groups, false, offsets, order, position,
                                           static_cast<int32_t*>(workspace), stream));
}

int trellis_dispatch(const uint16_t* x, const int32_t* position, int32_t tokens, int32_t top_k,
                     int32_t width, uint16_t* out, hipStream_t stream) {
    const int st = check_moves(tokens, top_k, width);
    if (st) return st;
    if (tokens == 0) return TRELLIS_OK;
    if (!x || !position || !out) return TRELLIS_ERR_NULL;
    if (!aligned(x, 2) || !aligned(position, 4) || !aligned(out, 2)) return TRELLIS_ERR_ALIGN;
    const bool vec = width % 8 == 0 && aligned(x, 16) && aligned(out, 16);
    return status_of(trellis::launch_dispatch(x, position, tokens, top_k, width, out, vec, stream));
}

int trellis_combine(const uint16_t* y, const float* weights, const int32_t* position,
                    int32_t tokens, int32_t top_k, int32_t width, uint16_t* out,
                    hipStream_t stream) {
    const int st = check_moves(tokens, top_k, width);
    if (st) return st;
    if (tokens == 0) return TRELLIS_OK;
    if (!y || !position || !out) return TRELLIS_ERR_NULL;
    if (!aligned(y, 2) || !aligned(weights, 4) || !aligned(position, 4) || !aligned(out, 2))
        return TRELLIS_ERR_ALIGN;
    const bool vec = width % 8 == 0 && aligned(y, 16) && aligned(out, 16);
    return status_of(trellis::launch_combine(y, weights, position, tokens, top_k, width, out, vec,
                                             stream));
}

int trellis_combine_backward(const uint16_t* dout, const uint16_t* y, const float* weights,
                             const int32_t* position, int32_t tokens, int32_t top_k,
                             int32_t width, uint16_t* dy, float* dweights, hipStream_t stream) {
    const int st = check_moves(tokens, top_k, width);
    if (st) return st;
    if (tokens == 0) return TRELLIS_OK;
    if (!dout || !y || !weights || !position || !dy || !dweights) return TRELLIS_ERR_NULL;
    if (!aligned(dout, 2) || !aligned(y, 2) || !aligned(weights, 4) || !aligned(position, 4) ||
        !aligned(dy, 2) || !aligned(dweights, 4))
        return TRELLIS_ERR_ALIGN;
    const bool vec = width % 8 == 0 && aligned(dout, 16) && aligned(y, 16) && aligned(dy, 16);
    return status_of(trellis::launch_combine_backward(dout, y, weights, position, tokens, top_k,
                                                      width, dy, dweights, vec, stream));
}

size_t trellis_adapters_workspace_bytes(const trellis_adapter_set* f, int32_t rows,
                                        int32_t backward) {
    if (check_adapters(f, rows)) return static_cast<size_t>(-1);
    return trellis::adapters_workspace_bytes(rows, f->in_features, f->out_features, f->rank,
                                             f->count, backward != 0);
}

int trellis_adapters(const uint16_t* x, const int32_t* ids, int32_t rows,
                     const trellis_adapter_set* f, const uint16_t* base, uint16_t* y, float* u,
                     void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int st = check_adapters(f, rows);
    if (st) return st;
    if (rows == 0) return TRELLIS_OK;
    if (!x || !ids || !y) return TRELLIS_ERR_NULL;
    if ((st = check_factors(f))) return st;
    if (!aligned(x, 2) || !aligned(ids, 4) || !aligned(base, 2) || !aligned(y, 2) || !aligned(u, 4))
        return TRELLIS_ERR_ALIGN;
    if ((st = check_workspace(workspace, workspace_bytes,
                              trellis_adapters_workspace_bytes(f, rows, 0))))
        return st;
    const bool vec_in = f->in_features % 8 == 0 && all16(x, f->a, nullptr);
    const bool vec_out = f->out_features % 8 == 0 && all16(base, y, f->b);
    return status_of(trellis::launch_adapters(x, ids, factors(f), rows, base, y, u, vec_in, vec_out,
                                              workspace, stream));
}

int trellis_adapters_backward(const uint16_t* dy, const uint16_t* x, const float* u,
                              const int32_t* ids, int32_t rows, const trellis_adapter_set* f,
                              const uint16_t* base, uint16_t* dx, uint16_t* da, uint16_t* db,
                              void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int st = check_adapters(f, rows);
    if (st) return st;
    if (!da || !db || (rows && (!dy || !x || !u || !ids || !dx))) return TRELLIS_ERR_NULL;
    if ((st = check_factors(f))) return st;
    if (!aligned(dy, 2) || !aligned(x, 2) || !aligned(u, 4) || !aligned(ids, 4) ||
        !aligned(base, 2) || !aligned(dx, 2) || !aligned(da, 2) || !aligned(db, 2))
        return TRELLIS_ERR_ALIGN;
    if ((st = check_workspace(workspace, workspace_bytes,
                              trellis_adapters_workspace_bytes(f, rows, 1))))
        return st;
    const bool vec_in = f->in_features % 8 == 0 && all16(x, f->a, base) && all16(dx, da, nullptr);
    const bool vec_out = f->out_features % 8 == 0 && all16(dy, f->b, db);
    return status_of(trellis::launch_adapters_backward(dy, x, u, ids, factors(f), rows, base, dx, da,
                                                       db, vec_in, vec_out, workspace, stream));
}

size_t trellis_experts_workspace_bytes(const trellis_geometry* g, int32_t rows, int32_t experts) {
    trellis::Dims d;
    if (trellis::check_geometry(g, &d) || check_groups(experts) || check_slots(rows, 1))
        return static_cast<size_t>(-1);
    return rows ? trellis::experts_workspace_bytes(g->axis, g->in_features, g->out_features, rows, experts) : 0;
}

int trellis_experts(const uint16_t* x, int32_t rows, const int32_t* offsets, int32_t experts,
                    const uint32_t* codes, const float* scales, const float* lut,
                    const trellis_geometry* g, uint16_t* y, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
    trellis::Dims d;
    int st = trellis::check_geometry(g, &d);
    if (st || (st = check_groups(experts)) || (st = check_slots(rows, 1))) return st;
    if (rows == 0) return TRELLIS_OK;
    if (!offsets) return TRELLIS_ERR_NULL;
    if ((st = trellis::check_operands(codes, scales, lut)) || (st = trellis::check_io(x, y))) return st;
    if (!aligned(offsets, 4)) return TRELLIS_ERR_ALIGN;
    if ((st = check_workspace(workspace, workspace_bytes,
                              trellis_experts_workspace_bytes(g, rows, experts))))
        return st;
    const size_t words = static_cast<size_t>(d.rows) * d.nb * 8 * g->k;
    const trellis::ExpertWeights w{codes,  scales, lut, d.lay, words, g->axis, g->k,
                                   g->in_features, g->out_features, experts};
    return status_of(trellis::launch_experts(x, rows, offsets, w, y, workspace, stream));
}

}  // extern "C"
