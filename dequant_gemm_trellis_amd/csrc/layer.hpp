// Launcher of a whole layer of experts for few tokens (layer.hip; internal to
// libtrellis.so, callers have validated arguments).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "groups.hpp"

namespace trellis {

constexpr int kLayerTokens = 32;   // at most: two 16-row operands
constexpr int kLayerChoices = 32;  // per token, at most

struct LayerArgs {
    const uint16_t* x;     // [tokens][hidden]
    const int32_t* ids;    // [tokens][top_k]
    const float* weights;  // the same, or null (ones)
    int tokens, top_k;
    ExpertWeights up;      // axis 1, hidden -> 2 inter: gate rows, then up rows
    ExpertWeights down;    // inter -> hidden
    uint16_t* out;         // [tokens][hidden]
};

size_t layer_workspace_bytes(int tokens, int top_k, int experts, int hidden, int inter, int axis_down);
hipError_t launch_layer(const LayerArgs& a, void* ws, hipStream_t st);

}  // namespace trellis
