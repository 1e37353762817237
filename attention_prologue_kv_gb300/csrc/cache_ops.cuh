// Drafted trees and caches of bounded size: arguments as the kernels take them, launches.
#pragma once

#include "attention_step.cuh"

namespace kvr {

struct TreeParams {
    const int64_t* query_start;
    const int64_t* parent;
    const int64_t* position_start;
    int64_t* mask;
    int64_t* positions;   // or NULL
    int32_t* status;
    int64_t T, N;
    int words;
};

struct KeyWeightParams {
    MlaParams m;          // lse is read, out is not used
    float* weight;
    const float* past;    // or NULL
    int64_t weight_stride, past_stride;
    float decay;
};

struct SelectParams {
    const float* weight;
    const int64_t* key_length;
    int64_t* kept;
    int64_t* kept_length;
    float* kept_weight;   // or NULL
    int32_t* status;
    int64_t weight_stride, weight_len, kept_weight_stride, kept_weight_len;
    int N, keep, sink, recent;
};

struct CompactParams {
    uint8_t* ckv;
    uint8_t* kc;
    const int64_t* table;   // NULL: Norm mode
    const int64_t* kept;
    const int64_t* kept_length;
    const int64_t* start;   // or NULL
    int32_t* status;
    int64_t N, d0, d1, max_blocks, max_keys, M;
    int cu, ku;             // units of a row in either cache
    int slices, su;         // slices of a row, units of a slice
};

cudaError_t launch_tree(const TreeParams& p, cudaStream_t s);
cudaError_t launch_key_weight_generic(const KeyWeightParams& p, int dtype, cudaStream_t s);
cudaError_t launch_key_weight_tc(const KeyWeightParams& p, int dtype, cudaStream_t s);
bool key_weight_tc_fits(const KeyWeightParams& p);           // whether its rows and work can be counted
int64_t key_weight_tc_workspace(const KeyWeightParams& p);   // bytes on the current device
cudaError_t launch_select(SelectParams p, cudaStream_t s);
cudaError_t launch_compact(CompactParams p, bool vec, cudaStream_t s);

}  // namespace kvr
