// dg_batch.h -- what api.hip and the launchers of the operators of a batch of
// different requests share: logit adjustments, routed experts, adapters.
#pragma once

#include "dg_internal.h"

namespace dg {

// Penalties, biases and masks on rows of logits (the contract of dg_adjust_rows).
struct AdjustRows {
    const void* x;
    void* y;
    int dtype;
    int64_t R, C, ld, ldy;
    dg_adjustments a;
};
hipError_t launch_adjust_rows(const AdjustRows& q, hipStream_t s);

// The router's choice (dg_moe_route), and the layer of the chosen experts (dg_moe_*).
struct MoeRoute {
    const void* x;
    int dtype;
    const float* bias;
    int32_t* ids;
    float* weights;
    int64_t M, E, ld;
    int k, score, renorm;
    float scale;
};
hipError_t launch_moe_route(const MoeRoute& r, hipStream_t s);
struct MoeLayer {
    bool q8;
    const void *Wg, *Wu, *Wd, *Xq;
    const int32_t* ids;
    const float* weights;
    void* Y;
    int ydtype;
    int64_t N, K, M, E;
    int k, act;
    void* ws;
};
size_t moe_workspace_bytes(int64_t N, int64_t K, int64_t M, int k);
hipError_t launch_moe(const MoeLayer& q, hipStream_t s);

// Low-rank adapters (dg_lora_rows).
struct LoraRows {
    const void* x;
    int dtype;
    const void *A, *B;
    int wdtype;
    const int32_t* adapter;
    const float* scale;
    const int32_t* ranks;
    const float* base;
    float* Y;
    int64_t M, N, K, R, L, ld;
    void* ws;
};
size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t R);
hipError_t launch_lora_rows(const LoraRows& q, hipStream_t s);

}  // namespace dg
