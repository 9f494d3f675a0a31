// moe.cuh -- host-side launchers of the mixture-of-experts training kernels (moe.cu).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace bsq {

constexpr int kRouteMaxExperts = 1024;  // the grouped GEMM's bound on groups
constexpr int kRouteMaxTopk = 32;       // one slot per lane of a warp

// Byte offsets of the router's workspace (moe.cu explains its use).
struct RouteWorkspace {
    int64_t nchunk, hist, prefix, psum, count, psum_block, bytes;
};
RouteWorkspace route_workspace(int64_t T, int64_t E);

struct RouteArgs {
    const void *logits;
    bool bf16;
    int64_t T, E, ldl;
    const uint8_t *mask;
    int topk;
    bool renorm;
    int32_t *ids;
    float *weights;
    int32_t *rows, *row_index, *row_off, *sf_row_off, *counts;
    float *prob_sums;  // NULL: not asked for
    float coef;
    float *loss;  // NULL: not asked for
    uint8_t *ws;
};
// Non-zero if a launch failed.
int launch_moe_route(const RouteArgs &a, int num_sms, cudaStream_t s);

struct RouteBwdArgs {
    const void *logits;
    bool bf16;
    int64_t T, E, ldl;
    int topk;
    bool renorm;
    const int32_t *ids;
    const float *weights, *dweights;
    const int32_t *counts;
    float coef;
    const float *dloss;
    void *dlogits;
    int64_t ldd;
};
int launch_moe_route_bwd(const RouteBwdArgs &a, int num_sms, cudaStream_t s);

int launch_moe_combine(const uint16_t *y, int64_t R, int64_t H, int64_t ldy, const int32_t *rows, const float *weights,
                       int64_t T, int topk, uint16_t *out, int64_t ldo, cudaStream_t s);
// y as bf16, or (y NULL) as MXFP8 codes with swizzled scales.
int launch_moe_combine_bwd(const uint16_t *dout, int64_t ldo, const uint16_t *y, int64_t ldy, const uint8_t *codes,
                           const uint8_t *sf, int64_t R, int64_t H, const int32_t *rows, const float *weights,
                           int64_t T, int topk, uint16_t *dy, int64_t lddy, float *dweights, cudaStream_t s);

// amax may be NULL.
int launch_swiglu_ckpt(const uint16_t *u, int64_t M, int64_t F, int64_t ldu, const int32_t *n_rows, uint16_t *h,
                       int64_t ldh, uint8_t *codes, uint8_t *sf, unsigned int *amax, cudaStream_t s);
int launch_swiglu_ckpt_bwd(const uint16_t *dh, int64_t lddh, const uint8_t *codes, const uint8_t *sf, int64_t M,
                           int64_t F, const int32_t *n_rows, uint16_t *du, int64_t lddu, uint16_t *h, int64_t ldh,
                           cudaStream_t s);

}  // namespace bsq
