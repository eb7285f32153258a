// stk_experts.hpp -- what the expert operators (route.hip, dispatch.hip,
// experts.hip, combine.hip, entry points in experts_api.hip) share: the
// element types, the launchers and their arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "stk_common.hpp"

namespace stk {

// Element types, stored as their bits.  Loads widen exactly; stores round
// once to nearest even.
struct F32 {
    using Store = float;
    static __device__ __forceinline__ float up(float v) { return v; }
    static __device__ __forceinline__ float down(float v) { return v; }
};
struct Bf16 {
    using Store = uint16_t;
    using V8 = __attribute__((ext_vector_type(8))) __bf16;
    static __device__ __forceinline__ float up(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ uint16_t down(float v)
    {
        return __builtin_bit_cast(uint16_t, (__bf16)v);
    }
};
struct F16 {
    using Store = uint16_t;
    using V8 = __attribute__((ext_vector_type(8))) _Float16;
    static __device__ __forceinline__ float up(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
    static __device__ __forceinline__ uint16_t down(float v)
    {
        return __builtin_bit_cast(uint16_t, (_Float16)v);
    }
};

// Keeps the order of a wave's LDS accesses (of different types) in the code;
// the hardware runs them in that order.
__device__ __forceinline__ void lds_order() { asm volatile("" ::: "memory"); }

// A launch holds fewer than 2^32 work-items (of more it runs the remainder,
// without an error); calls on more tokens than this go out in several (at
// most 64 lanes a token in route.hip, 256 in combine.hip).
constexpr int64_t kLaunchTokens = 1 << 23;

// Row choice (route.hip): the limits the register layouts cover.
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxK = 32;
constexpr int kRouteMaxGroups = 64;

struct RouteArgs {
    const void* z;            // [tokens][experts]
    const float* bias;        // [experts] or null
    int64_t tokens;
    int32_t experts, k, score, n_group, topk_group, group_top, renorm;
    float scale;
    float* weights;           // forward: [tokens][k]
    int32_t* chosen;          // forward: [tokens][k]
    const int32_t* chosen_in; // backward
    const float* grad_w;      // backward: [tokens][k]
    void* grad_z;             // backward: [tokens][experts]
};
hipError_t launch_route_forward(const RouteArgs& a, int dtype, hipStream_t stream);
hipError_t launch_route_backward(const RouteArgs& a, int dtype, hipStream_t stream);

struct DispatchArgs {
    const int32_t* chosen;    // [pairs]
    int32_t pairs, k, experts;
    int32_t* offsets;         // [experts + 1]
    int32_t* rows;            // [pairs]
    int32_t* slots;           // [pairs]
    uint32_t* counts;         // workspace: [experts][chunks], then [experts]
    int32_t chunks;           // 0: few pairs, no workspace
};
int32_t dispatch_chunks(int64_t pairs);
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t stream);

struct ExpertsArgs {
    const void* x;            // [tokens][K], or [pairs][K] when rows is null
    const void* w;            // [experts][M][K]
    const void* bias;         // [experts][M] or null
    const void* residual;     // [pairs][N] or null
    const int32_t* offsets;   // [experts + 1]
    const int32_t* rows;      // [pairs] or null
    const int32_t* slots;     // backward with rows: [tokens][k]
    int32_t tokens, pairs, k, experts, K, N, M, act;  // M = 2 N when gated, else N
    void* y;                  // forward: [pairs][N]
    float* z;                 // forward: [pairs][M] or null; backward: the forward's
    const void* dy;           // backward: [pairs][N]
    void* dx;                 // backward: like x, or null
    void* dw;                 // backward: like w, or null
    void* db;                 // backward: like bias, or null
    void* dz;                 // backward workspace: [pairs][M] (dy itself when act is none)
    float* dxr;               // backward workspace: [pairs][K] fp32 when rows is not null
    float* dbp;               // backward workspace: column sums by row tiles
    float* dwp;               // backward workspace: dw by shares of the rows, where there are several
};
// whether every launch of the call holds fewer than 2^32 work-items
bool experts_forward_fits(const ExpertsArgs& a);
bool experts_backward_fits(const ExpertsArgs& a);
hipError_t launch_experts_forward(const ExpertsArgs& a, int dtype, hipStream_t stream);
hipError_t launch_experts_backward(const ExpertsArgs& a, int dtype, hipStream_t stream);
hipError_t launch_experts_residual(const ExpertsArgs& a, void* dr, hipStream_t stream);  // dr: like y
int32_t experts_bias_tiles(int64_t pairs, int32_t experts);  // rows of dbp
int32_t experts_weight_shares(int64_t pairs, int32_t experts, int32_t K, int32_t M);  // of dwp, 1: none

struct CombineArgs {
    const void* y;            // [places][N]
    const float* w;           // [tokens][k] or null: all 1
    const int32_t* slots;     // [tokens][k]
    const void* residual;     // [tokens][N] or null
    int32_t tokens, k, places, N;
    int32_t keep_nan;         // forward: a NaN weight without a place counts
    void* out;                // forward: [tokens][N]
    const void* dout;         // backward: [tokens][N]
    void* dy;                 // backward: [places][N] or null
    float* dw;                // backward: [tokens][k] or null
    int32_t* kept;            // backward workspace: 64 partial counts
};
// y_f32: y holds fp32 whatever the type of out and residual.
hipError_t launch_combine_forward(const CombineArgs& a, int dtype, bool y_f32, hipStream_t stream);
hipError_t launch_combine_backward(const CombineArgs& a, int dtype, hipStream_t stream);

// Keeps a HIP status for soft_topk_last_hip_error() and returns SOFT_TOPK_EHIP.
int note_hip_error(hipError_t e);

}  // namespace stk
