// experts_api.hip -- C entry points of the expert operators: every argument
// is checked on the host before anything is launched.
#include <math.h>
#include <string.h>

#include "soft_topk.h"
#include "stk_experts.hpp"

using namespace stk;

namespace {

constexpr int64_t kMax32 = 0x7fffffffll;

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

bool half_type(int32_t dtype) { return dtype == SOFT_TOPK_BF16 || dtype == SOFT_TOPK_F16; }
bool any_type(int32_t dtype) { return dtype == SOFT_TOPK_F32 || half_type(dtype); }
bool in_range(int64_t n) { return n >= 1 && n <= kMax32; }
bool experts_ok(int32_t experts) { return experts >= 1 && experts <= kRouteMaxExperts; }

int done(hipError_t e) { return e == hipSuccess ? SOFT_TOPK_OK : note_hip_error(e); }

bool workspace_ok(const void* p, size_t have, size_t need)
{
    return need == 0 || (p && have >= need && (reinterpret_cast<uintptr_t>(p) & 255u) == 0);
}

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool route_ok(const soft_topk_route* r, int32_t dtype, int64_t tokens, int32_t experts)
{
    if (!r || !any_type(dtype) || !in_range(tokens) || !experts_ok(experts))
        return false;
    if (r->score < SOFT_TOPK_SCORE_SOFTMAX || r->score > SOFT_TOPK_SCORE_GIVEN || !isfinite(r->scale))
        return false;
    if (r->n_group < 1 || r->n_group > kRouteMaxGroups || experts % r->n_group != 0)
        return false;
    if (r->topk_group < 1 || r->topk_group > r->n_group || (r->group_top != 1 && r->group_top != 2))
        return false;
    if (r->renormalize != 0 && r->renormalize != 1)
        return false;
    return r->k >= 1 && r->k <= kRouteMaxK && r->k <= r->topk_group * (experts / r->n_group);
}

RouteArgs route_args(const soft_topk_route* r, const void* z, int64_t tokens, int32_t experts)
{
    RouteArgs a;
    memset(&a, 0, sizeof(a));
    a.z = z;
    a.tokens = tokens;
    a.experts = experts;
    a.k = r->k;
    a.score = r->score;
    a.n_group = r->n_group;
    a.topk_group = r->topk_group;
    a.group_top = r->group_top;
    a.renorm = r->renormalize;
    a.scale = r->scale;
    return a;
}

bool dispatch_ok(int64_t tokens, int32_t k, int32_t experts)
{
    return in_range(tokens) && k >= 1 && tokens * k <= kMax32 && experts_ok(experts);
}

// The products' sizes, and that no grid of theirs leaves 31 bits (64 is the
// smallest tile; whether the launches fit is asked once they are chosen).
bool product_ok(int32_t dtype, int64_t tokens, int64_t pairs, int32_t experts, int32_t K, int32_t N, int32_t act)
{
    if (!half_type(dtype) || !in_range(tokens) || !in_range(pairs) || !experts_ok(experts) || K < 1 || N < 1)
        return false;
    if (act < SOFT_TOPK_ACT_NONE || act > SOFT_TOPK_ACT_SWIGLU)
        return false;
    const int64_t M = act == SOFT_TOPK_ACT_SWIGLU ? 2ll * N : N;
    if (M > kMax32 - 512 || K > kMax32 - 512 || pairs > kMax32 - 512)
        return false;
    const int64_t tiles = pairs / 64 + 1 + experts;
    const int64_t across = (M > K ? M : K) / 64 + 1;
    if (tiles > kMax32 / across || (M / 64 + 1) > kMax32 / (K / 64 + 1) / experts)
        return false;
    return M / 64 + 1 <= 65535;  // the second grid dimension
}

ExpertsArgs experts_args(int64_t tokens, int64_t pairs, int32_t experts, int32_t K, int32_t N, int32_t act)
{
    ExpertsArgs a;
    memset(&a, 0, sizeof(a));
    a.tokens = (int32_t)tokens;
    a.pairs = (int32_t)pairs;
    a.experts = experts;
    a.K = K;
    a.N = N;
    a.act = act;
    a.M = act == SOFT_TOPK_ACT_SWIGLU ? 2 * N : N;
    return a;
}

// dz, the fp32 gradient of every row, the bias's partial sums, dw by shares
struct BackwardPlan {
    size_t dz, dxr, dbp, dwp, total;
};

BackwardPlan backward_plan(int64_t pairs, int32_t experts, int32_t K, int32_t N, int32_t act, bool has_rows)
{
    const size_t M = act == SOFT_TOPK_ACT_SWIGLU ? 2 * (size_t)N : (size_t)N;
    BackwardPlan p;
    p.dz = 0;
    p.dxr = p.dz + up256(act == SOFT_TOPK_ACT_NONE ? 0 : (size_t)pairs * M * 2);
    p.dbp = p.dxr + up256(has_rows ? (size_t)pairs * K * 4 : 0);
    p.dwp = p.dbp + up256((size_t)experts_bias_tiles(pairs, experts) * M * 4);
    const size_t shares = (size_t)experts_weight_shares(pairs, experts, K, (int32_t)M);
    p.total = p.dwp + (shares > 1 ? up256(shares * experts * M * K * 4) : 0);
    return p;
}

}  // namespace

extern "C" {

int soft_topk_route_forward(const void* scores, int32_t dtype, int64_t tokens, int32_t experts,
                            const soft_topk_route* route, const float* bias, float* out_weights,
                            int32_t* out_experts, void* stream)
{
    if (!scores || !out_weights || !out_experts || !route_ok(route, dtype, tokens, experts))
        return SOFT_TOPK_EINVAL;
    RouteArgs a = route_args(route, scores, tokens, experts);
    a.bias = bias;
    a.weights = out_weights;
    a.chosen = out_experts;
    return done(launch_route_forward(a, dtype, static_cast<hipStream_t>(stream)));
}

int soft_topk_route_backward(const float* grad_weights, const void* scores, int32_t dtype, int64_t tokens,
                             int32_t experts, const soft_topk_route* route, const int32_t* chosen, void* grad_scores,
                             void* stream)
{
    if (!grad_weights || !scores || !chosen || !grad_scores || !route_ok(route, dtype, tokens, experts))
        return SOFT_TOPK_EINVAL;
    RouteArgs a = route_args(route, scores, tokens, experts);
    a.chosen_in = chosen;
    a.grad_w = grad_weights;
    a.grad_z = grad_scores;
    return done(launch_route_backward(a, dtype, static_cast<hipStream_t>(stream)));
}

size_t soft_topk_dispatch_workspace_bytes(int64_t tokens, int32_t k, int32_t experts)
{
    if (!dispatch_ok(tokens, k, experts))
        return 0;
    // counts by expert and chunk, and the experts' totals
    const size_t chunks = (size_t)dispatch_chunks(tokens * k);
    return chunks ? up256((chunks + 1) * experts * sizeof(uint32_t)) : 0;
}

int soft_topk_dispatch(const int32_t* chosen, int64_t tokens, int32_t k, int32_t experts, int32_t* out_offsets,
                       int32_t* out_rows, int32_t* out_slots, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!chosen || !out_offsets || !out_rows || !out_slots || !dispatch_ok(tokens, k, experts))
        return SOFT_TOPK_EINVAL;
    if (!workspace_ok(workspace, workspace_bytes, soft_topk_dispatch_workspace_bytes(tokens, k, experts)))
        return SOFT_TOPK_EWORKSPACE;
    DispatchArgs a;
    a.chosen = chosen;
    a.pairs = (int32_t)(tokens * k);
    a.k = k;
    a.experts = experts;
    a.offsets = out_offsets;
    a.rows = out_rows;
    a.slots = out_slots;
    a.counts = static_cast<uint32_t*>(workspace);
    a.chunks = dispatch_chunks(a.pairs);
    return done(launch_dispatch(a, static_cast<hipStream_t>(stream)));
}

int soft_topk_experts_forward(const void* x, const void* w, const void* bias, const void* residual, int32_t dtype,
                              const int32_t* offsets, const int32_t* rows, int64_t tokens, int64_t pairs,
                              int32_t experts, int32_t K, int32_t N, int32_t act, void* out_y, float* out_z,
                              void* stream)
{
    if (!x || !w || !offsets || !out_y || !product_ok(dtype, tokens, pairs, experts, K, N, act) ||
        (!rows && tokens != pairs) || !aligned(x, 2) || !aligned(w, 2) || !aligned(out_y, 2) || !aligned(out_z, 4))
        return SOFT_TOPK_EINVAL;
    ExpertsArgs a = experts_args(tokens, pairs, experts, K, N, act);
    a.x = x;
    a.w = w;
    a.bias = bias;
    a.residual = residual;
    a.offsets = offsets;
    a.rows = rows;
    a.y = out_y;
    a.z = out_z;
    if (!experts_forward_fits(a))
        return SOFT_TOPK_EINVAL;
    return done(launch_experts_forward(a, dtype, static_cast<hipStream_t>(stream)));
}

size_t soft_topk_experts_backward_workspace_bytes(int64_t pairs, int32_t experts, int32_t K, int32_t N, int32_t act,
                                                  int32_t has_rows)
{
    if (!product_ok(SOFT_TOPK_BF16, pairs, pairs, experts, K, N, act))
        return 0;
    return backward_plan(pairs, experts, K, N, act, has_rows != 0).total;
}

int soft_topk_experts_backward(const void* grad_y, const void* x, const void* w, const float* z, int32_t dtype,
                               const int32_t* offsets, const int32_t* rows, const int32_t* slots, int64_t tokens,
                               int64_t pairs, int32_t k, int32_t experts, int32_t K, int32_t N, int32_t act,
                               void* grad_x, void* grad_w, void* grad_bias, void* workspace, size_t workspace_bytes,
                               void* stream)
{
    if (!grad_y || !x || !w || !offsets || !product_ok(dtype, tokens, pairs, experts, K, N, act))
        return SOFT_TOPK_EINVAL;
    if ((!z && act != SOFT_TOPK_ACT_NONE) || (!rows && tokens != pairs) || k < 1 ||
        (rows && grad_x && (!slots || tokens * k != pairs)))
        return SOFT_TOPK_EINVAL;
    const BackwardPlan p = backward_plan(pairs, experts, K, N, act, rows != nullptr);
    if (!workspace_ok(workspace, workspace_bytes, p.total))
        return SOFT_TOPK_EWORKSPACE;
    char* base = static_cast<char*>(workspace);
    ExpertsArgs a = experts_args(tokens, pairs, experts, K, N, act);
    a.x = x;
    a.w = w;
    a.offsets = offsets;
    a.rows = rows;
    a.slots = slots;
    a.k = k;
    a.z = act == SOFT_TOPK_ACT_NONE ? nullptr : const_cast<float*>(z);
    a.dy = grad_y;
    a.dx = grad_x;
    a.dw = grad_w;
    a.db = grad_bias;
    a.dz = act == SOFT_TOPK_ACT_NONE ? const_cast<void*>(grad_y) : base + p.dz;
    a.dxr = rows ? reinterpret_cast<float*>(base + p.dxr) : nullptr;
    a.dbp = reinterpret_cast<float*>(base + p.dbp);
    a.dwp = reinterpret_cast<float*>(base + p.dwp);
    if (!experts_backward_fits(a))
        return SOFT_TOPK_EINVAL;
    return done(launch_experts_backward(a, dtype, static_cast<hipStream_t>(stream)));
}

int soft_topk_experts_residual_backward(const void* grad_y, int32_t dtype, const int32_t* offsets, int64_t pairs,
                                        int32_t experts, int32_t N, void* grad_residual, void* stream)
{
    if (!grad_y || !offsets || !grad_residual || !half_type(dtype) || !in_range(pairs) || !experts_ok(experts) ||
        N < 1 || !aligned(grad_y, 2) || !aligned(grad_residual, 2))
        return SOFT_TOPK_EINVAL;
    ExpertsArgs a;
    memset(&a, 0, sizeof(a));
    a.pairs = (int32_t)pairs;
    a.experts = experts;
    a.N = N;
    a.offsets = offsets;
    a.dy = grad_y;
    return done(launch_experts_residual(a, grad_residual, static_cast<hipStream_t>(stream)));
}

int soft_topk_combine_forward_ex(const void* y, const float* weights, const int32_t* slots, const void* residual,
                                 int32_t dtype, int64_t tokens, int32_t k, int64_t places, int32_t N, int32_t flags,
                                 void* out, void* stream)
{
    if (!y || !weights || !slots || !out || !any_type(dtype) || !in_range(tokens) || k < 1 || tokens * k > kMax32 ||
        !in_range(places) || N < 1 || (flags & ~SOFT_TOPK_COMBINE_KEEP_NAN))
        return SOFT_TOPK_EINVAL;
    CombineArgs a;
    memset(&a, 0, sizeof(a));
    a.y = y;
    a.w = weights;
    a.slots = slots;
    a.residual = residual;
    a.tokens = (int32_t)tokens;
    a.k = k;
    a.places = (int32_t)places;
    a.N = N;
    a.keep_nan = flags & SOFT_TOPK_COMBINE_KEEP_NAN;
    a.out = out;
    return done(launch_combine_forward(a, dtype, dtype == SOFT_TOPK_F32, static_cast<hipStream_t>(stream)));
}

int soft_topk_combine_forward(const void* y, const float* weights, const int32_t* slots, const void* residual,
                              int32_t dtype, int64_t tokens, int32_t k, int64_t places, int32_t N, void* out,
                              void* stream)
{
    return soft_topk_combine_forward_ex(y, weights, slots, residual, dtype, tokens, k, places, N, 0, out, stream);
}

int soft_topk_combine_backward(const void* grad_out, const void* y, const float* weights, const int32_t* slots,
                               int32_t dtype, int64_t tokens, int32_t k, int64_t places, int32_t N, void* grad_y,
                               float* grad_weights, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!grad_out || !y || !weights || !slots || !any_type(dtype) || !in_range(tokens) || k < 1 ||
        tokens * k > kMax32 || !in_range(places) || N < 1)
        return SOFT_TOPK_EINVAL;
    if (!workspace_ok(workspace, workspace_bytes, 256))
        return SOFT_TOPK_EWORKSPACE;
    CombineArgs a;
    memset(&a, 0, sizeof(a));
    a.y = y;
    a.w = weights;
    a.slots = slots;
    a.tokens = (int32_t)tokens;
    a.k = k;
    a.places = (int32_t)places;
    a.N = N;
    a.dout = grad_out;
    a.dy = grad_y;
    a.dw = grad_weights;
    a.kept = static_cast<int32_t*>(workspace);
    return done(launch_combine_backward(a, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
