// combine.hip -- the weighted sum of the experts' outputs back to the
// tokens, and its gradient.
//
// out_t = residual_t + sum_j w_tj y[slot_tj] over the choices j of token t
// with 0 <= slot_tj < places, summed in fp32 in the order of j and rounded
// once.  Backward: dy[slot_tj] = w_tj dout_t, dw_tj = <dout_t, y[slot_tj]>
// (0 for a dropped choice), and the rows of dy behind the last place are 0.
// Every place belongs to one pair, so dy is written without atomics.
// A choice without a place is left out whatever its weight; with keep_nan a
// NaN weight there counts (times a row of zeros) and the token is NaN.
//
// Bound by memory: every row of y is read once (and of dy written once).  A
// token has a group of 8 to 256 lanes, by its length, each on eight
// neighbouring columns; eight choices' rows are in flight at once.  16,384
// tokens of 8 rows of 2048 bf16: forward 105 us (5.7 TB/s), gradients 224 us
// (5.1 TB/s); through the caches (no non-temporal loads and stores) 7% more.
#include "soft_topk.h"
#include "stk_experts.hpp"
#include "stk_prof.hpp"

namespace stk {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;       // choices whose rows are in flight
constexpr int kCounters = 64;   // work-groups that count the kept choices

using V4 = __attribute__((ext_vector_type(4))) uint32_t;

// Eight neighbouring elements as they lie in memory: what is loaded where a
// choice has a place stays in this form until it is used, so that no load is
// waited for in its branch.
template <class T>
struct Eight {
    using S = typename T::Store;
    static constexpr int kPieces = 8 * sizeof(S) / 16;
    V4 u[kPieces];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
            u[j] = V4{0u, 0u, 0u, 0u};
    }
    __device__ __forceinline__ void load(const void* base, int64_t at, int count, bool whole)
    {
        const S* p = reinterpret_cast<const S*>(base) + at;
        if (whole) {
#pragma unroll
            for (int j = 0; j < kPieces; ++j)
                u[j] = __builtin_nontemporal_load(reinterpret_cast<const V4*>(p) + j);
        } else {
            S s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[i] = i < count ? p[i] : S(0);
            __builtin_memcpy(u, s, sizeof(s));
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        S s[8];
        __builtin_memcpy(s, u, sizeof(s));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = T::up(s[i]);
    }
    static __device__ __forceinline__ void store(void* base, int64_t at, const float (&v)[8], int count, bool whole)
    {
        S* p = reinterpret_cast<S*>(base) + at;
        S s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s[i] = T::down(v[i]);
        if (whole) {
            V4 w[kPieces];
            __builtin_memcpy(w, s, sizeof(s));
#pragma unroll
            for (int j = 0; j < kPieces; ++j)
                __builtin_nontemporal_store(w[j], reinterpret_cast<V4*>(p) + j);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < count)
                    p[i] = s[i];
        }
    }
};

// kWhole: rows are whole, aligned 16-byte pieces.  lanes: of a token, a power
// of two.
template <class T, class Y, bool kWhole>
__global__ __launch_bounds__(kThreads) void combine_forward_kernel(CombineArgs a, int lanes)
{
    const int64_t t = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
    if (t >= a.tokens)
        return;
    // (unsigned: the step behind the last column may pass 2^31)
    for (uint32_t n = (threadIdx.x & (lanes - 1)) * 8; n < (uint32_t)a.N; n += lanes * 8) {
        const int count = (int)(a.N - n);
        Eight<T> add;
        add.zero();
        if (a.residual)
            add.load(a.residual, t * a.N + n, count, kWhole);
        float sum[8];
        for (int j0 = 0; j0 < a.k; j0 += kBatch) {
            float w[kBatch];
            Eight<Y> y[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int32_t place = j0 + j < a.k ? a.slots[t * a.k + j0 + j] : -1;
                w[j] = 0.0f;
                y[j].zero();
                if (place >= 0 && place < a.places) {
                    w[j] = a.w ? a.w[t * a.k + j0 + j] : 1.0f;
                    y[j].load(a.y, (int64_t)place * a.N + n, count, kWhole);
                } else if (a.keep_nan && j0 + j < a.k) {
                    const float lost = a.w[t * a.k + j0 + j];
                    w[j] = lost != lost ? lost : 0.0f;  // times a row of zeros
                }
            }
            if (j0 == 0)
                add.get(sum);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                float v[8];
                y[j].get(v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum[i] = fmaf(w[j], v[i], sum[i]);
            }
        }
        Eight<T>::store(a.out, t * a.N + n, sum, count, kWhole);
    }
}

// The last kCounters work-groups count the choices that have a place.
template <class T, bool kWhole>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(CombineArgs a, int lanes, int token_groups)
{
    __shared__ float part[kBatch][kThreads / kWave];
    const int lane = lane_id();
    const int wave = threadIdx.x / kWave;
    if ((int)blockIdx.x >= token_groups) {
        const int g = blockIdx.x - token_groups;
        const int64_t pairs = (int64_t)a.tokens * a.k;
        uint32_t n = 0u;
        for (int64_t q = (int64_t)g * kThreads + threadIdx.x; q < pairs; q += kCounters * kThreads) {
            const int32_t s = a.slots[q];
            n += s >= 0 && s < a.places;
        }
        n = wave_sum_u32(n);
        uint32_t* const counts = reinterpret_cast<uint32_t*>(&part[0][0]);
        if (lane == 0)
            counts[wave] = n;
        __syncthreads();
        if (threadIdx.x == 0)
            a.kept[g] = (int32_t)(counts[0] + counts[1] + counts[2] + counts[3]);
        return;
    }
    const int64_t t = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
    const bool live = t < a.tokens;
    const int own = threadIdx.x & (lanes - 1);
    for (int j0 = 0; j0 < a.k; j0 += kBatch) {
        int32_t place[kBatch];
        float w[kBatch], dot[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            place[j] = live && j0 + j < a.k ? a.slots[t * a.k + j0 + j] : -1;
            if (place[j] >= a.places)
                place[j] = -1;
            w[j] = place[j] >= 0 ? a.w[t * a.k + j0 + j] : 0.0f;
            dot[j] = 0.0f;
        }
        for (uint32_t n = own * 8; n < (uint32_t)a.N; n += lanes * 8) {
            if (!live)
                break;
            const int count = (int)(a.N - n);
            Eight<T> raw, y[kBatch];
            raw.load(a.dout, t * a.N + n, count, kWhole);
            if (a.dw) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    y[j].zero();
                    if (place[j] >= 0)
                        y[j].load(a.y, (int64_t)place[j] * a.N + n, count, kWhole);
                }
            }
            float d[8];
            raw.get(d);
            if (a.dy) {  // needs no y: stored while those are on their way
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (place[j] >= 0) {
                        float g[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            g[i] = w[j] * d[i];
                        Eight<T>::store(a.dy, (int64_t)place[j] * a.N + n, g, count, kWhole);
                    }
            }
            if (a.dw) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    float v[8];
                    y[j].get(v);
                    if (place[j] >= 0)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            dot[j] = fmaf(d[i], v[i], dot[j]);
                }
            }
        }
        if (!a.dw)
            continue;
        // a token's lanes, then its waves, in a fixed order
        const int within = lanes < kWave ? lanes : kWave;
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            for (int off = within >> 1; off > 0; off >>= 1)
                dot[j] += __shfl_xor(dot[j], off, kWave);
        if (lanes > kWave) {
            __syncthreads();
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    part[j][wave] = dot[j];
            __syncthreads();
            const int first = threadIdx.x / lanes * (lanes / kWave);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                dot[j] = 0.0f;
                for (int v = 0; v < lanes / kWave; ++v)
                    dot[j] += part[j][first + v];
            }
        }
        if (live && own == 0)
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (j0 + j < a.k)
                    a.dw[t * a.k + j0 + j] = dot[j];
    }
}

// The rows of dy behind the kept places.
template <class T>
__global__ __launch_bounds__(kThreads) void combine_rest_kernel(CombineArgs a)
{
    using S = typename T::Store;
    const int64_t kept = (int64_t)wave_sum_u32((uint32_t)a.kept[lane_id()]);
    const int64_t end = (int64_t)a.places * a.N;
    for (int64_t i = kept * a.N + (int64_t)blockIdx.x * kThreads + threadIdx.x; i < end;
         i += (int64_t)gridDim.x * kThreads)
        reinterpret_cast<S*>(a.dy)[i] = T::down(0.0f);
}
static_assert(kCounters == kWave, "one lane reads each count");

bool pieces(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int token_lanes(int N)
{
    int lanes = 8;
    while (lanes < kThreads && lanes * 8 < N)
        lanes *= 2;
    return lanes;
}

// Tokens t .. t + tokens - 1 of a call.
template <class T>
CombineArgs part_of(const CombineArgs& a, int64_t t, int32_t tokens)
{
    const int64_t row = (int64_t)a.N * sizeof(typename T::Store);
    CombineArgs p = a;
    p.tokens = tokens;
    p.slots = a.slots + t * a.k;
    p.w = a.w ? a.w + t * a.k : nullptr;
    p.residual = a.residual ? static_cast<const char*>(a.residual) + t * row : nullptr;
    p.out = a.out ? static_cast<char*>(a.out) + t * row : nullptr;
    p.dout = a.dout ? static_cast<const char*>(a.dout) + t * row : nullptr;
    p.dw = a.dw ? a.dw + t * a.k : nullptr;
    return p;
}

template <class T, class Y>
hipError_t forward(const CombineArgs& all, hipStream_t stream)
{
    const int lanes = token_lanes(all.N), per = kThreads / lanes;
    const bool whole = all.N % 8 == 0 && pieces(all.y) && pieces(all.residual) && pieces(all.out);
    for (int64_t t = 0; t < all.tokens; t += kLaunchTokens) {
        const CombineArgs a = part_of<T>(all, t, (int32_t)(all.tokens - t < kLaunchTokens ? all.tokens - t : kLaunchTokens));
        const dim3 grid((a.tokens + per - 1) / per), block(kThreads);
        if (whole)
            STK_LAUNCH(kKCombineForward, stream, (combine_forward_kernel<T, Y, true>), grid, block, 0, stream, a, lanes);
        else
            STK_LAUNCH(kKCombineForward, stream, (combine_forward_kernel<T, Y, false>), grid, block, 0, stream, a, lanes);
    }
    return hipGetLastError();
}

template <class T>
hipError_t backward(const CombineArgs& all, hipStream_t stream)
{
    const int lanes = token_lanes(all.N), per = kThreads / lanes;
    const bool whole = all.N % 8 == 0 && pieces(all.y) && pieces(all.dout) && pieces(all.dy);
    // the choices are counted beside the tokens, or, where those take several launches, in one more
    const bool one = all.tokens <= kLaunchTokens;
    auto launch = [&](const CombineArgs& a, int groups, int counters) {
        const dim3 grid(groups + counters), block(kThreads);
        if (whole)
            STK_LAUNCH(kKCombineBackward, stream, (combine_backward_kernel<T, true>), grid, block, 0, stream, a, lanes,
                       groups);
        else
            STK_LAUNCH(kKCombineBackward, stream, (combine_backward_kernel<T, false>), grid, block, 0, stream, a, lanes,
                       groups);
    };
    for (int64_t t = 0; t < all.tokens; t += kLaunchTokens) {
        const CombineArgs a = part_of<T>(all, t, (int32_t)(all.tokens - t < kLaunchTokens ? all.tokens - t : kLaunchTokens));
        launch(a, (a.tokens + per - 1) / per, all.dy && one ? kCounters : 0);
    }
    if (all.dy && !one)
        launch(all, 0, kCounters);
    if (all.dy)
        STK_LAUNCH(kKCombineBackward, stream, (combine_rest_kernel<T>), dim3(256), dim3(kThreads), 0, stream, all);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_combine_forward(const CombineArgs& a, int dtype, bool y_f32, hipStream_t stream)
{
    if (dtype == SOFT_TOPK_F32)
        return forward<F32, F32>(a, stream);
    if (dtype == SOFT_TOPK_BF16)
        return y_f32 ? forward<Bf16, F32>(a, stream) : forward<Bf16, Bf16>(a, stream);
    return y_f32 ? forward<F16, F32>(a, stream) : forward<F16, F16>(a, stream);
}

hipError_t launch_combine_backward(const CombineArgs& a, int dtype, hipStream_t stream)
{
    if (dtype == SOFT_TOPK_F32)
        return backward<F32>(a, stream);
    if (dtype == SOFT_TOPK_BF16)
        return backward<Bf16>(a, stream);
    return backward<F16>(a, stream);
}

}  // namespace stk
