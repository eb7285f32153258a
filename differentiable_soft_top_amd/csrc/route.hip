// route.hip -- expert routing: the hard top-k of every row of scores, as a
// choice of experts with weights, and its gradient.
//
// For a token's scores z over E experts: s = softmax(z), sigmoid(z) or z
// itself; u = s + bias decides the choice (the bias balances the experts'
// load and enters nothing else); with groups, a group's score is the sum of
// its group_top best u, and only the topk_group best groups stay open; the k
// best u are chosen, ties to the lowest index; w_j = scale s_j, divided by
// the sum over the chosen when renormalised.  An expert whose score or bias
// is -inf is never chosen; a slot left over gets expert -1 and weight 0.  A
// row with a NaN or +inf score or bias gets weights NaN and experts -1.
//
// u is compared in fp64: the order of two scores that differ by less than an
// fp32 rounding is then still the order of the formula.  (Without bias and
// groups, softmax and sigmoid order as the scores themselves, which fp32
// holds exactly.)
//
// A row has G = 16, 32 or 64 lanes, R scores each in registers.  The k-th
// largest of the G lane maxima (G >= 2 k) is a lower bound of the k-th
// largest score: only scores from it on, less the error of their fp32 form,
// are candidates, a dozen for 8 of 256.  They are gathered in LDS, get
// their u in fp64 and rank themselves against one another; the rank is the
// output slot.  Groups are ranked in fp32 when their scores differ by more
// than its error.  Rows this cannot decide (more candidates than slots, two
// groups too close, more groups than lanes) go through one by one, a wave each,
// in fp64 (slow_row).  Bound by the instructions of the ranking (560 vector
// ones a wave of four rows): 65,536 x 256 bf16, k = 8, 27 us where the bytes
// take 7; with groups and a bias, 32,768 x 256, 51 us.  (A wave a row and k
// rounds of its maximum in fp64 took 148 and 127 us.)  Where every row goes
// one by one: 65,536 x 256 of equal scores 239 us, 32,768 x 256 with 32 groups
// and k = 8 194 us.
#include "soft_topk.h"
#include "stk_experts.hpp"
#include "stk_prof.hpp"

namespace stk {

namespace {

constexpr int kRouteWaves = 4;  // of a work-group
constexpr float kLowest = -3.402823466e38f;

template <class T>
__device__ __forceinline__ float load_up(const void* p, int64_t i)
{
    return T::up(reinterpret_cast<const typename T::Store*>(p)[i]);
}

// The best (value, then lowest index) over the wave; every lane gets it.
__device__ __forceinline__ void wave_best(double& v, int& i)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const double ov = __shfl_xor(v, off, kWave);
        const int oi = __shfl_xor(i, off, kWave);
        if (ov > v || (ov == v && oi < i)) {
            v = ov;
            i = oi;
        }
    }
}

// e^x for x <= 0 and sigmoid, in fp64
__device__ __forceinline__ double exp64(double x) { return exp2_nonpos(x * kLog2e); }
__device__ __forceinline__ double sigmoid64(double z)
{
    const double e = exp64(-fabs(z));
    return (z >= 0.0 ? 1.0 : e) / (1.0 + e);
}

// What each chosen score counts in the renormalised sum.  Where every chosen
// sigmoid is below e^-600 they are e^z to rounding, taken relative to the
// largest: the quotient stays exact where the scores leave the fp64 range.
__device__ __forceinline__ double renorm_part(int score, double z, double zmax)
{
    if (score == SOFT_TOPK_SCORE_SOFTMAX)
        return exp64(z - zmax);
    if (score == SOFT_TOPK_SCORE_SIGMOID)
        return zmax < -600.0 ? exp64(z - zmax) : sigmoid64(z);
    return z;
}

// ---- lanes of a row ------------------------------------------------------------

template <int kCtrl>
__device__ __forceinline__ float dpp(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, false));
}
template <int kCtrl>
__device__ __forceinline__ int dpp(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, kCtrl, 0xf, 0xf, false);
}
template <int kCtrl>
__device__ __forceinline__ double dpp(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)dpp<kCtrl>((int)(uint32_t)u), hi = (uint32_t)dpp<kCtrl>((int)(u >> 32));
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// op over the row's G lanes, given to all of them: pairs, quads, the quads of
// a half and the halves of 16 lanes, then across.
template <int G, class V, class Op>
__device__ __forceinline__ V row_all(V v, const Op& op)
{
    v = op(v, dpp<0xb1>(v));   // quad_perm 1 0 3 2
    v = op(v, dpp<0x4e>(v));   // quad_perm 2 3 0 1
    v = op(v, dpp<0x141>(v));  // row_half_mirror
    v = op(v, dpp<0x140>(v));  // row_mirror
    if (G > 16)
        v = op(v, __shfl_xor(v, 16, kWave));
    if (G > 32)
        v = op(v, __shfl_xor(v, 32, kWave));
    return v;
}
template <int G>
__device__ __forceinline__ float row_max(float v)
{
    return row_all<G>(v, [](float x, float y) { return fmaxf(x, y); });
}
template <int G>
__device__ __forceinline__ float row_min(float v)
{
    return row_all<G>(v, [](float x, float y) { return fminf(x, y); });
}
template <int G, class V>
__device__ __forceinline__ V row_sum(V v)
{
    return row_all<G>(v, [](V x, V y) { return x + y; });
}

// f(other lane's v) for every other lane of the row
template <int kFrom, class V, class F>
__device__ __forceinline__ void turn16(V v, const F& f)
{
    if constexpr (kFrom < 16) {
        f(dpp<0x120 + kFrom>(v));  // row_ror
        turn16<kFrom + 1>(v, f);
    }
}
template <int G, class V, class F>
__device__ __forceinline__ void row_others(V v, const F& f)
{
    turn16<1>(v, f);
#pragma unroll
    for (int off = 16; off < G; off += 16) {
        const V o = __shfl_xor(v, off, kWave);
        f(o);
        turn16<1>(o, f);
    }
}

// inclusive scan over the row's lanes
template <int G>
__device__ __forceinline__ int row_scan(int v)
{
    // row_shr 1, 2, 4, 8: what comes from before the 16 lanes is 0
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
    if (G > 16) {
        const int lane = lane_id() & (G - 1);
#pragma unroll
        for (int off = 16; off < G; off += 16) {
            const int o = __shfl(v, off - 1, G);  // the scan of the 16 lanes before, whole by now
            if ((lane & ~15) == off)
                v += o;
        }
    }
    return v;
}

template <int G>
__device__ __forceinline__ uint64_t row_ballot(bool b)
{
    const uint64_t m = __ballot(b);
    if (G == kWave)
        return m;
    return (m >> (lane_id() & (kWave - G))) & ((1ull << (G & 63)) - 1ull);
}

// The weight of a lane that holds a chosen score (the others: 0).  top,
// total: of the row, where the softmax is not renormalised.
template <int G>
__device__ __forceinline__ double row_weight(const RouteArgs& a, bool chosen, float zf, float top, double total)
{
    const double z = (double)zf;
    double w = 0.0;
    if (a.renorm) {
        const double zmax = (double)row_max<G>(chosen ? zf : -INFINITY);
        if (chosen)
            w = renorm_part(a.score, z, zmax);
        const double s = row_sum<G>(w);
        w = s != 0.0 ? w / s : 0.0;
    } else if (chosen) {
        if (a.score == SOFT_TOPK_SCORE_SOFTMAX)
            w = exp64(z - (double)top) / total;
        else if (a.score == SOFT_TOPK_SCORE_SIGMOID)
            w = sigmoid64(z);
        else
            w = z;
    }
    return (double)a.scale * w;
}

// One row by a whole wave, all in fp64.  u: LDS for the row's values.
// Kept small in registers, since every row's kernel reserves what it needs.
template <class T>
__device__ __noinline__ void slow_row(const RouteArgs& a, int64_t t, double* u)
{
    const int lane = lane_id();
    const int E = a.experts;
    float top = -INFINITY;
    for (int e = lane; e < E; e += kWave)
        top = fmaxf(top, load_up<T>(a.z, t * E + e));
    top = row_max<kWave>(top);
    const bool plain = !a.bias && a.n_group == 1;  // ordered by the scores themselves
    const bool softmax = a.score == SOFT_TOPK_SCORE_SOFTMAX;
    double total = 0.0;
    if (softmax) {
        for (int e = lane; e < E; e += kWave) {
            const double z = (double)load_up<T>(a.z, t * E + e);
            total += z > -INFINITY ? exp64(z - (double)top) : 0.0;
        }
        total = row_sum<kWave>(total);
    }
    for (int e = lane; e < E; e += kWave) {
        double v = (double)load_up<T>(a.z, t * E + e);
        if (v > -INFINITY) {
            if (!plain && softmax)
                v = exp64(v - (double)top) / total;
            else if (!plain && a.score == SOFT_TOPK_SCORE_SIGMOID)
                v = sigmoid64(v);
            if (a.bias)
                v += (double)a.bias[e];
        }
        u[e] = v;
    }
    lds_order();
    if (a.n_group > 1) {
        const int size = E / a.n_group;
        double score = -INFINITY, second = -INFINITY;
        if (lane < a.n_group) {
            for (int i = 0; i < size; ++i) {
                const double v = u[lane * size + i];
                if (v > score) {
                    second = score;
                    score = v;
                } else if (v > second) {
                    second = v;
                }
            }
        }
        if (a.group_top == 2 && second > -INFINITY)
            score += second;
        uint64_t open = 0;
        for (int j = 0; j < a.topk_group; ++j) {
            double v = score;
            int i = lane;
            wave_best(v, i);
            if (v > -INFINITY)
                open |= 1ull << i;
            if (lane == i)
                score = -INFINITY;
        }
        lds_order();
        for (int e = lane; e < E; e += kWave)
            if (!((open >> (e / size)) & 1ull))
                u[e] = -INFINITY;
        lds_order();
    }
    // k rounds of the wave's best; lane j keeps round j's expert
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
        double v = -INFINITY;
        int at = 0x7fffffff;
        for (int e = lane; e < E; e += kWave)
            if (u[e] > v) {
                v = u[e];
                at = e;
            }
        wave_best(v, at);
        if (!(v > -INFINITY))
            break;
        lds_order();
        if ((at & (kWave - 1)) == lane)
            u[at] = -INFINITY;
        lds_order();
        if (lane == j)
            mine = at;
    }
    const double w = row_weight<kWave>(a, mine >= 0, mine >= 0 ? load_up<T>(a.z, t * E + mine) : 0.0f, top, total);
    if (lane < a.k) {
        a.weights[t * a.k + lane] = (float)w;
        a.chosen[t * a.k + lane] = mine;
    }
    lds_order();
}

// ---- forward -------------------------------------------------------------------

// Scores R of a lane: four neighbours from every 4 G on.
template <int G>
__device__ __forceinline__ int expert_of(int r, int own)
{
    return (r / 4 * G + own) * 4 + (r & 3);
}

template <class T, int G, int R>
__device__ __forceinline__ void load_row(const void* base, int64_t at, int E, int own, bool live, bool fours,
                                         float (&z)[R])
{
    using S = typename T::Store;
    const S* const p = reinterpret_cast<const S*>(base) + at;
#pragma unroll
    for (int c = 0; c < R / 4; ++c) {
        const int e = (c * G + own) * 4;
        S s[4];
        if (live && fours && e < E) {
            __builtin_memcpy(s, __builtin_assume_aligned(p + e, 4 * sizeof(S)), sizeof(s));
#pragma unroll
            for (int v = 0; v < 4; ++v)
                z[c * 4 + v] = T::up(s[v]);
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
                z[c * 4 + v] = live && e + v < E ? T::up(p[e + v]) : -INFINITY;
        }
    }
}

// What a candidate is ranked by.  kPlain: an integer that orders by the score
// and then by the lower index; else u, ties by the index.
template <bool kPlain>
struct Candidate;
template <>
struct Candidate<true> {
    uint64_t key;
    float z;
    int e;
    __device__ __forceinline__ void rank_by(const RouteArgs&, float, double) { key = ((uint64_t)float_to_key(z) << 32) | (uint32_t)~e; }
    __device__ __forceinline__ bool beats(const Candidate& o) const { return key > o.key; }
};
template <>
struct Candidate<false> {
    double key;
    float z;
    int e;
    // (softmax without a bias: in units of the row's sum)
    __device__ __forceinline__ void rank_by(const RouteArgs& a, float top, double total)
    {
        const double x = (double)z;
        if (a.score == SOFT_TOPK_SCORE_SIGMOID)
            key = sigmoid64(x);
        else if (a.score == SOFT_TOPK_SCORE_SOFTMAX)
            key = a.bias ? exp64(x - (double)top) / total : exp64(x - (double)top);
        else
            key = x;
        if (a.bias)
            key += (double)a.bias[e];
    }
    __device__ __forceinline__ bool beats(const Candidate& o) const { return key > o.key || (key == o.key && e < o.e); }
};

// Candidate slots of a row.
template <int G>
constexpr int kSlots = G == 16 ? 32 : G;

// The two best of `values`' group `own / L`, the L lanes of the group taking
// every L-th value (from places of their own, for the banks) and joining.
template <int L>
__device__ __forceinline__ void group_best(const float* values, int group, int part, int size, int turn, float& best,
                                           float& second)
{
    best = second = -INFINITY;
    const int n = (size - part + L - 1) / L;
    int i = n > 0 ? turn % n : 0;
#pragma unroll 4
    for (int m = 0; m < n; ++m) {
        const float x = values[group * size + i * L + part];
        second = fmaxf(second, fminf(best, x));
        best = fmaxf(best, x);
        i = i + 1 == n ? 0 : i + 1;
    }
#pragma unroll
    for (int off = 1; off < L; off <<= 1) {
        const float ob = __shfl_xor(best, off, kWave), os = __shfl_xor(second, off, kWave);
        second = fmaxf(fminf(best, ob), fmaxf(second, os));
        best = fmaxf(best, ob);
    }
}

// kPlain: no bias and no groups, ordered by the scores themselves.
template <class T, int G, int R, bool kPlain>
__global__ __launch_bounds__(kRouteWaves* kWave, kPlain ? 6 : 4) void route_forward_kernel(RouteArgs a, bool fours)
{
    using Cand = Candidate<kPlain>;
    constexpr int kRows = kWave / G;  // rows of a wave
    constexpr int kPerLane = kSlots<G> / G;
    // a wave's rows of fp32 values for the groups, later its candidates; or
    // one row of fp64 for slow_row
    constexpr int kValues = kPlain ? 0 : kRows * G * R * (int)sizeof(float);
    constexpr int kCands = kRows * kSlots<G> * (int)sizeof(Cand);
    constexpr int kSlow = G * R * (int)sizeof(double);
    constexpr int kLds = kValues > kCands ? (kValues > kSlow ? kValues : kSlow) : (kCands > kSlow ? kCands : kSlow);
    __shared__ __attribute__((aligned(16))) char lds[kRouteWaves][kLds];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int own = lane & (G - 1), row = lane / G;
    const int64_t t0 = ((int64_t)blockIdx.x * kRouteWaves + wave) * kRows;
    const int64_t t = t0 + row;
    const bool live = t < a.tokens;
    const int E = a.experts;
    const bool softmax = a.score == SOFT_TOPK_SCORE_SOFTMAX, sigm = a.score == SOFT_TOPK_SCORE_SIGMOID;

    float z[R];
    load_row<T, G, R>(a.z, t * E, E, own, live, fours, z);
    float mine = -INFINITY;  // this lane's largest value
    bool bad = false;
#pragma unroll
    for (int r = 0; r < R; r += 2) {
        bad |= __builtin_isunordered(z[r], z[r + 1]);
        mine = fmaxf(mine, fmaxf(z[r], z[r + 1]));
    }
    const float top = row_max<G>(mine);
    bad |= top == INFINITY;
    double total = 0.0;
    // The weights or u need it: in fp64, so that a weight is rounded once and
    // agrees with the gradient's p (65,536 x 256 bf16: 40 us, with fp32
    // exponentials 29).
    if (softmax && (!a.renorm || (!kPlain && a.bias))) {
#pragma unroll 4
        for (int r = 0; r < R; ++r)
            total += z[r] > -INFINITY ? exp64((double)z[r] - (double)top) : 0.0;
        total = row_sum<G>(total);
    }

    // the values in fp32, and how far they may be from u
    float v[R], error = 0.0f;
    bool slow = false;
#pragma unroll
    for (int r = 0; r < R; ++r)
        v[r] = z[r];
    if constexpr (!kPlain) {
        float b[R], high = 0.0f;
        const float unit = softmax && a.bias ? (float)(1.0 / total) : 1.0f;
        if (a.bias) {
            load_row<F32, G, R>(a.bias, 0, E, own, true, fours, b);
#pragma unroll
            for (int r = 0; r < R; ++r)
                bad |= !(b[r] < INFINITY);
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r)
                b[r] = 0.0f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (sigm)
                v[r] = __builtin_amdgcn_rcpf(1.0f + __expf(-z[r]));
            else if (softmax)
                v[r] = __expf(z[r] - top) * unit;
            // (a sum below the lowest number counts as it: u, in fp64, is one)
            v[r] = fminf(z[r], b[r]) > -INFINITY ? fmaxf(v[r] + b[r], kLowest) : -INFINITY;
            high = fmaxf(high, v[r] > -INFINITY ? fabsf(v[r]) : 0.0f);
        }
        // sigmoid and exponential: below 2^-22 each (|z| e^-|z| < 0.4); the sum rounds by 2^-24 of itself
        error = (a.score == SOFT_TOPK_SCORE_GIVEN ? 0.0f : 0x1p-20f) + row_max<G>(high) * 0x1p-22f;
        bad = row_ballot<G>(bad) != 0;
        if (a.n_group > G) {
            slow = !bad;
        } else if (a.n_group > 1) {
            float* const values = reinterpret_cast<float*>(lds[wave]) + row * (G * R);
#pragma unroll
            for (int c = 0; c < R / 4; ++c)
                *reinterpret_cast<float4*>(values + (c * G + own) * 4) =
                    make_float4(v[c * 4], v[c * 4 + 1], v[c * 4 + 2], v[c * 4 + 3]);
            lds_order();
            const int size = E / a.n_group;
            const int share = a.n_group * 4 <= G ? 4 : (a.n_group * 2 <= G ? 2 : 1);  // lanes of a group
            const int group = own / share, part = own % share;
            const int from = group < a.n_group ? group : 0, turn = (group >> 1) + row * 4;
            float best, second;
            if (share == 4)
                group_best<4>(values, from, part, size, turn, best, second);
            else if (share == 2)
                group_best<2>(values, from, part, size, turn, best, second);
            else
                group_best<1>(values, from, part, size, turn, best, second);
            // one lane speaks for its group
            const bool speaks = group < a.n_group && part == 0;
            float score = a.group_top == 2 && second > -INFINITY ? fmaxf(best + second, kLowest) : best;
            score = speaks ? score : -INFINITY;
            int ahead = 0;  // groups before this one
            row_others<G>(score, [&](float o) { ahead += o > score; });
            const bool open = score > -INFINITY && ahead < a.topk_group;
            // decided where the last open and the first closed group differ by more than both errors
            const float last = row_min<G>(open ? score : INFINITY);
            const float first = row_max<G>(!open ? score : -INFINITY);
            const uint64_t mask = row_ballot<G>(open);
            if (!bad && (__popcll(mask) > a.topk_group || (first > -INFINITY && !(last - first > 6.0f * error))))
                slow = true;
            const uint32_t inverse = ((1u << 20) + (uint32_t)size - 1u) / (uint32_t)size;  // e / size for e size < 2^20
            auto closed = [&](int e) {
                const uint32_t at = ((uint32_t)e * inverse >> 20) * (uint32_t)share;
                return G > 32 ? !((mask >> (at & 63u)) & 1ull) : !(((uint32_t)mask >> (at & 31u)) & 1u);
            };
            if (size % 4 == 0) {
#pragma unroll
                for (int c = 0; c < R / 4; ++c) {
                    const bool shut = closed((c * G + own) * 4);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        v[c * 4 + r] = shut ? -INFINITY : v[c * 4 + r];
                }
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    v[r] = closed(expert_of<G>(r, own)) ? -INFINITY : v[r];
            }
            lds_order();
        }
        mine = -INFINITY;
#pragma unroll
        for (int r = 0; r < R; ++r)
            mine = fmaxf(mine, v[r]);
    } else {
        bad = row_ballot<G>(bad) != 0;
    }

    // the k-th largest lane maximum bounds the k-th largest value from below
    // (at least the lowest number: -inf is no candidate)
    int above = 0;
    row_others<G>(mine, [&](float o) { above += o > mine; });
    const float bound = fmaxf(row_min<G>(above < a.k ? mine : INFINITY) - 2.0f * error, kLowest);
    int held = 0;
#pragma unroll
    for (int r = 0; r < R; ++r)
        held += v[r] >= bound ? 1 : 0;
    const int upto = row_scan<G>(held);
    const int count = row_sum<G>(held);
    if (!bad && count > kSlots<G>)
        slow = true;
    const int all = bad || slow ? 0 : count;
    Cand* const cand = reinterpret_cast<Cand*>(lds[wave]) + row * kSlots<G>;
    if (all) {
        Cand* to = cand + (upto - held);
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (v[r] >= bound) {
                to->z = z[r];
                to->e = expert_of<G>(r, own);
                ++to;
            }
    }
    lds_order();
    Cand c[kPerLane];
    int rank[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        rank[i] = 0;
        c[i].key = 0;
        c[i].z = 0.0f;
        c[i].e = -1;
        if (own + i * G < all) {
            c[i].z = cand[own + i * G].z;
            c[i].e = cand[own + i * G].e;
            c[i].rank_by(a, top, total);
            cand[own + i * G].key = c[i].key;
        }
    }
    lds_order();
    const bool more = kPerLane > 1 && __ballot(all > G) != 0ull;  // some row of the wave has a second one a lane
#pragma unroll 4
    for (int n = 0; n < all; ++n) {
        Cand o;
        o.key = cand[n].key;
        if (!kPlain)
            o.e = cand[n].e;
        rank[0] += o.beats(c[0]);
        if (more)
            rank[kPerLane - 1] += kPerLane > 1 && o.beats(c[kPerLane - 1]);
    }
    lds_order();
    // lane j takes rank j (k <= G)
    const int chosen = all < a.k ? all : a.k;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
        if (c[i].e >= 0 && rank[i] < a.k) {
            cand[rank[i]].z = c[i].z;
            cand[rank[i]].e = c[i].e;
        }
    lds_order();
    const bool have = own < chosen;
    float zc = 0.0f;
    int e = -1;
    if (have) {
        zc = cand[own].z;
        e = cand[own].e;
    }
    const double w = row_weight<G>(a, have, zc, top, total);
    if (live && !slow && own < a.k) {
        a.weights[t * a.k + own] = bad ? NAN : (float)w;
        a.chosen[t * a.k + own] = e;
    }
    lds_order();
    for (uint64_t left = __ballot(slow && live && own == 0); left != 0ull; left &= left - 1ull)
        slow_row<T>(a, t0 + (int)__builtin_ctzll(left) / G, reinterpret_cast<double*>(lds[wave]));
}

// Gradient of the weights with respect to the scores.  With S = sum of the
// chosen and w = s / S (renormalised) or s:
//   softmax, renormalised: dz_j = w_j (g_j - sum g w);  not: dz_i = p_i (g_i - sum g p)
//   sigmoid, renormalised: dz_j = (1 - s_j) w_j (g_j - sum g w);  not: g_j s_j (1 - s_j)
//   given,   renormalised: dz_j = (g_j - sum g w) / S;  not: g_j
// times scale; g_i = 0 where i was not chosen, and only the softmax that is
// not renormalised has a gradient there.  A row without choice has none: 0,
// or NaN where its scores hold a NaN or +inf.
// The row is put together in LDS and written once: 32,768 x 256 fp32 10 us,
// 3.3 TB/s of writes; the softmax that is not renormalised, which takes an
// fp64 exponential of every score, 65,536 x 256 bf16 34 us (22 in fp32, whose
// sum and p do not agree: 1 - sum p of the chosen is lost below 1e-8).
template <class T, int G, int R>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_backward_kernel(RouteArgs a, bool fours)
{
    constexpr int kRows = kWave / G;
    __shared__ __attribute__((aligned(16))) float lds[kRouteWaves][kRows][G * R];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int own = lane & (G - 1), row = lane / G;
    const int64_t t = ((int64_t)blockIdx.x * kRouteWaves + wave) * kRows + row;
    const bool live = t < a.tokens;
    const int E = a.experts;
    float* const out = lds[wave][row];
    int e = -1;
    double g = 0.0, z = -INFINITY;
    if (live && own < a.k) {
        e = a.chosen_in[t * a.k + own];
        if (e < 0 || e >= E)
            e = -1;
        if (e >= 0) {
            g = (double)a.scale * (double)a.grad_w[t * a.k + own];
            z = (double)load_up<T>(a.z, t * E + e);
        }
    }
    const bool any = row_ballot<G>(e >= 0) != 0;
    // a row without choice may be one that is not finite
    bool bad = false;
    if (__ballot(live && !any) != 0ull) {
        float v[R];
        load_row<T, G, R>(a.z, t * E, E, own, live && !any, fours, v);
#pragma unroll
        for (int r = 0; r < R; ++r)
            bad |= !(v[r] < INFINITY);
        bad = row_ballot<G>(bad) != 0;
    }
    const bool whole = a.score == SOFT_TOPK_SCORE_SOFTMAX && !a.renorm;
    double p = 0.0, dz = 0.0, spread = 0.0;
    if (whole) {
        // fp64 all along: g - spread cancels where the chosen hold nearly all of the row, and the sum has to be
        // that of the very p it is formed with
        float v[R], top = -INFINITY;
        load_row<T, G, R>(a.z, t * E, E, own, live, fours, v);
#pragma unroll
        for (int r = 0; r < R; ++r)
            top = fmaxf(top, v[r]);
        top = row_max<G>(top);
        double part[R], sum = 0.0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            part[r] = any && v[r] > -INFINITY ? exp64((double)v[r] - (double)top) : 0.0;
            sum += part[r];
        }
        sum = row_sum<G>(sum);
        p = e >= 0 ? exp64(z - (double)top) / sum : 0.0;
        spread = row_sum<G>(g * p);
        dz = p * (g - spread);
        const double f = any ? -spread / sum : 0.0;
#pragma unroll
        for (int c = 0; c < R / 4; ++c)
            *reinterpret_cast<float4*>(out + (c * G + own) * 4) =
                make_float4((float)(part[c * 4] * f), (float)(part[c * 4 + 1] * f), (float)(part[c * 4 + 2] * f),
                            (float)(part[c * 4 + 3] * f));
    } else {
#pragma unroll
        for (int c = 0; c < R / 4; ++c)
            *reinterpret_cast<float4*>(out + (c * G + own) * 4) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (a.renorm) {
            const double zmax = (double)row_max<G>((float)z);  // z is a float
            const double part = e >= 0 ? renorm_part(a.score, z, zmax) : 0.0;
            const double s = row_sum<G>(part);
            const double w = s != 0.0 ? part / s : 0.0;
            dz = g - row_sum<G>(g * w);
            if (a.score == SOFT_TOPK_SCORE_GIVEN)
                dz = s != 0.0 ? dz / s : 0.0;
            else
                dz *= w;
        } else {
            dz = g;
        }
        if (a.score == SOFT_TOPK_SCORE_SIGMOID) {
            dz *= sigmoid64(-z);  // 1 - s
            if (!a.renorm)
                dz *= sigmoid64(z);
        }
    }
    // an expert named twice: its first lane writes the sum
    if (e < 0)
        dz = 0.0;
    double mine = dz;
    bool first = e >= 0;
    for (int j = 0; j < a.k; ++j) {
        const int oe = __shfl(e, j, G);
        if (row_ballot<G>(oe == e && e >= 0 && j != own) == 0)
            continue;
        const double od = __shfl(dz, j, G);
        if (oe == e && e >= 0 && j != own) {
            first &= j > own;
            mine += whole ? od + p * spread : od;
        }
    }
    lds_order();
    if (first)
        out[e] = (float)mine;
    if (bad) {
#pragma unroll
        for (int c = 0; c < R / 4; ++c)
            *reinterpret_cast<float4*>(out + (c * G + own) * 4) = make_float4(NAN, NAN, NAN, NAN);
    }
    lds_order();
    if (!live)
        return;
    using S = typename T::Store;
    S* const to = reinterpret_cast<S*>(a.grad_z) + t * E;
#pragma unroll
    for (int c = 0; c < R / 4; ++c) {
        const int i = (c * G + own) * 4;
        const float4 q = *reinterpret_cast<const float4*>(out + i);
        const S s[4] = {T::down(q.x), T::down(q.y), T::down(q.z), T::down(q.w)};
        if (fours && i < E) {
            __builtin_memcpy(__builtin_assume_aligned(to + i, 4 * sizeof(S)), s, sizeof(s));
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (i + v < E)
                    to[i + v] = s[v];
        }
    }
}

template <class T, int G, int R>
void route_launch(const RouteArgs& a, bool forward, bool fours, hipStream_t stream)
{
    constexpr int kRows = kRouteWaves * kWave / G;
    const dim3 grid((unsigned)((a.tokens + kRows - 1) / kRows)), block(kRouteWaves * kWave);
    if (forward && !a.bias && a.n_group == 1)
        STK_LAUNCH(kKRouteForward, stream, (route_forward_kernel<T, G, R, true>), grid, block, 0, stream, a, fours);
    else if (forward)
        STK_LAUNCH(kKRouteForward, stream, (route_forward_kernel<T, G, R, false>), grid, block, 0, stream, a, fours);
    else
        STK_LAUNCH(kKRouteBackward, stream, (route_backward_kernel<T, G, R>), grid, block, 0, stream, a, fours);
}

// G at least twice k (the bound by lane maxima then leaves few candidates)
// and large enough for 16 scores a lane.
template <class T, int G>
void route_by_size(const RouteArgs& a, bool forward, bool fours, hipStream_t stream)
{
    if (a.experts <= G * 4)
        route_launch<T, G, 4>(a, forward, fours, stream);
    else if (a.experts <= G * 8)
        route_launch<T, G, 8>(a, forward, fours, stream);
    else
        route_launch<T, G, 16>(a, forward, fours, stream);
}

template <class T>
void route_typed(const RouteArgs& a, bool forward, hipStream_t stream)
{
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.z) | reinterpret_cast<uintptr_t>(a.grad_z);
    const bool fours = a.experts % 4 == 0 && base % (4 * sizeof(typename T::Store)) == 0 &&
                       reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    if (a.k <= 8 && a.experts <= 256)
        route_by_size<T, 16>(a, forward, fours, stream);
    else if (a.k <= 16 && a.experts <= 512)
        route_by_size<T, 32>(a, forward, fours, stream);
    else
        route_by_size<T, 64>(a, forward, fours, stream);
}

hipError_t route_by_type(const RouteArgs& a, int dtype, bool forward, hipStream_t stream)
{
    const int64_t row = (int64_t)a.experts * (dtype == SOFT_TOPK_F32 ? 4 : 2);  // bytes
    for (int64_t t = 0; t < a.tokens; t += kLaunchTokens) {
        RouteArgs part = a;
        part.tokens = a.tokens - t < kLaunchTokens ? a.tokens - t : kLaunchTokens;
        part.z = static_cast<const char*>(a.z) + t * row;
        if (forward) {
            part.weights = a.weights + t * a.k;
            part.chosen = a.chosen + t * a.k;
        } else {
            part.chosen_in = a.chosen_in + t * a.k;
            part.grad_w = a.grad_w + t * a.k;
            part.grad_z = static_cast<char*>(a.grad_z) + t * row;
        }
        if (dtype == SOFT_TOPK_F32)
            route_typed<F32>(part, forward, stream);
        else if (dtype == SOFT_TOPK_BF16)
            route_typed<Bf16>(part, forward, stream);
        else
            route_typed<F16>(part, forward, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_route_forward(const RouteArgs& a, int dtype, hipStream_t stream)
{
    return route_by_type(a, dtype, true, stream);
}

hipError_t launch_route_backward(const RouteArgs& a, int dtype, hipStream_t stream)
{
    return route_by_type(a, dtype, false, stream);
}

}  // namespace stk
