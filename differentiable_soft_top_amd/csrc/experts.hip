// experts.hip -- the experts' products: rows of x, in the order of their
// experts, times their expert's weights, with bias, activation and residual
// in the epilogue; and its gradient.
//
// Row r of expert e (offsets[e] <= r < offsets[e + 1]), source s = rows[r]
// (r itself without rows):
//   z_r = W_e x_s + b_e;  y_r = act(z_r) + residual_r
// act: none, silu z s(z), gelu z Phi(z) (exact, by erfc), or swiglu, whose W_e
// has 2 N rows: y = silu(z[:N]) z[N:].  Backward, with dz = dy act'(z):
//   dx_s = sum over the places of s of W_e^T dz_r;  dW_e = sum_r dz_r x_s^T;
//   db_e = sum_r dz_r
// One group and no rows make it a dense layer.  Rows behind offsets[E] give
// 0.  Sums are fp32; z is kept in fp32, dz is rounded to the element type
// once because the matrix cores take it so.
//
// Every product runs as output tiles of 16x16x32 matrix instructions.  The
// first operand ("P") is the one whose index is contiguous in the output, so
// a lane's four results are four neighbours in memory; the second ("Q") is
// the output's row.  An operand lies in memory either with the summed index
// contiguous (tiles [row][64] in LDS, read as 16-byte fragments) or with its
// own index contiguous (tiles [64][column], read through the transposing
// LDS load).
#include "soft_topk.h"
#include "stk_experts.hpp"
#include "stk_prof.hpp"

namespace stk {

namespace {

constexpr int kBK = 64;  // summed index per step
using V4F = __attribute__((ext_vector_type(4))) float;
using V4S = __attribute__((ext_vector_type(4))) short;
using V8S = __attribute__((ext_vector_type(8))) short;

__device__ __forceinline__ V4F mma(V8S p, V8S q, V4F c, Bf16)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(Bf16::V8, p), __builtin_bit_cast(Bf16::V8, q), c,
                                                   0, 0, 0);
}
__device__ __forceinline__ V4F mma(V8S p, V8S q, V4F c, F16)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(F16::V8, p), __builtin_bit_cast(F16::V8, q), c, 0,
                                                  0, 0);
}

// ---- where a row tile lies -------------------------------------------------

// The experts' row tiles, counted by every wave for itself: lane l sums the
// tiles of its run of experts, a wave scan makes them places.  Offsets that
// fall may name more tiles than a launch has row tiles: a lane's are cut at
// kMostTiles (a launch has fewer), so that the sums stay in 32 bits, and the
// kernels take no more than they have.
constexpr int kMostTiles = 1 << 24;
struct Tiles {
    int per, mine, upto, total;  // experts per lane; this lane's tiles; up to and with it; all
    int start, end;              // rows of this lane's first expert
    int behind;                  // offsets[experts]
};

__device__ __forceinline__ int clamp_row(int32_t v, int pairs) { return v < 0 ? 0 : (v > pairs ? pairs : v); }

__device__ __forceinline__ int tiles_of(int start, int end, int rows)
{
    return end > start ? (end - start + rows - 1) / rows : 0;
}

__device__ __forceinline__ int expert_tiles(const ExpertsArgs& a, int e, int rows)
{
    return tiles_of(clamp_row(a.offsets[e], a.pairs), clamp_row(a.offsets[e + 1], a.pairs), rows);
}

__device__ __forceinline__ Tiles count_tiles(const ExpertsArgs& a, int rows)
{
    Tiles t;
    const int lane = lane_id();
    t.per = (a.experts + kWave - 1) / kWave;
    t.behind = clamp_row(a.offsets[a.experts], a.pairs);
    const int first = lane * t.per < a.experts ? lane * t.per : a.experts;
    const int next = first < a.experts ? first + 1 : a.experts;
    t.start = clamp_row(a.offsets[first], a.pairs);
    t.end = clamp_row(a.offsets[next], a.pairs);
    t.mine = tiles_of(t.start, t.end, rows);
    for (int i = 1; i < t.per; ++i)
        if (first + i < a.experts)
            t.mine += expert_tiles(a, first + i, rows);
    t.mine = t.mine < kMostTiles ? t.mine : kMostTiles;
    t.upto = t.mine;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int o = __shfl_up(t.upto, off, kWave);
        if (lane >= off)
            t.upto += o;
    }
    t.total = __builtin_amdgcn_readlane(t.upto, kWave - 1);
    return t;
}

// The row tiles that this launch of `across` columns works on: all of them,
// unless the offsets fall.
__device__ __forceinline__ int launched_tiles(const Tiles& t, int across)
{
    const int most = (int)gridDim.x / across;
    return t.total < most ? t.total : most;
}

// The expert that holds row tile `tile` (below t.total), the first of its row
// tiles, and its rows.
__device__ __forceinline__ void find_expert(const ExpertsArgs& a, const Tiles& t, int tile, int rows, int& e, int& first,
                                            int& start, int& end)
{
    const uint64_t past = __ballot(t.upto > tile);
    const int lane = (int)__builtin_ctzll(past);
    first = __builtin_amdgcn_readlane(t.upto - t.mine, lane);
    start = __builtin_amdgcn_readlane(t.start, lane);
    end = __builtin_amdgcn_readlane(t.end, lane);
    e = lane * t.per;
    while (tile >= first + tiles_of(start, end, rows)) {
        first += tiles_of(start, end, rows);
        ++e;
        start = clamp_row(a.offsets[e], a.pairs);
        end = clamp_row(a.offsets[e + 1], a.pairs);
    }
}

// Place `at` of `down` x `across` tiles, taken 8 rows of tiles at a time,
// column by column: the 32 tiles an XCD works on at once are then 8 x 4 (or
// 4 x 8 where there are 4 rows), which share 12 operand panels among 64
// loads, where 1 x 32 share 33.  Measured at 8192^3: half of the L2 requests
// missed in row order.
template <int kRows = 8>
__device__ __forceinline__ void tile_place(int at, int down, int across, int& i, int& j)
{
    const int group = at / (kRows * across);
    const int rows = down - group * kRows < kRows ? down - group * kRows : kRows;
    const int in = at - group * kRows * across;
    i = group * kRows + in % rows;
    j = in / rows;
}

// Expert, rows and column tile of an output tile.
__device__ __forceinline__ void find_tile(const ExpertsArgs& a, const Tiles& t, int tile, int across, int rows, int& e,
                                          int& row0, int& end, int& column)
{
    int first, i;
    find_expert(a, t, tile / across, rows, e, first, row0, end);
    tile_place(tile - first * across, tiles_of(row0, end, rows), across, i, column);
    row0 += i * rows;
}

// Work-groups go to the 8 XCDs in turn; neighbouring tiles, which share
// operands, belong on one XCD behind one L2.
__device__ __forceinline__ int xcd_order(int id, int total)
{
    const int q = total / 8, r = total % 8, x = id % 8;
    return x * q + (x < r ? x : r) + id / 8;
}

// The same in runs of 8 tiles; the tiles behind the last whole 64 in turn.
__device__ __forceinline__ int xcd_eights(int id, int total)
{
    return id < total / 64 * 64 ? (id / 64 * 8 + id % 8) * 8 + id / 8 % 8 : id;
}

// ---- operands ----------------------------------------------------------------

// 8 elements from p, of which `valid` exist (the others 0)
__device__ __forceinline__ V8S load8(const uint16_t* p, int valid)
{
    V8S v = {0, 0, 0, 0, 0, 0, 0, 0};
    if (valid >= 8) {
        __builtin_memcpy(&v, p, 16);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < valid)
                v[j] = (short)p[j];
    }
    return v;
}

// A team of kT threads works on a tile's steps (Shape); this thread in it.
template <int kT>
__device__ __forceinline__ int own_thread()
{
    return (int)threadIdx.x & (kT - 1);
}

// A tile of kRows rows with the summed index contiguous: LDS [kRows][64],
// its 16-byte chunks permuted in each row by the row's number, so that the
// 16 rows of a fragment lie in different banks.
template <int kRows, int kT>
struct RowTile {
    static constexpr int kBytes = kRows * kBK * 2;
    static constexpr int kLoads = kRows * 8 / kT;
    static constexpr int kReads = 1;  // LDS reads of a fragment
    const uint16_t* base;
    const uint16_t* p[kLoads];  // null: a row of zeros
    int c;

    static __device__ __forceinline__ int row_of(int i) { return i * (kT / 8) + own_thread<kT>() / 8; }
    __device__ __forceinline__ void start(const void* q)
    {
        base = reinterpret_cast<const uint16_t*>(q);
        c = (own_thread<kT>() & 7) ^ ((row_of(0) >> 1) & 7);
    }
    // row i of this thread begins `elements` from the base (negative: zeros)
    __device__ __forceinline__ void set(int i, int64_t elements) { p[i] = elements < 0 ? nullptr : base + elements; }
    __device__ __forceinline__ void fetch(int step, int sum, V8S* v) const
    {
        const int k = step * kBK + c * 8;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            v[i] = load8(p[i] + k, p[i] ? sum - k : 0);
    }
    static __device__ __forceinline__ void put(char* lds, const V8S* v)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            *reinterpret_cast<V8S*>(lds + (i * kT + own_thread<kT>()) * 16) = v[i];
    }
    // the fragment of rows r0 .. r0 + 15, half kk of the step
    static __device__ __forceinline__ V8S frag(const char* lds, int r0, int kk)
    {
        const int lane = lane_id();
        const int row = r0 + (lane & 15);
        const int ch = (kk * 4 + (lane >> 4)) ^ ((row >> 1) & 7);
        return *reinterpret_cast<const V8S*>(lds + row * 128 + ch * 16);
    }
};

// A tile of kCols columns whose own index is contiguous: LDS [64][kCols],
// its 32-byte granules permuted by the row's low bits, so that the eight
// rows of a transposing load lie in different banks.
template <int kCols, int kT>
struct ColTile {
    static constexpr int kBytes = kCols * kBK * 2;
    static constexpr int kPerRow = kCols / 8;
    static constexpr int kLoads = kBK * kPerRow / kT;
    static constexpr int kReads = 2;

    static __device__ __forceinline__ int row_of(int i) { return (i * kT + own_thread<kT>()) / kPerRow; }
    static_assert(kCols >= 64, "four granules a row");
    // (64 columns: two rows share the banks, their four granules each)
    static __device__ __forceinline__ int mix(int row)
    {
        return kCols == 64 ? ((row >> 1) & 1) | (((row >> 3) & 1) << 1) : (row & 3) | (((row >> 3) & 1) << 2);
    }
    // first column of chunk i of this thread
    static __device__ __forceinline__ int col_of(int i)
    {
        const int ch = (i * kT + own_thread<kT>()) % kPerRow;
        return ((((ch >> 1) ^ mix(row_of(i))) << 1) | (ch & 1)) * 8;
    }
    static __device__ __forceinline__ void put(char* lds, const V8S* v)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            *reinterpret_cast<V8S*>(lds + (i * kT + own_thread<kT>()) * 16) = v[i];
    }
    // the fragment of columns c0 .. c0 + 15, half kk of the step
    static __device__ __forceinline__ V8S frag(const char* lds, int c0, int kk)
    {
        const int lane = lane_id();
        const int i = lane & 15, g = lane >> 4;
        const int row = kk * 32 + g * 8 + (i >> 2);
        const int at = row * (kCols * 2) + (((c0 >> 4) ^ mix(row)) << 5) + (i & 3) * 8;  // mix(row + 4) is the same
        using Lds = __attribute__((address_space(3))) V4S;
        const V4S lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)(lds + at));
        const V4S hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)(lds + at + 4 * kCols * 2));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// ---- loads that go from memory into LDS without registers ----------------------
//
// Taken where every 16-byte chunk of a row is whole and aligned.  A load is
// an offset below 2^32 from a base in scalar registers, which moves on by a
// step; an offset of kNone lies behind the buffer's end and loads zeros
// (behind the summed index, or a row without source).
constexpr uint32_t kNone = 0xffffffffu;
constexpr uint32_t kBufferEnd = 0xfffffff0u;
using V4U = __attribute__((ext_vector_type(4))) uint32_t;

// Buffer resource at p: no stride, kBufferEnd bytes, raw 32-bit data.
__device__ __forceinline__ V4U buffer_at(const char* p)
{
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    V4U r;
    r.x = __builtin_amdgcn_readfirstlane((uint32_t)u);
    r.y = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32) & 0xffffu);
    r.z = kBufferEnd;
    r.w = 0x00020000u;
    return r;
}

// 16 bytes a lane for each offset, to lds + lane * 16 and every kStride bytes
// on.  Written out so that the compiler does not wait for the loads before the
// next LDS read: step_barrier() does, once.  They return nothing in registers.
// The five wait states are those a vector memory instruction needs behind a
// vector one that wrote its scalars, which the compiler cannot keep inside the
// text; m0 needs one.
template <int kStride>
__device__ __forceinline__ void load_lds(V4U buffer, const uint32_t (&offset)[2], uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %3, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds"
                 :
                 : "s"(lds), "v"(offset[0]), "v"(offset[1]), "s"(buffer), "i"(kStride)
                 : "memory", "m0", "scc");
}
template <int kStride>
__device__ __forceinline__ void load_lds(V4U buffer, const uint32_t (&offset)[4], uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %5, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %6\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %5, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %6\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %5, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %6\n\ts_nop 0\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
                 :
                 : "s"(lds), "v"(offset[0]), "v"(offset[1]), "v"(offset[2]), "v"(offset[3]), "s"(buffer), "i"(kStride)
                 : "memory", "m0", "scc");
}

__device__ __forceinline__ uint32_t lds_address(const char* p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

template <int kRows, int kT>
struct RowLoad {
    using Tile = RowTile<kRows, kT>;
    static constexpr int kLoads = Tile::kLoads;
    const char* base;
    uint32_t at[kLoads];
    int c;

    __device__ __forceinline__ void start(const void* p)
    {
        base = reinterpret_cast<const char*>(p);
        c = (own_thread<kT>() & 7) ^ ((Tile::row_of(0) >> 1) & 7);
    }
    // row i of this thread begins `elements` from the base (negative: zeros)
    __device__ __forceinline__ void set(int i, int64_t elements)
    {
        at[i] = elements < 0 ? kNone : (uint32_t)(elements * 2 + c * 16);
    }
    __device__ __forceinline__ void issue(const char* lds, int step, int sum) const
    {
        const V4U buffer = buffer_at(base + (int64_t)step * (kBK * 2));
        const bool in = step * kBK + c * 8 < sum;
        const uint32_t to = __builtin_amdgcn_readfirstlane(lds_address(lds) + own_thread<kT>() / kWave * (kWave * 16));
        uint32_t from[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            from[i] = in ? at[i] : kNone;
        load_lds<kT * 16>(buffer, from, to);
    }
};

// Columns c0 .. c0 + kCols - 1 of rows of `ld` elements.  The chunks of a
// thread lie kRows rows apart in one column.
template <int kCols, int kT>
struct ColLoad {
    using Tile = ColTile<kCols, kT>;
    static constexpr int kLoads = Tile::kLoads;
    static constexpr int kRows = kT / Tile::kPerRow;
    static_assert(kRows % 16 == 0, "the column permutation repeats every 16 rows");
    const char* base;
    uint32_t ld;   // bytes
    int row;       // of chunk 0
    uint32_t col;  // bytes

    __device__ __forceinline__ void start(const void* p, int elements, int c0, int cols)
    {
        base = reinterpret_cast<const char*>(p);
        ld = (uint32_t)elements * 2u;
        row = Tile::row_of(0);
        const int c = c0 + Tile::col_of(0);
        col = (uint32_t)(c < cols ? c : cols - 8) * 2u;  // columns behind the last are not stored
    }
    // rows first .. first + 63 of the matrix, zeros behind the first `left` of them
    __device__ __forceinline__ void issue(const char* lds, int64_t first, int left) const
    {
        const V4U buffer = buffer_at(base + first * (int64_t)ld);
        const uint32_t to = __builtin_amdgcn_readfirstlane(lds_address(lds) + own_thread<kT>() / kWave * (kWave * 16));
        const uint32_t at = (uint32_t)row * ld + col;
        uint32_t from[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            from[i] = row < left - i * kRows ? at + (uint32_t)(i * kRows) * ld : kNone;
        load_lds<kT * 16>(buffer, from, to);
    }
    // the rows named, zeros where one is not in [0, end)
    __device__ __forceinline__ void issue_rows(const char* lds, const int (&rows)[kLoads], int end) const
    {
        const V4U buffer = buffer_at(base);
        const uint32_t to = __builtin_amdgcn_readfirstlane(lds_address(lds) + own_thread<kT>() / kWave * (kWave * 16));
        uint32_t from[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            from[i] = (uint32_t)rows[i] < (uint32_t)end ? (uint32_t)rows[i] * ld + col : kNone;
        load_lds<kT * 16>(buffer, from, to);
    }
};

// Every load of this wave has arrived, and every wave is here: what was
// loaded can be read, and what was read before can be overwritten.
__device__ __forceinline__ void step_barrier()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Half a step's fragments of a wave, and their products.
template <class TP, class TQ, int kFP, int kFQ>
struct Half {
    V8S p[kFP], q[kFQ];
    static constexpr int kReads = kFP * TP::kReads + kFQ * TQ::kReads, kMma = kFP * kFQ;

    __device__ __forceinline__ void read(const char* lds, int p0, int q0, int kk)
    {
#pragma unroll
        for (int i = 0; i < kFQ; ++i)
            q[i] = TQ::frag(lds + TP::kBytes, q0 + i * 16, kk);
#pragma unroll
        for (int i = 0; i < kFP; ++i)
            p[i] = TP::frag(lds, p0 + i * 16, kk);
    }
    template <class T>
    __device__ __forceinline__ void multiply(V4F (&acc)[kFP][kFQ]) const
    {
#pragma unroll
        for (int i = 0; i < kFP; ++i)
#pragma unroll
            for (int j = 0; j < kFQ; ++j)
                acc[i][j] = mma(p[i], q[j], acc[i][j], T{});
    }
    // issue order: a read behind every kGap products
    static __device__ __forceinline__ void interleave()
    {
        constexpr int kGap = kMma / kReads > 1 ? kMma / kReads : 1;
#pragma unroll
        for (int i = 0; i < kReads; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, kGap, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        if constexpr (kMma > kReads * kGap)
            __builtin_amdgcn_sched_group_barrier(0x008, kMma - kReads * kGap, 0);
    }
};

// All steps of a tile, two steps' operands in LDS.  `issue(at, s)` starts the
// loads of step s.  A half's fragments are read while the other half's
// products run, so a wave has products to issue on both sides of the one
// barrier of a step, behind which the step's buffer is loaded anew.
// A wave whose part of the tile lies behind the last row or column (`busy`
// false) only loads: the others have the matrix cores to themselves.
template <class T, class TP, class TQ, int kFP, int kFQ, class Issue>
__device__ __forceinline__ void direct_steps(char* lds, int steps, int p0, int q0, bool busy, V4F (&acc)[kFP][kFQ],
                                             const Issue& issue)
{
    constexpr int kStep = TP::kBytes + TQ::kBytes;
    using H = Half<TP, TQ, kFP, kFQ>;
    H first, second;
    issue(lds, 0);
    step_barrier();
    if (steps > 1)
        issue(lds + kStep, 1);
    if (!busy) {
        for (int s = 0; s + 1 < steps; ++s) {
            step_barrier();
            if (s + 2 < steps)
                issue(lds + (s & 1) * kStep, s + 2);
        }
        return;
    }
    first.read(lds, p0, q0, 0);
    for (int s = 0; s + 1 < steps; ++s) {
        char* const now = lds + (s & 1) * kStep;
        char* const next = lds + (~s & 1) * kStep;
        second.read(now, p0, q0, 1);
        first.template multiply<T>(acc);
        H::interleave();
        step_barrier();
        if (s + 2 < steps)
            issue(now, s + 2);
        first.read(next, p0, q0, 0);
        second.template multiply<T>(acc);
        H::interleave();
    }
    second.read(lds + (~steps & 1) * kStep, p0, q0, 1);
    first.template multiply<T>(acc);
    second.template multiply<T>(acc);
}

// One step's products, for tiles that come through registers.
template <class T, class TP, class TQ, int kFP, int kFQ>
__device__ __forceinline__ void step_mma(const char* lds, int p0, int q0, V4F (&acc)[kFP][kFQ])
{
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
        Half<TP, TQ, kFP, kFQ> h;
        h.read(lds, p0, q0, kk);
        h.template multiply<T>(acc);
    }
}

// ---- activations ---------------------------------------------------------------

// (the reciprocal to one unit in the last place, as the exponential)
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

__device__ __forceinline__ float silu(float z) { return z * sigmoid(z); }
// Phi(z) by erfc, which keeps the negative tail (1 + erf is off by 4% at -5 and 0 from -5.6 on)
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(z * -0.70710678f); }
__device__ __forceinline__ float gelu(float z) { return z * normal_cdf(z); }

__device__ __forceinline__ float act_slope(int act, float z)
{
    if (act == SOFT_TOPK_ACT_SILU) {
        const float s = sigmoid(z);
        return s * (1.0f + z * (1.0f - s));
    }
    if (act == SOFT_TOPK_ACT_GELU)
        return normal_cdf(z) + z * 0.39894228f * __expf(-0.5f * z * z);
    return 1.0f;
}

// ---- output --------------------------------------------------------------------
//
// A lane's results are four neighbours in one of 16 rows.  They go through
// LDS, 16 rows of a wave at a time, and come back as eight neighbours a lane,
// with a row's lanes side by side: whole lines are stored, and residual and
// bias are loaded 16 bytes at a time.  (Stored from the registers they were
// laid out in, 32 bytes of 16 rows at a time, a tile's end took 30 us.)

// whether eight neighbours from a multiple of eight can move at once
__host__ __device__ __forceinline__ bool eights(const void* p, int ld)
{
    return (ld & 7) == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

template <class T>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&v)[8], int count, bool whole)
{
    typename T::Store* p = reinterpret_cast<typename T::Store*>(base) + at;
    if (whole) {
        typename T::Store s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[j] = T::down(v[j]);
#pragma unroll
        for (int j = 0; j < (int)sizeof(s) / 16; ++j) {
            V4U u;
            __builtin_memcpy(&u, reinterpret_cast<const char*>(s) + j * 16, 16);
            __builtin_nontemporal_store(u, reinterpret_cast<V4U*>(p) + j);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < count)
                p[j] = T::down(v[j]);
    }
}

template <class T>
__device__ __forceinline__ void load8f(const void* base, int64_t at, float (&v)[8], int count, bool whole)
{
    const typename T::Store* p = reinterpret_cast<const typename T::Store*>(base) + at;
    if (whole) {
        typename T::Store s[8];
#pragma unroll
        for (int j = 0; j < (int)sizeof(s) / 16; ++j) {
            const V4U u = __builtin_nontemporal_load(reinterpret_cast<const V4U*>(p) + j);
            __builtin_memcpy(reinterpret_cast<char*>(s) + j * 16, &u, 16);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = T::up(s[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = j < count ? T::up(p[j]) : 0.0f;
    }
}

// f(row, v, up) for this lane's rows of the wave's results: eight neighbours
// from column lane_col() on (gated: of the gate and of its up columns).
template <int kFP, int kFQ, bool kGated>
struct Emit {
    static constexpr int kCols = kFP * 16, kOut = kGated ? kCols / 2 : kCols;
    static constexpr int kStride = kCols * 4 + 16;  // bytes of a row, shifted by a bank group each
    static constexpr int kBytes = 16 * kStride;     // a wave's
    static constexpr int kLanes = kOut / 8;         // lanes of a row

    static __device__ __forceinline__ int lane_col() { return lane_id() % kLanes * 8; }

    template <class F>
    static __device__ __forceinline__ void rows(char* lds, const V4F (&acc)[kFP][kFQ], const F& f)
    {
        const int lane = lane_id();
        char* const own = lds + threadIdx.x / kWave * kBytes;
        char* const to = own + (lane & 15) * kStride + (lane >> 4) * 16;
        const int col = kGated ? (lane_col() >> 4) * 32 + (lane_col() & 15) : lane_col();
        const char* const from = own + lane / kLanes % 16 * kStride + col * 4;
#pragma unroll
        for (int j = 0; j < kFQ; ++j) {
#pragma unroll
            for (int i = 0; i < kFP; ++i)
                *reinterpret_cast<V4F*>(to + i * 64) = acc[i][j];
            lds_order();
#pragma unroll 1
            for (int r = 0; r < 16; r += kWave / kLanes) {  // (unrolled, the code outgrows its cache)
                float v[8], up[8];
                *reinterpret_cast<V4F*>(v) = *reinterpret_cast<const V4F*>(from + r * kStride);
                *reinterpret_cast<V4F*>(v + 4) = *reinterpret_cast<const V4F*>(from + r * kStride + 16);
                if (kGated) {
                    *reinterpret_cast<V4F*>(up) = *reinterpret_cast<const V4F*>(from + r * kStride + 64);
                    *reinterpret_cast<V4F*>(up + 4) = *reinterpret_cast<const V4F*>(from + r * kStride + 80);
                }
                if (kLanes >= 4 || lane / kLanes < 16)
                    f(j * 16 + r + lane / kLanes, v, up);
            }
            lds_order();
        }
    }
};

// ---- kernels -------------------------------------------------------------------

template <bool kFirst, class A, class B>
struct Pick {
    using type = A;
};
template <class A, class B>
struct Pick<false, A, B> {
    using type = B;
};

// A tile of kBP x kBQ results by kWP x kWQ waves.  kTeams such teams share
// the tile's steps, each with operands of its own in LDS, and are joined in
// their order: many steps on few tiles.
template <int kBP_, int kBQ_, int kWP_, int kWQ_, int kTeams_>
struct Shape {
    static constexpr int kBP = kBP_, kBQ = kBQ_, kWP = kWP_, kWQ = kWQ_, kTeams = kTeams_;
    static constexpr int kT = kWP * kWQ * kWave, kAll = kT * kTeams;
    static constexpr int kFP = kBP / kWP / 16, kFQ = kBQ / kWQ / 16;
};

template <class S>
__device__ __forceinline__ void wave_place(int& p0, int& q0)
{
    const int wave = __builtin_amdgcn_readfirstlane(own_thread<S::kT>() / kWave);
    p0 = wave % S::kWP * (S::kFP * 16);
    q0 = wave / S::kWP * (S::kFQ * 16);
}

template <class S>
__device__ __forceinline__ int own_team()
{
    return S::kTeams == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / S::kT);
}

// The teams' results added in their order; true for the team that has the
// sum.  Every operand in LDS has been read when this returns.
template <class S>
__device__ __forceinline__ bool join_teams(char* lds, V4F (&acc)[S::kFP][S::kFQ])
{
    __syncthreads();
    if constexpr (S::kTeams > 1) {
        constexpr int kFrags = S::kFP * S::kFQ;
        const int team = own_team<S>();
        V4F* const part = reinterpret_cast<V4F*>(lds) + own_thread<S::kT>();
        if (team > 0) {
#pragma unroll
            for (int i = 0; i < kFrags; ++i)
                part[((team - 1) * kFrags + i) * S::kT] = acc[i / S::kFQ][i % S::kFQ];
        }
        __syncthreads();
        if (team == 0) {
#pragma unroll
            for (int t = 0; t + 1 < S::kTeams; ++t)
#pragma unroll
                for (int i = 0; i < kFrags; ++i)
                    acc[i / S::kFQ][i % S::kFQ] += part[(t * kFrags + i) * S::kT];
        }
        __syncthreads();
        return team == 0;
    }
    return true;
}

template <class T>
__device__ __forceinline__ void zero_rows(void* out, int row0, int end, int col0, int cols, int ld)
{
    const int n = (end - row0) * cols;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int64_t r = row0 + i / cols;
        const int c = col0 + i % cols;
        if (c < ld)
            reinterpret_cast<typename T::Store*>(out)[r * ld + c] = T::down(0.0f);
    }
}

template <class T, class S, bool kGated, bool kDirect>
__global__ __launch_bounds__(S::kAll) void experts_forward_kernel(ExpertsArgs a)
{
    using TP = RowTile<S::kBP, S::kT>;
    using TQ = RowTile<S::kBQ, S::kT>;
    constexpr int kStep = TP::kBytes + TQ::kBytes;
    constexpr int kTeam = kStep * (kDirect ? 2 : 1);  // a team's operands
    __shared__ __attribute__((aligned(16))) char lds_all[kTeam * S::kTeams];
    constexpr int kCols = kGated ? S::kBP / 2 : S::kBP;  // columns of y in a tile
    const Tiles t = count_tiles(a, S::kBQ);
    const int across = (a.N + kCols - 1) / kCols;
    const int id = blockIdx.x, total = launched_tiles(t, across) * across;
    if (id >= total) {
        const int over = id - total;
        const int64_t r0 = t.behind + (int64_t)(over / across) * S::kBQ;
        const int64_t end = r0 + S::kBQ < a.pairs ? r0 + S::kBQ : a.pairs;
        if (r0 < end) {
            zero_rows<T>(a.y, (int)r0, (int)end, over % across * kCols, kCols, a.N);
            if (a.z) {
                zero_rows<F32>(a.z, (int)r0, (int)end, over % across * kCols, kCols, a.M);
                if (kGated)
                    zero_rows<F32>(a.z, (int)r0, (int)end, a.N + over % across * kCols, kCols, a.M);
            }
        }
        return;
    }
    const int tile = xcd_order(id, total);
    int e, row0, end, column;
    find_tile(a, t, tile, across, S::kBQ, e, row0, end, column);
    const int n0 = column * kCols;

    const uint16_t* const w = reinterpret_cast<const uint16_t*>(a.w) + ((int64_t)e * a.M + n0) * a.K;
    const uint16_t* const x = reinterpret_cast<const uint16_t*>(a.x) + (a.rows ? 0 : (int64_t)row0 * a.K);
    // where a row begins in w and x (negative: it has none)
    auto w_row = [&](int i) -> int64_t {
        const int r = TP::row_of(i);
        // gated tiles take 16 gate rows and their 16 up rows in turn
        const int n = kGated ? (r >> 5) * 16 + (r & 15) : r;
        return n < a.N - n0 ? (int64_t)(n + (kGated && (r & 16) ? a.N : 0)) * a.K : -1;
    };
    auto x_row = [&](int i) -> int64_t {
        const int r = TQ::row_of(i);
        if (r >= end - row0)
            return -1;
        const int s = a.rows ? a.rows[row0 + r] : r;
        return !a.rows || (s >= 0 && s < a.tokens) ? (int64_t)s * a.K : -1;
    };
    int p0, q0;
    wave_place<S>(p0, q0);
    V4F acc[S::kFP][S::kFQ] = {};
    const int team = own_team<S>();
    char* const lds = lds_all + team * kTeam;
    const int steps = (a.K + kBK * S::kTeams - 1) / (kBK * S::kTeams);  // a team's
    typename Pick<kDirect, RowLoad<S::kBP, S::kT>, TP>::type tp;
    typename Pick<kDirect, RowLoad<S::kBQ, S::kT>, TQ>::type tq;
    tp.start(w);
    tq.start(x);
#pragma unroll
    for (int i = 0; i < TP::kLoads; ++i)
        tp.set(i, w_row(i));
#pragma unroll
    for (int i = 0; i < TQ::kLoads; ++i)
        tq.set(i, x_row(i));
    if constexpr (kDirect) {
        direct_steps<T, TP, TQ>(lds, steps, p0, q0, q0 < end - row0 && (kGated ? p0 / 2 : p0) < a.N - n0, acc,
                                [&](const char* at, int s) {
            tp.issue(at, s * S::kTeams + team, a.K);
            tq.issue(at + TP::kBytes, s * S::kTeams + team, a.K);
        });
    } else {
        V8S vp[TP::kLoads], vq[TQ::kLoads];
        tp.fetch(team, a.K, vp);
        tq.fetch(team, a.K, vq);
        for (int s = 0; s < steps; ++s) {
            __syncthreads();
            TP::put(lds, vp);
            TQ::put(lds + TP::kBytes, vq);
            __syncthreads();
            if (s + 1 < steps) {
                tp.fetch((s + 1) * S::kTeams + team, a.K, vp);
                tq.fetch((s + 1) * S::kTeams + team, a.K, vq);
            }
            step_mma<T, TP, TQ>(lds, p0, q0, acc);
        }
    }

    if (!join_teams<S>(lds_all, acc))
        return;
    using Out = Emit<S::kFP, S::kFQ, kGated>;
    const int col = n0 + p0 / (kGated ? 2 : 1) + Out::lane_col();
    const int count = a.N - col < 8 ? a.N - col : 8;
    const bool wy = eights(a.y, a.N), wr = eights(a.residual, a.N), wz = eights(a.z, a.N), wb = eights(a.bias, a.N);
    float bias[8] = {}, bias_up[8] = {};
    if (a.bias && count > 0) {
        load8f<T>(a.bias, (int64_t)e * a.M + col, bias, count, wb);
        if (kGated)
            load8f<T>(a.bias, (int64_t)e * a.M + a.N + col, bias_up, count, wb);
    }
    Out::rows(lds_all, acc, [&](int r, float (&v)[8], float (&up)[8]) {
        const int64_t row = row0 + q0 + r;
        if (row >= end || count <= 0)
            return;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            v[q] += bias[q];
            up[q] = kGated ? up[q] + bias_up[q] : 0.0f;
        }
        if (a.z) {
            store8<F32>(a.z, row * a.M + col, v, count, wz);
            if (kGated)
                store8<F32>(a.z, row * a.M + a.N + col, up, count, wz);
        }
        if (kGated) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] *= sigmoid(v[q]) * up[q];
        } else if (a.act == SOFT_TOPK_ACT_SILU) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = silu(v[q]);
        } else if (a.act == SOFT_TOPK_ACT_GELU) {
#pragma unroll 1
            for (int q = 0; q < 8; ++q)
                v[q] = gelu(v[q]);
        }
        if (a.residual) {
            float add[8];
            load8f<T>(a.residual, row * a.N + col, add, count, wr);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] += add[q];
        }
        store8<T>(a.y, row * a.N + col, v, count, wy);
    });
}

// dz = dy act'(z) for 64 rows of one expert and 512 columns: a lane takes
// eight neighbouring columns (gated: of the gate and of its up columns), the
// four waves every fourth row; and the column sums of the tile for the bias,
// joined in the order of the waves.  Bound by its bytes, z in fp32 the most
// (65,536 x 2 x 1024 228 us); with GELU by erfc's instructions, 8192 x 4096
// 67 us (58 with erf, which loses the tail).
constexpr int kActRows = 64;
constexpr int kActCols = 512;

// kWhole: every row is whole, aligned 16-byte pieces (a constant, since a
// load in a branch is waited for there: 232 us with it, 65,536 x 2 x 1024).
template <class T, bool kGated, bool kWhole>
__global__ __launch_bounds__(256) void experts_slope_kernel(ExpertsArgs a)
{
    __shared__ float part[3][kGated ? 2 : 1][kActCols];
    const Tiles t = count_tiles(a, kActRows);
    const int tile = blockIdx.x;
    if (tile >= t.total)
        return;
    int e, row0, end, column;
    find_tile(a, t, tile, 1, kActRows, e, row0, end, column);
    end = row0 + kActRows < end ? row0 + kActRows : end;
    const int wave = threadIdx.x / kWave;
    const int n = blockIdx.y * kActCols + lane_id() * 8;
    const int count = a.N - n < 8 ? a.N - n : 8;
    float sg[8] = {}, su[8] = {};
    if (count > 0) {
        for (int64_t r = row0 + wave; r < end; r += 4) {
            float d[8], z[8], u[8];
            load8f<T>(a.dy, r * a.N + n, d, count, kWhole);
            if (a.z)
                load8f<F32>(a.z, r * a.M + n, z, count, kWhole);
            if (kGated) {
                load8f<F32>(a.z, r * a.M + a.N + n, u, count, kWhole);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float s = sigmoid(z[q]), g = d[q];
                    d[q] = g * u[q] * s * (1.0f + z[q] * (1.0f - s));
                    u[q] = g * z[q] * s;
                    su[q] += u[q];
                }
                store8<T>(a.dz, r * a.M + a.N + n, u, count, kWhole);
            } else if (a.z) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    d[q] *= act_slope(a.act, z[q]);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q)
                sg[q] += d[q];
            if (a.dz != a.dy)
                store8<T>(a.dz, r * a.M + n, d, count, kWhole);
        }
    }
    if (!a.db)
        return;
    if (wave > 0) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            part[wave - 1][0][lane_id() * 8 + q] = sg[q];
            if (kGated)
                part[wave - 1][kGated ? 1 : 0][lane_id() * 8 + q] = su[q];
        }
    }
    __syncthreads();
    if (wave > 0 || count <= 0)
        return;
#pragma unroll
    for (int w = 0; w < 3; ++w)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            sg[q] += part[w][0][lane_id() * 8 + q];
            if (kGated)
                su[q] += part[w][kGated ? 1 : 0][lane_id() * 8 + q];
        }
    store8<F32>(a.dbp, (int64_t)tile * a.M + n, sg, count, (a.N & 7) == 0);
    if (kGated)
        store8<F32>(a.dbp, (int64_t)tile * a.M + a.N + n, su, count, (a.N & 7) == 0);
}

// db_e: the sums of its tiles; 16 waves take every 16th tile of 64 columns
// each, and are joined in their order.
constexpr int kBiasWaves = 16;

template <class T>
__global__ __launch_bounds__(kBiasWaves* kWave) void experts_bias_kernel(ExpertsArgs a, int tiles)
{
    __shared__ float part[kBiasWaves][kWave];
    const Tiles t = count_tiles(a, kActRows);
    const int e = blockIdx.x, lane = e / t.per;
    int first = __builtin_amdgcn_readlane(t.upto - t.mine, lane);
    for (int i = lane * t.per; i < e; ++i)
        first += expert_tiles(a, i, kActRows);
    // (within the table of tiles, where the offsets fall)
    const int left = tiles - first, own = expert_tiles(a, e, kActRows);
    const int count = own < left ? own : left;
    const int n = blockIdx.y * kWave + lane_id(), wave = threadIdx.x / kWave;
    float s = 0.0f;
    if (n < a.M) {
#pragma unroll 4
        for (int i = wave; i < count; i += kBiasWaves)
            s += a.dbp[(int64_t)(first + i) * a.M + n];
    }
    part[wave][lane_id()] = s;
    __syncthreads();
    if (wave > 0 || n >= a.M)
        return;
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kBiasWaves; ++w)
        s += part[w][lane_id()];
    reinterpret_cast<typename T::Store*>(a.db)[(int64_t)e * a.M + n] = T::down(s);
}

// The residual's gradient: dy before the last row of the last expert, 0 from
// there on (y is 0 there whatever the residual holds).  kWhole: both are
// aligned 16-byte pieces.  Bound by memory: 65,536 x 2048 bf16 88 us, 6.1 TB/s.
constexpr int kResidualBlocks = 2048;
constexpr int kResidualLoads = 4;  // pieces of a thread in flight

template <bool kWhole>
__global__ __launch_bounds__(256) void experts_residual_kernel(ExpertsArgs a, uint16_t* dr)
{
    const uint16_t* const dy = reinterpret_cast<const uint16_t*>(a.dy);
    const int64_t n = (int64_t)a.pairs * a.N, kept = (int64_t)clamp_row(a.offsets[a.experts], a.pairs) * a.N;
    constexpr int64_t kApart = 256 * 8;  // elements between a thread's pieces
    for (int64_t first = (int64_t)blockIdx.x * (kApart * kResidualLoads); first < n;
         first += (int64_t)gridDim.x * (kApart * kResidualLoads)) {
        const int64_t at = first + threadIdx.x * 8;
        if (kWhole && first + kApart * kResidualLoads <= kept) {
            V4U u[kResidualLoads];
#pragma unroll
            for (int i = 0; i < kResidualLoads; ++i)
                u[i] = __builtin_nontemporal_load(reinterpret_cast<const V4U*>(dy + at + i * kApart));
#pragma unroll
            for (int i = 0; i < kResidualLoads; ++i)
                __builtin_nontemporal_store(u[i], reinterpret_cast<V4U*>(dr + at + i * kApart));
        } else if (kWhole && first >= kept && first + kApart * kResidualLoads <= n) {
#pragma unroll
            for (int i = 0; i < kResidualLoads; ++i)
                __builtin_nontemporal_store(V4U{0u, 0u, 0u, 0u}, reinterpret_cast<V4U*>(dr + at + i * kApart));
        } else {
#pragma unroll 8
            for (int j = 0; j < 8 * kResidualLoads; ++j) {
                const int64_t e = first + j * 256 + threadIdx.x;
                if (e < n)
                    dr[e] = e < kept ? dy[e] : (uint16_t)0;
            }
        }
    }
}

// dx of every place: dz (rows) times W_e (its columns), summed over M.
// 8192^3 776 us, 1417 TFLOP/s; 65,536 rows of 64 uneven experts, 2048 to 2048,
// 640 us: its row tiles are 12% part-filled, 32 steps leave a tile's start and
// end 15% of it, and the fp32 rows out are 0.5 GB.
template <class T, class S, bool kDirect>
__global__ __launch_bounds__(S::kAll) void experts_input_kernel(ExpertsArgs a)
{
    using TP = ColTile<S::kBP, S::kT>;
    using TQ = RowTile<S::kBQ, S::kT>;
    constexpr int kStep = TP::kBytes + TQ::kBytes;
    constexpr int kTeam = kStep * (kDirect ? 2 : 1);  // a team's operands
    __shared__ __attribute__((aligned(16))) char lds_all[kTeam * S::kTeams];
    const Tiles t = count_tiles(a, S::kBQ);
    const int across = (a.K + S::kBP - 1) / S::kBP;
    const int id = blockIdx.x, total = launched_tiles(t, across) * across;
    if (id >= total) {
        const int over = id - total;
        const int64_t r0 = t.behind + (int64_t)(over / across) * S::kBQ;
        const int64_t end = r0 + S::kBQ < a.pairs ? r0 + S::kBQ : a.pairs;
        if (!a.dxr && r0 < end)
            zero_rows<T>(a.dx, (int)r0, (int)end, over % across * S::kBP, S::kBP, a.K);
        return;
    }
    const int tile = xcd_order(id, total);
    int e, row0, end, column;
    find_tile(a, t, tile, across, S::kBQ, e, row0, end, column);
    const int c0 = column * S::kBP;
    const uint16_t* w = reinterpret_cast<const uint16_t*>(a.w) + (int64_t)e * a.M * a.K;
    typename Pick<kDirect, RowLoad<S::kBQ, S::kT>, TQ>::type tq;
    tq.start(reinterpret_cast<const uint16_t*>(a.dz) + (int64_t)row0 * a.M);
#pragma unroll
    for (int i = 0; i < TQ::kLoads; ++i) {
        const int r = TQ::row_of(i);
        tq.set(i, r < end - row0 ? (int64_t)r * a.M : -1);
    }
    int p0, q0;
    wave_place<S>(p0, q0);
    V4F acc[S::kFP][S::kFQ] = {};
    const int team = own_team<S>();
    char* const lds = lds_all + team * kTeam;
    const int steps = (a.M + kBK * S::kTeams - 1) / (kBK * S::kTeams);  // a team's
    if constexpr (kDirect) {
        ColLoad<S::kBP, S::kT> tp;
        tp.start(w, a.K, c0, a.K);
        direct_steps<T, TP, TQ>(lds, steps, p0, q0, q0 < end - row0 && p0 < a.K - c0, acc, [&](const char* at, int s) {
            const int step = s * S::kTeams + team;
            tp.issue(at, (int64_t)step * kBK, a.M - step * kBK);
            tq.issue(at + TP::kBytes, step, a.M);
        });
    } else {
        V8S vp[TP::kLoads], vq[TQ::kLoads];
        auto fetch = [&](int round) {
            const int s = round * S::kTeams + team;
#pragma unroll
            for (int i = 0; i < TP::kLoads; ++i) {
                const int m = s * kBK + TP::row_of(i), c = c0 + TP::col_of(i);
                vp[i] = load8(w + (int64_t)m * a.K + c, m < a.M ? a.K - c : 0);
            }
            tq.fetch(s, a.M, vq);
        };
        fetch(0);
        for (int s = 0; s < steps; ++s) {
            __syncthreads();
            TP::put(lds, vp);
            TQ::put(lds + TP::kBytes, vq);
            __syncthreads();
            if (s + 1 < steps)
                fetch(s + 1);
            step_mma<T, TP, TQ>(lds, p0, q0, acc);
        }
    }
    if (!join_teams<S>(lds_all, acc))
        return;
    using Out = Emit<S::kFP, S::kFQ, false>;
    const int col = c0 + p0 + Out::lane_col();
    const int count = a.K - col < 8 ? a.K - col : 8;
    const bool whole = a.dxr ? eights(a.dxr, a.K) : eights(a.dx, a.K);
    Out::rows(lds_all, acc, [&](int r, float (&v)[8], float (&)[8]) {
        const int64_t row = row0 + q0 + r;
        if (row >= end || count <= 0)
            return;
        if (a.dxr)
            store8<F32>(a.dxr, row * a.K + col, v, count, whole);
        else
            store8<T>(a.dx, row * a.K + col, v, count, whole);
    });
}

// dW_e: dz (columns) times x (columns), summed over the expert's rows.
// 8192^3 780 us, 1410 TFLOP/s; 65,536 rows of 64 uneven experts, 2048 x 2048,
// 600 us.
// kRows: x is gathered by a.rows (a constant: with both forms in one loop the
// compiler waits for the loads just issued to merge their registers, 1160
// against 1420 TFLOP/s at 8192^3).
template <class T, class S, bool kDirect, bool kRows>
__global__ __launch_bounds__(S::kAll) void experts_weight_kernel(ExpertsArgs a)
{
    using TP = ColTile<S::kBP, S::kT>;
    using TQ = ColTile<S::kBQ, S::kT>;
    constexpr int kStep = TP::kBytes + TQ::kBytes;
    constexpr int kTeam = kStep * (kDirect ? 2 : 1);  // a team's operands
    __shared__ __attribute__((aligned(16))) char lds_all[kTeam * S::kTeams];
    const int across = (a.K + S::kBP - 1) / S::kBP, down = (a.M + S::kBQ - 1) / S::kBQ;
    // A tile costs its expert's rows.  Eight tiles (4 x 2) go to an XCD in
    // turn, so that every XCD has its share of every expert (whole experts an
    // XCD in turn left some with twice the rows of others).
    const int tile = a.experts == 1 ? xcd_order(blockIdx.x, gridDim.x) : xcd_eights(blockIdx.x, gridDim.x);
    const int e = tile / (across * down);
    int i, j;
    if (a.experts == 1)
        tile_place(tile % (across * down), down, across, i, j);
    else
        tile_place<4>(tile % (across * down), down, across, i, j);
    const int c0 = j * S::kBP, m0 = i * S::kBQ;
    int row0 = clamp_row(a.offsets[e], a.pairs), end = clamp_row(a.offsets[e + 1], a.pairs);
    if (gridDim.y > 1) {  // this work-group's share of the expert's rows
        const int64_t share = ((int64_t)end - row0 + kBK * gridDim.y - 1) / (kBK * (int64_t)gridDim.y) * kBK;
        const int64_t first = row0 + share * blockIdx.y;
        row0 = first < end ? (int)first : end;
        end = end - row0 < share ? end : row0 + (int)share;
    }
    int p0, q0;
    wave_place<S>(p0, q0);
    V4F acc[S::kFP][S::kFQ] = {};
    const int team = own_team<S>();
    char* const lds = lds_all + team * kTeam;
    const int steps = end > row0 ? (end - row0 + kBK * S::kTeams - 1) / (kBK * S::kTeams) : 0;  // a team's
    // the row of x that chunk i of step s comes from (-1: zeros)
    auto source = [&](int s, int i) {
        const int r = row0 + s * kBK + TP::row_of(i);
        const int src = r >= end ? -1 : (a.rows ? a.rows[r] : r);
        return src < a.tokens ? src : -1;
    };
    if constexpr (kDirect) {
        ColLoad<S::kBP, S::kT> tp;
        ColLoad<S::kBQ, S::kT> tq;
        tp.start(a.x, a.K, c0, a.K);
        tq.start(a.dz, a.M, m0, a.M);
        // the sources of a step's rows are read one step ahead of their loads
        int src[TP::kLoads];
        auto find = [&](int s) {
#pragma unroll
            for (int i = 0; i < TP::kLoads; ++i) {
                const int r = row0 + (s * S::kTeams + team) * kBK + TP::row_of(i);
                src[i] = a.rows[r < end ? r : end - 1];
            }
        };
        auto issue = [&](const char* at, int s) {
            const int64_t first = row0 + (int64_t)(s * S::kTeams + team) * kBK;
            const int left = end - (int)first;
            if constexpr (kRows) {
                int from[TP::kLoads];
#pragma unroll
                for (int i = 0; i < TP::kLoads; ++i)
                    from[i] = TP::row_of(i) < left ? src[i] : -1;
                tp.issue_rows(at, from, a.tokens);
                find(s + 1);
            } else {
                tp.issue(at, first, left);
            }
            tq.issue(at + TP::kBytes, first, left);
        };
        if (steps) {
            if constexpr (kRows)
                find(0);
            direct_steps<T, TP, TQ>(lds, steps, p0, q0, p0 < a.K - c0 && q0 < a.M - m0, acc, issue);
        }
    } else {
        V8S vp[TP::kLoads], vq[TQ::kLoads];
        auto fetch = [&](int round) {
            const int s = round * S::kTeams + team;
#pragma unroll
            for (int i = 0; i < TP::kLoads; ++i) {
                const int src = source(s, i), c = c0 + TP::col_of(i);
                vp[i] = load8(reinterpret_cast<const uint16_t*>(a.x) + (int64_t)src * a.K + c, src >= 0 ? a.K - c : 0);
            }
#pragma unroll
            for (int i = 0; i < TQ::kLoads; ++i) {
                const int r = row0 + s * kBK + TQ::row_of(i), c = m0 + TQ::col_of(i);
                vq[i] = load8(reinterpret_cast<const uint16_t*>(a.dz) + (int64_t)r * a.M + c, r < end ? a.M - c : 0);
            }
        };
        if (steps)
            fetch(0);
        for (int s = 0; s < steps; ++s) {
            __syncthreads();
            TP::put(lds, vp);
            TQ::put(lds + TP::kBytes, vq);
            __syncthreads();
            if (s + 1 < steps)
                fetch(s + 1);
            step_mma<T, TP, TQ>(lds, p0, q0, acc);
        }
    }
    if (!join_teams<S>(lds_all, acc))
        return;
    using Out = Emit<S::kFP, S::kFQ, false>;
    const int col = c0 + p0 + Out::lane_col();
    const int count = a.K - col < 8 ? a.K - col : 8;
    const bool whole = gridDim.y > 1 ? eights(a.dwp, a.K) : eights(a.dw, a.K);
    Out::rows(lds_all, acc, [&](int r, float (&v)[8], float (&)[8]) {
        const int m = m0 + q0 + r;
        if (m >= a.M || count <= 0)
            return;
        if (gridDim.y > 1)
            store8<F32>(a.dwp, (((int64_t)blockIdx.y * a.experts + e) * a.M + m) * a.K + col, v, count, whole);
        else
            store8<T>(a.dw, ((int64_t)e * a.M + m) * a.K + col, v, count, whole);
    });
}

// dW from the shares of its rows, in their order.
template <class T>
__global__ __launch_bounds__(256) void experts_join_kernel(ExpertsArgs a, int shares)
{
    const int64_t n = (int64_t)a.experts * a.M * a.K;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        float s = 0.0f;
#pragma unroll 4
        for (int j = 0; j < shares; ++j)
            s += a.dwp[j * n + i];
        reinterpret_cast<typename T::Store*>(a.dw)[i] = T::down(s);
    }
}

// The shapes, and where they win (forward, bf16, us; the gradients keep the
// order).  Columns x rows, with the teams on a tile's steps:
//                                  64x64   128x128  128x128  128x256  256x256
//   rows, K -> N                   4 teams 2 teams
//   256, 4096 -> 4096                 23       36       49       55       83
//   512, 4096 -> 4096                 42       37       50       54       83
//   1024, 4096 -> 4096                80       41       53       56       83
//   2048, 4096 -> 4096               152       78       76       63       86
//   3000, 4096 -> 4096               224      112      120      115       89
//   64 experts x 128, 1024 -> 1024    64       38       28       38       33
//   64 experts x 256, 2048 -> 2048   458      240      206      203      158
// A shape is best up to one tile a CU (256): what is left idle by a larger
// one costs more than the operands it reads less.  Beyond, the largest, if
// an expert fills its rows.
using Big = Shape<256, 256, 2, 4, 1>;
using Wide = Shape<128, 256, 2, 4, 1>;
using Small = Shape<128, 128, 2, 2, 1>;
using Mid = Shape<128, 128, 2, 2, 2>;
using Tiny = Shape<64, 64, 2, 2, 4>;
enum class Size { kTiny, kMid, kSmall, kWide, kBig };
constexpr int kCus = 256;

int ceil_div(int64_t a, int b) { return (int)((a + b - 1) / b); }

// row tiles that cover any split of the pairs, and the rows behind
int row_tiles(const ExpertsArgs& a, int rows) { return ceil_div(a.pairs, rows) + a.experts; }

// whole, aligned 16-byte chunks
bool chunks(const void* p, int ld) { return (ld & 7) == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <class T, class S, bool kDirect>
void forward_launch(const ExpertsArgs& a, hipStream_t stream)
{
    if (a.M != a.N) {
        const dim3 grid((unsigned)row_tiles(a, S::kBQ) * ceil_div(a.N, S::kBP / 2));
        STK_LAUNCH(kKExpertsForward, stream, (experts_forward_kernel<T, S, true, kDirect>), grid, dim3(S::kAll), 0,
                   stream, a);
    } else {
        const dim3 grid((unsigned)row_tiles(a, S::kBQ) * ceil_div(a.N, S::kBP));
        STK_LAUNCH(kKExpertsForward, stream, (experts_forward_kernel<T, S, false, kDirect>), grid, dim3(S::kAll), 0,
                   stream, a);
    }
}

// Tiles of the products with `width` columns, if the rows were spread evenly.
int64_t even_tiles(const ExpertsArgs& a, int columns, int rows, int width)
{
    const int used = a.pairs < a.experts ? a.pairs : a.experts;
    return (int64_t)used * ceil_div(ceil_div(a.pairs, used), rows) * ceil_div(width, columns);
}

Size product_size(const ExpertsArgs& a, int width, bool direct)
{
    // (through registers the small tiles win up to two a CU: 2331 rows of 17
    // experts, 1001 -> 523, 22 us against 37, with bias and GELU 28 against 48)
    if (even_tiles(a, 64, 64, width) <= (direct ? kCus : 2 * kCus))
        return Size::kTiny;
    if (!direct)
        return Size::kSmall;
    if (even_tiles(a, 128, 128, width) <= kCus)
        return Size::kMid;
    if (a.pairs / a.experts < 256)
        return Size::kSmall;
    return even_tiles(a, 128, 256, width) <= kCus ? Size::kWide : Size::kBig;
}

// Whether the loads into LDS reach what they need by 32-bit offsets: 256 rows
// of a tile, gathered rows from the first token, an up row from its gate row.
bool in_reach(int64_t rows, int64_t elements) { return rows * elements * 2 < (int64_t)kBufferEnd - 1024; }
bool near(const ExpertsArgs& a)
{
    return in_reach(256, a.K) && in_reach(256, a.M) && (a.M == a.N || in_reach((int64_t)a.N + 256, a.K)) &&
           (!a.rows || in_reach(a.tokens, a.K));
}

bool forward_direct(const ExpertsArgs& a) { return chunks(a.x, a.K) && chunks(a.w, a.K) && near(a); }
bool weight_direct(const ExpertsArgs& a) { return chunks(a.x, a.K) && chunks(a.dz, a.M) && near(a); }
bool input_direct(const ExpertsArgs& a) { return chunks(a.w, a.K) && chunks(a.dz, a.M) && near(a); }

template <class T>
hipError_t forward(const ExpertsArgs& a, hipStream_t stream)
{
    const bool direct = forward_direct(a);
    const Size size = product_size(a, a.M, direct);
    if (size == Size::kTiny)
        direct ? forward_launch<T, Tiny, true>(a, stream) : forward_launch<T, Tiny, false>(a, stream);
    else if (size == Size::kMid)
        forward_launch<T, Mid, true>(a, stream);
    else if (size == Size::kWide)
        forward_launch<T, Wide, true>(a, stream);
    else if (size == Size::kBig)
        forward_launch<T, Big, true>(a, stream);
    else
        direct ? forward_launch<T, Small, true>(a, stream) : forward_launch<T, Small, false>(a, stream);
    return hipGetLastError();
}

int64_t weight_tiles(int experts, int K, int M, int columns, int rows)
{
    return (int64_t)experts * ceil_div(K, columns) * ceil_div(M, rows);
}

// The same for dW, [M][K] of every expert, whose steps are the expert's rows.
Size weight_size(const ExpertsArgs& a, bool direct)
{
    if (weight_tiles(a.experts, a.K, a.M, 64, 64) <= kCus)
        return Size::kTiny;
    if (!direct)
        return Size::kSmall;
    if (weight_tiles(a.experts, a.K, a.M, 128, 128) <= kCus)
        return Size::kMid;
    return weight_tiles(a.experts, a.K, a.M, 128, 256) <= kCus ? Size::kWide : Size::kBig;
}

template <class T, class S, bool kDirect>
void weight_launch(const ExpertsArgs& a, int shares, hipStream_t stream)
{
    const dim3 grid((unsigned)a.experts * ceil_div(a.K, S::kBP) * ceil_div(a.M, S::kBQ), shares);
    if (a.rows)
        STK_LAUNCH(kKExpertsBackward, stream, (experts_weight_kernel<T, S, kDirect, true>), grid, dim3(S::kAll), 0, stream,
                   a);
    else
        STK_LAUNCH(kKExpertsBackward, stream, (experts_weight_kernel<T, S, kDirect, false>), grid, dim3(S::kAll), 0,
                   stream, a);
    if (shares > 1)
        STK_LAUNCH(kKExpertsBackward, stream, (experts_join_kernel<T>), dim3(1024), dim3(256), 0, stream, a, shares);
}

template <class T, class S, bool kDirect>
void input_launch(const ExpertsArgs& a, hipStream_t stream)
{
    const dim3 grid((unsigned)row_tiles(a, S::kBQ) * ceil_div(a.K, S::kBP));
    STK_LAUNCH(kKExpertsBackward, stream, (experts_input_kernel<T, S, kDirect>), grid, dim3(S::kAll), 0, stream, a);
}

template <class T, bool kGated, bool kWhole>
void slope_launch(const ExpertsArgs& a, hipStream_t stream)
{
    const dim3 grid(row_tiles(a, kActRows), ceil_div(a.N, kActCols));
    STK_LAUNCH(kKExpertsBackward, stream, (experts_slope_kernel<T, kGated, kWhole>), grid, dim3(256), 0, stream, a);
}

template <class T>
hipError_t backward(const ExpertsArgs& a, int dtype, hipStream_t stream)
{
    if (a.dz != a.dy || a.db) {
        const bool whole = eights(a.dy, a.N) && eights(a.z, a.N) && eights(a.dz, a.N);
        if (a.M != a.N && whole)
            slope_launch<T, true, true>(a, stream);
        else if (a.M != a.N)
            slope_launch<T, true, false>(a, stream);
        else if (whole)
            slope_launch<T, false, true>(a, stream);
        else
            slope_launch<T, false, false>(a, stream);
    }
    if (a.db) {
        const dim3 grid(a.experts, ceil_div(a.M, kWave));
        STK_LAUNCH(kKExpertsBackward, stream, (experts_bias_kernel<T>), grid, dim3(kBiasWaves * kWave), 0, stream, a,
                   (int)experts_bias_tiles(a.pairs, a.experts));
    }
    if (a.dw) {
        const bool direct = weight_direct(a);
        const int shares = experts_weight_shares(a.pairs, a.experts, a.K, a.M);
        const Size size = weight_size(a, direct);
        if (size == Size::kTiny)
            direct ? weight_launch<T, Tiny, true>(a, shares, stream) : weight_launch<T, Tiny, false>(a, shares, stream);
        else if (size == Size::kMid)
            weight_launch<T, Mid, true>(a, 1, stream);
        else if (size == Size::kWide)
            weight_launch<T, Wide, true>(a, 1, stream);
        else if (size == Size::kBig)
            weight_launch<T, Big, true>(a, 1, stream);
        else
            weight_launch<T, Small, false>(a, 1, stream);
    }
    if (a.dx) {
        const bool direct = input_direct(a);
        const Size size = product_size(a, a.K, direct);
        if (size == Size::kTiny)
            direct ? input_launch<T, Tiny, true>(a, stream) : input_launch<T, Tiny, false>(a, stream);
        else if (size == Size::kMid)
            input_launch<T, Mid, true>(a, stream);
        else if (size == Size::kWide)
            input_launch<T, Wide, true>(a, stream);
        else if (size == Size::kBig)
            input_launch<T, Big, true>(a, stream);
        else
            direct ? input_launch<T, Small, true>(a, stream) : input_launch<T, Small, false>(a, stream);
        if (a.dxr) {
            CombineArgs c = {};
            c.y = a.dxr;
            c.slots = a.slots;
            c.tokens = a.tokens;
            c.k = a.k;
            c.places = a.pairs;
            c.N = a.K;
            c.out = a.dx;
            const hipError_t r = launch_combine_forward(c, dtype, true, stream);
            if (r != hipSuccess)
                return r;
        }
    }
    return hipGetLastError();
}

// f of the shape of that size
template <class F>
bool with_shape(Size size, const F& f)
{
    switch (size) {
    case Size::kTiny: return f(Tiny{});
    case Size::kMid: return f(Mid{});
    case Size::kSmall: return f(Small{});
    case Size::kWide: return f(Wide{});
    default: return f(Big{});
    }
}

bool launch_fits(int64_t groups, int threads) { return groups * threads < (1ll << 32); }

// the row tiles of a product across `width` columns, `halves`: two of w to one
bool product_fits(const ExpertsArgs& a, Size size, int width, int halves)
{
    return with_shape(size, [&](auto s) {
        return launch_fits((int64_t)row_tiles(a, s.kBQ) * ceil_div(width, s.kBP / halves), s.kAll);
    });
}

}  // namespace

bool experts_forward_fits(const ExpertsArgs& a)
{
    return product_fits(a, product_size(a, a.M, forward_direct(a)), a.N, a.M != a.N ? 2 : 1);
}

bool experts_backward_fits(const ExpertsArgs& a)
{
    if ((a.dz != a.dy || a.db) && !launch_fits(row_tiles(a, kActRows), 256))
        return false;
    if (a.dw && !with_shape(weight_size(a, weight_direct(a)), [&](auto s) {
            return launch_fits(weight_tiles(a.experts, a.K, a.M, s.kBP, s.kBQ), s.kAll);
        }))
        return false;
    return !a.dx || product_fits(a, product_size(a, a.K, input_direct(a)), a.K, 1);
}

// Work-groups on the rows of one tile of dW: as many as fill the chip once,
// each with four steps a team at least (65,536 rows of one expert, 256 x 256:
// 253 us by one, 36 by 16).
int32_t experts_weight_shares(int64_t pairs, int32_t experts, int32_t K, int32_t M)
{
    const int64_t tiles = weight_tiles(experts, K, M, 64, 64);
    if (tiles > kCus)
        return 1;
    const int64_t most = pairs / experts / (kBK * Tiny::kTeams * 4), wanted = kCus / tiles;
    const int64_t n = most < wanted ? most : wanted;
    return n > 1 ? (int32_t)n : 1;
}

int32_t experts_bias_tiles(int64_t pairs, int32_t experts)
{
    return (int32_t)((pairs + kActRows - 1) / kActRows + experts);
}

hipError_t launch_experts_forward(const ExpertsArgs& a, int dtype, hipStream_t stream)
{
    return dtype == SOFT_TOPK_BF16 ? forward<Bf16>(a, stream) : forward<F16>(a, stream);
}

hipError_t launch_experts_residual(const ExpertsArgs& a, void* dr, hipStream_t stream)
{
    const bool whole = ((reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(dr)) & 15) == 0;
    uint16_t* const to = static_cast<uint16_t*>(dr);
    const dim3 grid(kResidualBlocks), block(256);
    if (whole)
        STK_LAUNCH(kKExpertsBackward, stream, (experts_residual_kernel<true>), grid, block, 0, stream, a, to);
    else
        STK_LAUNCH(kKExpertsBackward, stream, (experts_residual_kernel<false>), grid, block, 0, stream, a, to);
    return hipGetLastError();
}

hipError_t launch_experts_backward(const ExpertsArgs& a, int dtype, hipStream_t stream)
{
    return dtype == SOFT_TOPK_BF16 ? backward<Bf16>(a, dtype, stream) : backward<F16>(a, dtype, stream);
}

}  // namespace stk
