// Products of 16-bit activations with MX fp4 weights for few rows, and the
// router and experts of a mixture-of-experts layer.
#pragma once

#include "common.hpp"
#include "norm_kernel.hpp"
#include "w4_stream.hpp"

namespace gr {
namespace w4 {

// ---- C = act(X W~^T + bias) -------------------------------------------------------

struct LinearArgs {
    const uint16_t* x;
    const uint8_t* w;
    const uint8_t* s;
    const uint16_t* bias;  // nullptr for none
    uint16_t* c;
    int64_t M, N, K, ldx, ldw, lds, ldc;
    int act;
    int kw;          // waves that share a unit's K: a power of two
    float* partial;  // split K: a matrix of M x ldp sums for each split, else nullptr
    int64_t ldp;
    int64_t span;    // k of one split, a multiple of 128
};

// The bias of a column: from LDS if it is among the workgroup's first ones.
template <typename E, typename Args>
__device__ __forceinline__ float staged_bias(const Args& a, const uint16_t* staged, uint32_t at, int64_t col) {
    return a.bias == nullptr ? 0.0f : E::widen(at < blockDim.x ? staged[at] : a.bias[col]);
}

// Rows of one column, `rows` of them there.
template <typename E, typename Args, int R>
__device__ __forceinline__ void write_rows(const Args& a, uint16_t* to, int64_t rows, float bias, Column<R> v) {
    act::dispatch(a.act, [&](auto tag) {
#pragma unroll
        for (int j = 0; j < R; ++j) v.v[j] = mx::exact_act<decltype(tag)::value>(v.v[j] + bias);
    });
#pragma unroll
    for (int j = 0; j < R; ++j)
        if (j < rows) to[j * a.ldc] = E::round(v.v[j]);
}

// 16 * MT rows of X from m0 on, and the k of one split.
template <typename E>
struct LinearUnits {
    static constexpr bool kPair = false;
    const LinearArgs& a;
    const uint8_t *w, *s;
    int64_t K, ldw, lds, m0, k0;
    float* partial;
    uint16_t* bias;  // LDS: the workgroup's first columns' bias, one per thread
    int u0;
    struct Run {
        int from, end;
    };
    __device__ __forceinline__ Run run(int u) const { return {u, 0x7FFFFFFF}; }
    __device__ __forceinline__ uint16_t early(int u0, int u1) const {
        const int64_t col = (int64_t)u0 * 16 + threadIdx.x;
        return a.bias != nullptr && col < (int64_t)u1 * 16 && col < a.N ? a.bias[col] : 0;
    }
    __device__ __forceinline__ void late(int, uint16_t v) const { bias[threadIdx.x] = v; }
    __device__ __forceinline__ Range range(int64_t k) const { return {k, K - k}; }
    __device__ __forceinline__ const uint16_t* x(const Run&, int, int m, const Range& range) const {
        return m0 + m < a.M ? a.x + (m0 + m) * a.ldx + k0 + range.k : nullptr;
    }
    __device__ __forceinline__ bool takes(const Range&, int) const { return true; }
    __device__ __forceinline__ int rows(const Run& run, int i) const {
        const int64_t left = a.N - (int64_t)(run.from + i) * 16;
        return left < 16 ? (int)left : 16;
    }
    __device__ __forceinline__ Tile tile(const Run& run, int i, const Range& range) const {
        const int64_t n = (int64_t)(run.from + i) * 16;
        return tile_at(w + n * ldw, ldw, s + n * lds, lds, rows(run, i), K, range.k);
    }
    __device__ __forceinline__ bool wanted(const Run& run, int i, int m, int n) const {
        return m0 + m < a.M && (int64_t)(run.from + i) * 16 + n < a.N;
    }
    template <int R>
    __device__ __forceinline__ void finish(const Run& run, int i, int m, int n, const Column<R>& v) const {
        const int64_t col = (int64_t)(run.from + i) * 16 + n, rows = a.M - (m0 + m);
        if (partial != nullptr) {
            float* const to = partial + (m0 + m) * a.ldp + col;
#pragma unroll
            for (int j = 0; j < R; ++j)
                if (j < rows) to[j * a.ldp] = v.v[j];
            return;
        }
        write_rows<E>(a, a.c + (m0 + m) * a.ldc + col, rows, staged_bias<E>(a, bias, (run.from - u0 + i) * 16 + n, col), v);
    }
};

// Registers for two workgroups of 8 waves, or one of 16, per CU with 16 rows of X, which
// take 64 of them.
constexpr int waves_per_simd(int MT, int PL, int ST) { return PL * ST <= 4 && MT == 1 ? 4 : 2; }

template <typename E, int NW, int MT, int ST, bool PASSES>
__global__ void __launch_bounds__(64 * NW, waves_per_simd(MT, 1, ST)) linear_w4_kernel(LinearArgs a) {
    // 16 waves: one batch of 8 units, as many as a workgroup has where N is below 2^15
    constexpr int TB = MT == 1 ? (NW == 16 && !PASSES ? 8 : 4) : 2, BUFS = NW == 16 ? 1 : 2;
    __shared__ Lds<NW, MT, TB, BUFS, PASSES> lds;
    const int64_t units = (a.N + 15) / 16;
    const int64_t k0 = blockIdx.z * a.span, K = a.K - k0 < a.span ? a.K - k0 : a.span;
    float* const partial = a.partial != nullptr ? a.partial + blockIdx.z * a.M * a.ldp : nullptr;
    __shared__ uint16_t bias[64 * NW];
    const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
    const LinearUnits<E> p{a,     a.w + k0 / 2, a.s + k0 / 32, K, a.ldw, a.lds, (int64_t)blockIdx.y * (16 * MT), k0,
                           partial, bias, u0};
    stream_units<E, 1, ST>(p, lds, u0, u1, a.kw);
}

// ---- both operands in MX fp4 --------------------------------------------------------

struct Fp4Args {
    const uint8_t *x, *sx, *w, *s;
    const uint16_t* bias;  // nullptr for none
    uint16_t* c;
    int64_t M, N, K, ldx, ldsx, ldw, lds, ldc;
    int act;
    int kw;
};

// E: the output's type.
template <typename E>
struct Fp4Units {
    static constexpr bool kPair = false;
    const Fp4Args& a;
    int64_t K, ldw, lds, m0;
    uint16_t* bias;  // as in LinearUnits
    int u0;
    struct Run {
        int from, end;
    };
    __device__ __forceinline__ Run run(int u) const { return {u, 0x7FFFFFFF}; }
    __device__ __forceinline__ uint16_t early(int u0, int u1) const {
        const int64_t col = (int64_t)u0 * 16 + threadIdx.x;
        return a.bias != nullptr && col < (int64_t)u1 * 16 && col < a.N ? a.bias[col] : 0;
    }
    __device__ __forceinline__ void late(int, uint16_t v) const { bias[threadIdx.x] = v; }
    __device__ __forceinline__ Range range(int64_t k) const { return {k, K - k}; }
    __device__ __forceinline__ const uint8_t* x(int m, const Range& range) const {
        return m0 + m < a.M ? a.x + (m0 + m) * a.ldx + range.k / 2 : nullptr;
    }
    __device__ __forceinline__ const uint8_t* x_scale(int m, const Range& range) const {
        return a.sx + (m0 + m) * a.ldsx + range.k / 32;
    }
    __device__ __forceinline__ int rows(const Run& run, int i) const {
        const int64_t left = a.N - (int64_t)(run.from + i) * 16;
        return left < 16 ? (int)left : 16;
    }
    __device__ __forceinline__ Tile tile(const Run& run, int i, const Range& range) const {
        const int64_t n = (int64_t)(run.from + i) * 16;
        return tile_at(a.w + n * ldw, ldw, a.s + n * lds, lds, rows(run, i), K, range.k);
    }
    __device__ __forceinline__ bool wanted(const Run& run, int i, int m, int n) const {
        return m0 + m < a.M && (int64_t)(run.from + i) * 16 + n < a.N;
    }
    template <int R>
    __device__ __forceinline__ void finish(const Run& run, int i, int m, int n, const Column<R>& v) const {
        const int64_t col = (int64_t)(run.from + i) * 16 + n;
        write_rows<E>(a, a.c + (m0 + m) * a.ldc + col, a.M - (m0 + m),
                      staged_bias<E>(a, bias, (run.from - u0 + i) * 16 + n, col), v);
    }
};

template <typename E, int MT, int ST, bool PASSES>
__global__ void __launch_bounds__(512, 4) fp4_stream_kernel(Fp4Args a) {
    // few units per barrier, so that two workgroups' sums fit in LDS
    constexpr int TB = 4 / MT;
    __shared__ Lds<8, MT, TB, 2, PASSES> lds;
    __shared__ uint16_t bias[512];
    const int64_t units = (a.N + 15) / 16;
    const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
    const Fp4Units<E> p{a, a.K, a.ldw, a.lds, (int64_t)blockIdx.y * (16 * MT), bias, u0};
    stream_units<ElemFp4, 1, ST>(p, lds, u0, u1, a.kw);
}

// C from the splits' sums, added in order; 4 columns per thread.
constexpr int kSumThreads = 256;

template <typename E>
__global__ void __launch_bounds__(kSumThreads) linear_w4_sum_kernel(LinearArgs a) {
    const int64_t n = ((int64_t)blockIdx.x * kSumThreads + threadIdx.x) * 4, m = blockIdx.y;
    if (n >= a.N) return;
    const int splits = (int)((a.K + a.span - 1) / a.span);
    const float* p = a.partial + m * a.ldp + n;
    f32x4 v = *(const f32x4*)p;
    for (int s = 1; s < splits; ++s) {
        p += a.M * a.ldp;
        const f32x4 w = *(const f32x4*)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += w[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < a.N) {
            float x = v[i];
            if (a.bias != nullptr) x += E::widen(a.bias[n + i]);
            a.c[m * a.ldc + n + i] = E::round(mx::exact_activate(x, a.act));
        }
}

// ---- mixture of experts -----------------------------------------------------------
//
//   out[t] = sum_j weight[t][j] * (W2[e] * h + b2[e]),  h = act(g) * u,
//   (g, u) = W13[e] * x[t] + b13[e],  e = id[t][j]
//
// Three kernels, the first two on the core above: h for every (expert, token)
// pair; y = W2[e] * (weight * h) for every pair, in fp32; a token's sum over its
// pairs.  They work on the experts that at least one token chose, so each of
// their weights is read once, and on chunks of 64 tokens (a bit each in an expert's
// 64-bit set).  Pairs are numbered by expert, then token: the number is the row of
// h and y.  h holds weight * act(g) * u in two bfloat16 parts (high and the
// rest's high: 16 bits and fp32's range, infinities included), so that the second
// product starts from nearly fp32 values.
//
// 32 tokens with 8 of 64 experts, 4096 x 2048: 113 us for the first product (561 MB,
// 5.0 TB/s), 67 for the second (295 MB, 4.4 TB/s), 5 for the sum.  One token with 4
// experts of 2048 x 1024: 9 and 6 us, a launch, the ids and a trip for the weights each.

constexpr int kChunk = 64;         // tokens per chunk
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
// Which tokens chose which expert, for one chunk, in dynamic LDS: as much as E
// experts and topk choices need.
struct Routing {
    unsigned long long* tokens;  // of each expert
    uint16_t* expert;            // the chosen experts, ascending
    uint16_t* row;               // first pair of each; [chosen]: pairs in all
    uint16_t* row_of;            // the same by expert number
    uint16_t* tile;              // tiles of 16 pairs: slot in `expert` * 4 + tile of that expert
    float* weight;               // a pair's weight (gate and up)
    uint8_t* token;              // a pair's token
    int tiles;
};

// sum over the experts of ceil(pairs / 16) < experts + pairs / 16
__host__ __device__ constexpr int max_tiles(int E, int topk) { return E + kChunk * topk / 16; }
__host__ __device__ constexpr int routing_bytes(int E, int topk) {
    return 8 * E + 8 + 3 * 4 * kChunk * topk + 2 * (3 * E + 2 + max_tiles(E, topk)) + kChunk * topk;
}

// The tables for at most 8 choices: lane 8i + q holds choice i next to choice q, so one
// comparison serves all pairs of choices, and the 8 bits of a ballot that belong to
// i count.  Every wave fills the tables with the same values and reads only after its
// own writes, so there is no barrier.
constexpr int kFewChoices = 8;

__device__ __forceinline__ void route_few(Routing& r, const int32_t* ids, const float* weights, int32_t* pair, int n,
                                          int topk, int E) {
    const int lane = threadIdx.x % 64, i = lane / 8, q = lane % 8, count = n * topk;
    const int e = i < count ? ids[i] : -1, eq = q < count ? ids[q] : -1;
    const int t = (uint32_t)i / (uint32_t)topk, tq = (uint32_t)q / (uint32_t)topk;
    const float share = weights != nullptr && q < count ? weights[q] : 0.0f;
    const auto bits = [&](bool x) { return (uint32_t)(__ballot(x) >> (8 * i)) & 255u; };  // q's, of this i
    // choices of the same expert by the same token are one pair, with their weights' sum
    const bool same = e == eq && t == tq;
    const unsigned long long again = __ballot(same && q < i);
    const bool is = (uint32_t)e < (uint32_t)E && (again >> (8 * i) & 255u) == 0;
    const bool is_q = (uint32_t)eq < (uint32_t)E && (again >> (8 * q) & 255u) == 0;
    const int row = __popc(bits(is_q && (eq < e || (eq == e && tq < t))));
    const bool first = is && bits(is_q && eq == e && tq < t) == 0;
    float weight = same ? share : 0.0f;
    uint32_t tokens = is_q && eq == e ? 1u << tq : 0u;
    weight += mx::dppf<mx::kQuadXor1>(weight);
    tokens |= mx::dpp<mx::kQuadXor1>(tokens);
    weight += mx::dppf<mx::kQuadXor2>(weight);
    tokens |= mx::dpp<mx::kQuadXor2>(tokens);
    weight += mx::dppf<mx::kRowHalfMirror>(weight);
    tokens |= mx::dpp<mx::kRowHalfMirror>(tokens);
    const unsigned long long experts = __ballot(first && q == 0);
    const int slot = __popc(bits((experts >> (8 * q) & 1) != 0 && eq < e));
    const int pairs = __popcll(__ballot(is && q == 0));
    r.tiles = __popcll(experts);
    if (q == 0) {
        if (is) {
            r.token[row] = (uint8_t)t;
            r.weight[row] = weight;
        }
        if (first) {
            r.tokens[e] = tokens;
            r.expert[slot] = (uint16_t)e;
            r.row[slot] = (uint16_t)row;
            r.tile[slot] = (uint16_t)(slot * 4);
        }
        if (pair != nullptr && i < count && threadIdx.x < 64) pair[i] = is ? row : -1;
    }
    if (lane == 0) r.row[r.tiles] = (uint16_t)pairs;
}

// The routing of the chunk's ids (n tokens x topk); called by the whole
// workgroup.  Ids outside [0, E) choose nothing, and a token that names an
// expert twice is one pair.  With `weights` each pair's weight is put down too, and
// with `pair` the pair of each choice (-1: none, or named before).
__device__ __forceinline__ Routing route(const int32_t* ids, const float* weights, int32_t* pair, int n, int topk,
                                         int E) {
    extern __shared__ unsigned long long routing_lds[];
    Routing r;
    r.tokens = routing_lds;
    int* const tiles_of_all = reinterpret_cast<int*>(r.tokens + E);
    r.weight = reinterpret_cast<float*>(tiles_of_all + 2);
    int32_t* const id = reinterpret_cast<int32_t*>(r.weight + kChunk * topk);
    float* const share = reinterpret_cast<float*>(id + kChunk * topk);
    r.expert = reinterpret_cast<uint16_t*>(share + kChunk * topk);
    r.row = r.expert + E + 1;
    r.row_of = r.row + E + 1;
    r.tile = r.row_of + E;
    r.token = reinterpret_cast<uint8_t*>(r.tile + max_tiles(E, topk));
    if (n * topk <= kFewChoices) {
        route_few(r, ids, weights, pair, n, topk, E);
        return r;
    }
    for (int i = threadIdx.x; i < n * topk; i += blockDim.x) {
        id[i] = ids[i];
        if (weights != nullptr) share[i] = weights[i];
    }
    for (int e = threadIdx.x; e < E; e += blockDim.x) r.tokens[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n * topk; i += blockDim.x) {
        const uint32_t e = (uint32_t)id[i];
        if (e < (uint32_t)E) atomicOr(&r.tokens[e], 1ull << (i / topk));
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int count = 0, rows = 0, tiles = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + lane;
            const unsigned long long set = e < E ? r.tokens[e] : 0;
            const unsigned long long chosen = __ballot(set != 0);
            const int pairs = __popcll(set);
            const int mine = pairs | (pairs + 15) / 16 << 16;  // both sums in one: at most 4096 pairs, 256 tiles
            int upto = mine;                                   // inclusive, over the lanes
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int o = __shfl_up(upto, d);
                if (lane >= d) upto += o;
            }
            if (set != 0) {
                const int at = count + __popcll(chosen & ((1ull << lane) - 1));
                const uint16_t row = (uint16_t)(rows + ((upto - mine) & 0xFFFF));
                r.expert[at] = (uint16_t)e;
                r.row[at] = row;
                r.row_of[e] = row;
                const int first = tiles + ((upto - mine) >> 16);
                for (int i = 0; i * 16 < pairs; ++i) r.tile[first + i] = (uint16_t)(at * 4 + i);
            }
            const int all = __shfl(upto, 63);
            count += __popcll(chosen);
            rows += all & 0xFFFF;
            tiles += all >> 16;
        }
        if (lane == 0) {
            r.row[count] = (uint16_t)rows;
            *tiles_of_all = tiles;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * topk; i += blockDim.x) {
        const int32_t e = id[i];
        const int t = i / topk, j = i % topk;
        int row = -1;
        if ((uint32_t)e < (uint32_t)E) {
            row = r.row_of[e] + __popcll(r.tokens[e] & ((1ull << t) - 1));
            float weight = 0.0f;
            for (int q = 0; q < topk; ++q)
                if (id[t * topk + q] == e) {
                    if (q < j) row = -1;
                    if (weights != nullptr) weight += share[t * topk + q];
                }
            if (row >= 0) {
                r.token[row] = (uint8_t)t;
                r.weight[row] = weight;
            }
        }
        if (pair != nullptr) pair[i] = row;
    }
    r.tiles = __builtin_amdgcn_readfirstlane(*tiles_of_all);
    __syncthreads();
    return r;
}

struct MoeArgs {
    const uint16_t* x;
    const int32_t* ids;
    const float* weights;
    const uint8_t *w13, *s13, *w2, *s2;
    const uint16_t *b13, *b2;  // nullptr for none
    uint16_t* h;               // two planes of T * topk rows of I (bfloat16)
    float* y;                  // T * topk rows of H
    int32_t* pair;             // T x topk: the row of h and y of each choice, -1 for none
    uint16_t* c;
    int64_t T, H, I, ldx, ldc;
    int E, topk, act;
    int kw13, kw2;             // waves that share a unit's K in the two products
};

// Units with the same X: a tile of pairs of one expert.
struct MoeRun {
    int end, expert, row, pairs, col;  // row: the tile's first pair; pairs: from there to the expert's end
};

// item: 16 columns for a tile of pairs, `tiles` for each.
__device__ __forceinline__ MoeRun moe_run(const Routing& r, int item, int tiles) {
    const int tile = item / tiles;
    const int at = __builtin_amdgcn_readfirstlane(r.tile[tile]);
    const int row = __builtin_amdgcn_readfirstlane(r.row[at / 4]) + at % 4 * 16;
    return {(tile + 1) * tiles, __builtin_amdgcn_readfirstlane(r.expert[at / 4]), row,
            __builtin_amdgcn_readfirstlane(r.row[at / 4 + 1]) - row, (item - tile * tiles) * 16};
}

// The items [first, last) of a workgroup, `tiles` for each tile of pairs: all of one
// tile of pairs where there are workgroups enough (a change of X costs a trip to
// memory), else an equal share of all.
struct Items {
    int first, last;
};

__device__ __forceinline__ Items items_of(int pair_tiles, int tiles) {
    const int wgs = gridDim.x, wg = blockIdx.x;
    if (pair_tiles > wgs) {
        const int64_t all = (int64_t)pair_tiles * tiles;
        return {(int)(all * wg / wgs), (int)(all * (wg + 1) / wgs)};
    }
    if (pair_tiles == 0) return {0, 0};
    const int each = wgs / pair_tiles, tile = wg / each, part = wg % each;
    if (tile >= pair_tiles) return {0, 0};
    return {tile * tiles + (int)((int64_t)tiles * part / each), tile * tiles + (int)((int64_t)tiles * (part + 1) / each)};
}

constexpr float kBf16Max = 0x1.FEp127f;

// Units of the first product: 16 columns of h for a tile of pairs, gate and up.
template <typename E>
struct GateUpUnits {
    static constexpr bool kPair = true;
    const MoeArgs& a;
    const Routing& r;
    int64_t K, ldw, lds, t0;
    int tiles;  // of 16 columns of h
    __device__ __forceinline__ int early(int, int) const { return 0; }
    __device__ __forceinline__ void late(int, int) const {}
    __device__ __forceinline__ MoeRun run(int u) const {
        MoeRun run = moe_run(r, u / 2, tiles);
        run.end *= 2;
        return run;
    }
    __device__ __forceinline__ Range range(int64_t k) const { return {k, K - k}; }
    __device__ __forceinline__ const uint16_t* x(const MoeRun& run, int, int m, const Range& range) const {
        return m < run.pairs ? a.x + (t0 + r.token[run.row + m]) * a.ldx + range.k : nullptr;
    }
    __device__ __forceinline__ bool takes(const Range&, int) const { return true; }
    __device__ __forceinline__ int rows(const MoeRun&, int) const { return 16; }  // H and I are multiples of 16
    __device__ __forceinline__ Tile tile(const MoeRun& run, int i, const Range& range) const {
        const int64_t n = (2 * (int64_t)run.expert + i % 2) * a.I + run.col + i / 2 * 16;
        return tile_at(a.w13 + n * ldw, ldw, a.s13 + n * lds, lds, 16, K, range.k);
    }
    __device__ __forceinline__ bool wanted(const MoeRun& run, int, int m, int) const { return m < run.pairs; }
    __device__ __forceinline__ void finish(const MoeRun& run, int i, int m, int n, const Column<1>& gate,
                                           const Column<1>& up) const {
        const int64_t col = run.col + i / 2 * 16 + n;
        float g = gate.v[0], v = up.v[0];
        if (a.b13 != nullptr) {
            g += E::widen(a.b13[2 * (int64_t)run.expert * a.I + col]);
            v += E::widen(a.b13[(2 * (int64_t)run.expert + 1) * a.I + col]);
        }
        const float h = mx::exact_activate(g, a.act) * v * r.weight[run.row + m];
        // (a finite h never has an infinite high part, and an infinite one has no low part)
        const float high = __builtin_amdgcn_fmed3f(h, -kBf16Max, kBf16Max);
        const bool finite = __builtin_fabsf(h) < __builtin_inff();
        const uint16_t part = to_bf16(finite ? high : h);
        const int64_t to = (t0 * a.topk + run.row + m) * a.I + col;
        a.h[to] = part;
        a.h[a.T * a.topk * a.I + to] = finite ? to_bf16(h - ElemBF16::widen(part)) : 0;
    }
};

constexpr int kMoeBatch = 4;

template <typename E, int NW, int ST, bool PASSES>
__global__ void __launch_bounds__(64 * NW, waves_per_simd(1, 1, ST)) moe_gate_up_kernel(MoeArgs a) {
    __shared__ Lds<NW, 1, kMoeBatch, NW == 16 ? 1 : 2, PASSES> lds;
    const int64_t t0 = (int64_t)blockIdx.y * kChunk;
    const int n_tok = (int)(a.T - t0 < kChunk ? a.T - t0 : kChunk);
    const int64_t first = t0 * a.topk;
    const Routing r =
        route(a.ids + first, a.weights + first, blockIdx.x == 0 ? a.pair + first : nullptr, n_tok, a.topk, a.E);
    const int tiles = (int)(a.I / 16);
    const GateUpUnits<E> p{a, r, a.H, a.H / 2, a.H / 32, t0, tiles};
    const Items items = items_of(r.tiles, tiles);
    stream_units<E, 1, ST>(p, lds, items.first * 2, items.last * 2, a.kw13);
}

// Units of the second product: 16 columns of the output for a tile of pairs.
struct DownUnits {
    static constexpr bool kPair = false;
    const MoeArgs& a;
    const Routing& r;
    int64_t K, ldw, lds, first;  // first: the chunk's first row of h and y
    int tiles;                   // of 16 columns
    __device__ __forceinline__ int early(int, int) const { return 0; }
    __device__ __forceinline__ void late(int, int) const {}
    __device__ __forceinline__ MoeRun run(int u) const { return moe_run(r, u, tiles); }
    __device__ __forceinline__ Range range(int64_t k) const { return {k, K - k}; }
    __device__ __forceinline__ const uint16_t* x(const MoeRun& run, int plane, int m, const Range& range) const {
        return m < run.pairs ? a.h + (plane * (a.T * a.topk) + first + run.row + m) * a.I + range.k : nullptr;
    }
    __device__ __forceinline__ bool takes(const Range&, int) const { return true; }
    __device__ __forceinline__ int rows(const MoeRun&, int) const { return 16; }  // H and I are multiples of 16
    __device__ __forceinline__ Tile tile(const MoeRun& run, int i, const Range& range) const {
        const int64_t n = (int64_t)run.expert * a.H + run.col + i * 16;
        return tile_at(a.w2 + n * ldw, ldw, a.s2 + n * lds, lds, 16, K, range.k);
    }
    __device__ __forceinline__ bool wanted(const MoeRun& run, int, int m, int) const { return m < run.pairs; }
    __device__ __forceinline__ void finish(const MoeRun& run, int i, int m, int n, const Column<1>& v) const {
        a.y[(first + run.row + m) * a.H + run.col + i * 16 + n] = v.v[0];
    }
};

template <int NW, int ST, bool PASSES>
__global__ void __launch_bounds__(64 * NW, waves_per_simd(1, 2, ST)) moe_down_kernel(MoeArgs a) {
    __shared__ Lds<NW, 1, kMoeBatch, NW == 16 ? 1 : 2, PASSES> lds;
    const int64_t t0 = (int64_t)blockIdx.y * kChunk;
    const int n_tok = (int)(a.T - t0 < kChunk ? a.T - t0 : kChunk);
    const Routing r = route(a.ids + t0 * a.topk, nullptr, nullptr, n_tok, a.topk, a.E);
    const int tiles = (int)(a.H / 16);
    const DownUnits p{a, r, a.I, a.I / 2, a.I / 32, t0 * a.topk, tiles};
    const Items items = items_of(r.tiles, tiles);
    stream_units<ElemBF16, 2, ST>(p, lds, items.first, items.last, a.kw2);
}

// The second product for few tokens and few chosen experts, with the sum over the experts
// in it: the experts' rows of W2 side by side are one long K, of which a wave holds a
// part of one expert; row m of X is token m's h where it chose that expert, else 0.
constexpr int kFewTokens = 16;
constexpr int kFewSteps = 2;

template <typename E>
struct DownFewUnits {
    static constexpr bool kPair = false;
    const MoeArgs& a;
    const Routing& r;
    int64_t K, ldw, lds;
    int parts;  // of kFewSteps * 128 k of one expert
    struct Run {
        int from, end;
    };
    struct Range {
        int64_t k, left;
        int expert, row;  // the expert's first pair
        unsigned long long tokens;
    };
    __device__ __forceinline__ int early(int, int) const { return 0; }
    __device__ __forceinline__ void late(int, int) const {}
    __device__ __forceinline__ Run run(int u) const { return {u, 0x7FFFFFFF}; }
    __device__ __forceinline__ Range range(int64_t k) const {
        const int part = (int)(k / (128 * kFewSteps)), slot = part / parts;
        if (slot >= r.tiles) return {0, 0, 0, 0, 0};
        const int64_t at = (int64_t)(part - slot * parts) * (128 * kFewSteps);
        const int e = __builtin_amdgcn_readfirstlane(r.expert[slot]);
        return {at, a.I - at, e, __builtin_amdgcn_readfirstlane(r.row[slot]), r.tokens[e]};
    }
    // (a token's h is 0 in the parts of the experts that it did not choose)
    __device__ __forceinline__ bool takes(const Range& range, int m) const { return (range.tokens >> m & 1) != 0; }
    __device__ __forceinline__ const uint16_t* x(const Run&, int plane, int m, const Range& range) const {
        if (!takes(range, m)) return nullptr;
        const int row = range.row + __popcll(range.tokens & ((1ull << m) - 1));
        return a.h + (plane * (a.T * a.topk) + row) * a.I + range.k;
    }
    __device__ __forceinline__ int rows(const Run&, int) const { return 16; }
    __device__ __forceinline__ Tile tile(const Run& run, int i, const Range& range) const {
        const int64_t n = (int64_t)range.expert * a.H + (run.from + i) * 16;
        return tile_at(a.w2 + n * ldw, ldw, a.s2 + n * lds, lds, 16, a.I, range.k);
    }
    __device__ __forceinline__ bool wanted(const Run&, int, int m, int) const { return m < a.T; }
    __device__ __forceinline__ void finish(const Run& run, int i, int m, int n, const Column<1>& sum) const {
        const int64_t col = (run.from + i) * 16 + n;
        float v = sum.v[0];
        if (a.b2 != nullptr) {
            for (int j = 0; j < a.topk; ++j) {
                const uint32_t e = (uint32_t)a.ids[m * a.topk + j];
                if (e < (uint32_t)a.E)
                    v = __builtin_fmaf(a.weights[m * a.topk + j], E::widen(a.b2[(int64_t)e * a.H + col]), v);
            }
        }
        a.c[m * a.ldc + col] = E::round(v);
    }
};

template <typename E, bool PASSES>
__global__ void __launch_bounds__(1024, 4) moe_down_few_kernel(MoeArgs a) {
    __shared__ Lds<16, 1, 4, 1, PASSES> lds;
    const Routing r = route(a.ids, nullptr, nullptr, (int)a.T, a.topk, a.E);
    const int parts = (int)((a.I + 128 * kFewSteps - 1) / (128 * kFewSteps)), units = (int)(a.H / 16);
    const DownFewUnits<E> p{a, r, (int64_t)r.tiles * parts * (128 * kFewSteps), a.I / 2, a.I / 32, parts};
    stream_units<ElemBF16, 2, kFewSteps>(p, lds, (int)((int64_t)units * blockIdx.x / gridDim.x),
                                         (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x), 16);
}

// out: 4 columns per thread; the sum goes through a token's choices in order.
constexpr int kCombineThreads = 256;

template <typename E>
__global__ void __launch_bounds__(kCombineThreads) moe_combine_kernel(MoeArgs a) {
    const int64_t col = ((int64_t)blockIdx.x * kCombineThreads + threadIdx.x) * 4;
    if (col >= a.H) return;
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        const int64_t first = t / kChunk * kChunk * a.topk;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (a.I > 0) {
            for (int j = 0; j < a.topk; ++j) {
                const int row = a.pair[t * a.topk + j];
                if (row >= 0) {
                    const f32x4 y = *(const f32x4*)(a.y + (first + row) * a.H + col);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] += y[i];
                }
            }
        }
        if (a.b2 != nullptr) {
            for (int j = 0; j < a.topk; ++j) {
                const uint32_t e = (uint32_t)a.ids[t * a.topk + j];
                if (e < (uint32_t)a.E) {
                    const float weight = a.weights[t * a.topk + j];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = __builtin_fmaf(weight, E::widen(a.b2[(int64_t)e * a.H + col + i]), v[i]);
                }
            }
        }
        u32x2 out;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            out[i] = (uint32_t)E::round(v[2 * i]) | (uint32_t)E::round(v[2 * i + 1]) << 16;
        *(u32x2_any*)(a.c + t * a.ldc + col) = out;
    }
}

// ---- router ------------------------------------------------------------------------
//
//   logit[t][e] = sum_k x[t][k] * Wr[e][k] + bias[e], fp32
//   the topk largest, in order (ties: lower index first; NaN above infinity),
//   weight[j] = exp(logit_j - max) / sum over the chosen (renorm) or over all E
//
// One kernel: a workgroup takes 16 tokens and every expert.  Its waves share K, each with
// a few steps of 32 k for NT tiles of 16 experts in flight at once.  The logits meet
// in LDS, and each wave then picks for one token.  One CU reads some 35 KB a
// microsecond: 4096 x 64 takes 20 us for one token.
// Few tokens and a large Wr take two: logits of 16 tokens and 16 experts over slices
// of 512 k by a workgroup each, partial sums to the workspace; then a wave per token
// adds the slices in order and picks.

constexpr int kRouteWaves = 16;
constexpr int kRouteThreads = 64 * kRouteWaves;

struct RouteArgs {
    const uint16_t* x;
    const uint16_t* w;
    const float* bias;  // nullptr for none
    int32_t* ids;
    float* weights;
    int64_t T, H, ldx, ldw;
    int E, topk, renorm;
    float* partial;  // two kernels: slices x T x E
};

// Order-preserving bits of a float, at least 1; NaN above everything.
__device__ __forceinline__ uint32_t order_bits(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    if ((b & mx::kAbsMask) > mx::kInfBits) return 0xFFFFFFFFu;
    // -0 and +0 are equal
    const uint32_t z = (b & mx::kAbsMask) == 0 ? 0u : b;
    return (z & 0x80000000u) != 0 ? ~z : z | 0x80000000u;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    const auto most = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    x = most(x, mx::dpp<mx::kQuadXor1>(x));
    x = most(x, mx::dpp<mx::kQuadXor2>(x));
    x = most(x, mx::dpp<mx::kRowHalfMirror>(x));
    x = most(x, mx::dpp<mx::kRowMirror>(x));
    return mx::over_32(mx::over_16(x, most), most);
}

// The topk of one token's E logits, by one wave; PER logits per lane (expert
// = lane + 64 * i).
template <int PER, typename F>
__device__ __forceinline__ void pick(F logit_of, int E, int topk, int renorm, int32_t* ids, float* weights) {
    const int lane = threadIdx.x % 64;
    float v[PER];
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        v[i] = e < E ? logit_of(e) : 0.0f;
        key[i] = e < E ? order_bits(v[i]) : 0u;
    }
    int my_id = 0;
    float my_logit = 0.0f, top = 0.0f;
    for (int j = 0; j < topk; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) m = key[i] > m ? key[i] : m;
        m = (uint32_t)__builtin_amdgcn_readfirstlane((int)wave_max(m));
        int id = 0, owner = -1;
        float logit = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const unsigned long long has = __ballot(key[i] == m);
            if (owner < 0 && has != 0) {
                owner = __ffsll(has) - 1;
                id = owner + 64 * i;
                logit = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v[i]), owner));
                if (lane == owner) key[i] = 0;
            }
        }
        if (j == 0) top = logit;
        if (lane == j) {
            my_id = id;
            my_logit = logit;
        }
    }
    // exp(x - top) of the chosen, in lanes 0 .. topk - 1, or of all for the sum
    const float mine = lane < topk ? expf(my_logit - top) : 0.0f;
    float sum = mine;
    if (!renorm) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 64 * i < E) sum += expf(v[i] - top);
    }
    sum = mx::wave_sum(sum);
    if (lane < topk) {
        ids[lane] = my_id;
        weights[lane] = mine / sum;
    }
}

// acc[nt] += X times tile nt of Wr over the steps [first, last) of 32 k, U of them in
// flight; x and w are the lane's rows.
template <typename E, int NT, int U>
__device__ __forceinline__ void route_product(const uint16_t* x, const uint16_t* const (&w)[NT], int64_t H,
                                              int64_t first, int64_t last, f32x4 (&acc)[NT]) {
    const int g = threadIdx.x % 64 / 16;
    const int64_t whole = H / 32, until = last < whole ? last : whole;
    for (int64_t k = first; k < until; k += U) {
        u32x4 xv[U], wv[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k + u < until) {
                xv[u] = *(const u32x4_any*)(x + (k + u) * 32 + g * 8);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) wv[u][nt] = *(const u32x4_any*)(w[nt] + (k + u) * 32 + g * 8);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k + u < until) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    acc[nt] =
                        E::mfma16(__builtin_bit_cast(f16x8, xv[u]), __builtin_bit_cast(f16x8, wv[u][nt]), acc[nt]);
            }
    }
    if (whole < last && whole >= first) {  // the tail of H: absent values are 0 on both sides
        const int left = (int)(H - whole * 32) - g * 8, n = left < 8 ? left : 8;
        u32x4 xt = {0u, 0u, 0u, 0u};
        if (n > 0) xt = mx::load8(x + whole * 32 + g * 8, n);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            u32x4 wt = {0u, 0u, 0u, 0u};
            if (n > 0) wt = mx::load8(w[nt] + whole * 32 + g * 8, n);
            acc[nt] = E::mfma16(__builtin_bit_cast(f16x8, xt), __builtin_bit_cast(f16x8, wt), acc[nt]);
        }
    }
}

// NT tiles of 16 experts at a time; PER * 64 experts at most.
template <typename E, int NT, int PER>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(RouteArgs a) {
    __shared__ float part[kRouteWaves][NT][256];
    __shared__ float logits[16][64 * PER];
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t t0 = (int64_t)blockIdx.x * 16;
    const int64_t t = t0 + lane % 16 < a.T ? t0 + lane % 16 : a.T - 1;
    const int64_t steps = (a.H + 31) / 32;
    for (int e0 = 0; e0 < a.E; e0 += 16 * NT) {
        const uint16_t* w[NT];
        f32x4 acc[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int e = e0 + nt * 16 + lane % 16 < a.E ? e0 + nt * 16 + lane % 16 : a.E - 1;
            w[nt] = a.w + (int64_t)e * a.ldw;
            acc[nt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        route_product<E, NT, NT == 4 ? 2 : 4>(a.x + t * a.ldx, w, a.H, steps * wave / kRouteWaves,
                                              steps * (wave + 1) / kRouteWaves, acc);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) *(f32x4*)&part[wave][nt][lane * 4] = acc[nt];
        __syncthreads();
        for (int i = threadIdx.x; i < NT * 256; i += kRouteThreads) {
            const int nt = i / 256, at = i % 256, m = at / 64 * 4 + at % 4, e = e0 + nt * 16 + at / 4 % 16;
            float v = 0.0f;
#pragma unroll
            for (int j = 0; j < kRouteWaves; ++j) v += part[j][nt][at];
            if (e < a.E) {
                if (a.bias != nullptr) v += a.bias[e];
                logits[m][e] = v;
            }
        }
        __syncthreads();
    }
    const int64_t mine = t0 + wave;
    if (mine < a.T)
        pick<PER>([&](int e) { return logits[wave][e]; }, a.E, a.topk, a.renorm, a.ids + mine * a.topk,
                  a.weights + mine * a.topk);
}

constexpr int kSliceSteps = 16;  // of 32 k
constexpr int kSliceWaves = 4;
constexpr int kPickWaves = 4;

// Grid: tiles of 16 experts, slices, tiles of 16 tokens.
template <typename E>
__global__ void __launch_bounds__(64 * kSliceWaves) moe_logits_kernel(RouteArgs a) {
    __shared__ float part[kSliceWaves][256];
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t t0 = (int64_t)blockIdx.z * 16;
    const int64_t t = t0 + lane % 16 < a.T ? t0 + lane % 16 : a.T - 1;
    const int e0 = blockIdx.x * 16, e = e0 + lane % 16 < a.E ? e0 + lane % 16 : a.E - 1;
    const int64_t steps = (a.H + 31) / 32, first = (int64_t)blockIdx.y * kSliceSteps;
    const int64_t mine = first + wave * (kSliceSteps / kSliceWaves), past = mine + kSliceSteps / kSliceWaves;
    const uint16_t* const w[1] = {a.w + (int64_t)e * a.ldw};
    f32x4 acc[1] = {};
    route_product<E, 1, kSliceSteps / kSliceWaves>(a.x + t * a.ldx, w, a.H, mine, past < steps ? past : steps, acc);
    *(f32x4*)&part[wave][lane * 4] = acc[0];
    __syncthreads();
    const int at = threadIdx.x, m = at / 64 * 4 + at % 4, col = e0 + at / 4 % 16;
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < kSliceWaves; ++j) v += part[j][at];
    if (t0 + m < a.T && col < a.E) a.partial[((int64_t)blockIdx.y * a.T + t0 + m) * a.E + col] = v;
}

template <int PER>
__global__ void __launch_bounds__(64 * kPickWaves) moe_pick_kernel(RouteArgs a) {
    const int64_t t = (int64_t)blockIdx.x * kPickWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    if (t >= a.T) return;
    const int slices = (int)((a.H + 32 * kSliceSteps - 1) / (32 * kSliceSteps));
    pick<PER>(
        [&](int e) {
            float v = 0.0f;
#pragma unroll 8
            for (int s = 0; s < slices; ++s) v += a.partial[((int64_t)s * a.T + t) * a.E + e];
            return a.bias != nullptr ? v + a.bias[e] : v;
        },
        a.E, a.topk, a.renorm, a.ids + t * a.topk, a.weights + t * a.topk);
}

}  // namespace w4
}  // namespace gr
