// Element types that bring an epilogue of their own to the transposed-B kernels
// (tile3t, tile128, the row-blocked stream and the small-M stream): the products
// of training.
//
//   Plain   C = round(acc)
//   Two     the same for two products at once, and sums over rows
//   Gated   rows n and n + half of Bt are a pair: C[m][n] = act(g + b) * (u + b'),
//           with (g, u) the pair's sums in fp32; optionally g and u themselves, rounded,
//           for a backward pass
//   Poly    C = round(alpha acc + beta D + diag I) over a batch, D of C's shape and
//           element type, with C written a second time transposed; TRI: C is symmetric,
//           only tiles on or below the diagonal are computed
//
// A wave stages its accumulators 32 rows at a time in LDS of its own as fp32
// and reads them back with 8 consecutive columns per lane, so that every operand
// of the epilogue and every store is 16 bytes per lane in whole row segments.  After the
// first barrier the LDS is the wave's alone, and a wave's LDS operations complete in
// order.
#pragma once

#include "norm_kernel.hpp"

namespace gr {
namespace own {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Two values rounded to nearest even and packed (v_cvt_pk_bf16_f32; two
// v_cvt_f16_f32).
template <typename E>
__device__ __forceinline__ uint32_t round2(float a, float b) {
    if constexpr (E::kIsF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
template <typename E>
__device__ __forceinline__ u32x4 round8(const float (&v)[8]) {
    return u32x4{round2<E>(v[0], v[1]), round2<E>(v[2], v[3]), round2<E>(v[4], v[5]), round2<E>(v[6], v[7])};
}
template <typename E>
__device__ __forceinline__ float widen8(const u32x4& v, int i) {
    return E::widen((uint16_t)(v[i / 2] >> (16 * (i % 2))));
}

// Columns n .. n + 7 of a row, those in [n_min, N) only; dst is column n.
template <bool EDGE, bool NT = true>
__device__ __forceinline__ void put8(uint16_t* dst, const u32x4& v, int64_t n, int64_t n_min, int64_t N) {
    if (!EDGE || (n >= n_min && n + 8 <= N)) {
        if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(dst));
        else *reinterpret_cast<u32x4_any*>(dst) = v;
    } else {
        const int64_t first = n < n_min ? n_min - n : 0;
        const int64_t end = N - n < 8 ? N - n : 8;
        if (end > first) epi::store_run(dst, v, (int)first, (int)(end - first));
    }
}

template <typename E>
__device__ __forceinline__ void put4(uint16_t* dst, const float (&v)[4], int64_t n, int64_t n_min, int64_t N) {
    const uint32_t lo = round2<E>(v[0], v[1]), hi = round2<E>(v[2], v[3]);
    typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
    if (n >= n_min && n + 4 <= N) {
        *reinterpret_cast<u32x2_any*>(dst) = u32x2{lo, hi};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i >= n_min && n + i < N) dst[i] = (uint16_t)((i < 2 ? lo : hi) >> (16 * (i % 2)));
    }
}

// fp32 staging of 32 rows of a wave tile: 16-byte chunk c of row r at slot c XOR r.
template <int CHUNKS>
__device__ __forceinline__ uint32_t stage_off(uint32_t row, uint32_t chunk) {
    return row * (CHUNKS * 16) + ((chunk ^ (row & (CHUNKS - 1))) << 4);
}

// Calls f(round, row in the round, c) for the 32-row rounds of a wave tile, with the
// lanes on groups of 8 columns c of OUT_COLS columns.
template <int OUT_COLS, typename Acc, typename F>
__device__ __forceinline__ void by_rows(Acc& acc, uint8_t* region, uint32_t lane, F f) {
    constexpr int FM = epi::AccTile<Acc>::FM, FN = epi::AccTile<Acc>::FN;
    constexpr int CHUNKS = 8 * FN;
    constexpr uint32_t LPR = OUT_COLS / 8;  // lanes per row
    constexpr uint32_t RPI = 64 / LPR;      // rows per iteration
#pragma unroll 1
    for (int i = 0; i < FM; ++i) {
        epi::stage_fp32_rows(acc, region, lane,
                             [](uint32_t row, uint32_t chunk) { return stage_off<CHUNKS>(row, chunk); });
#pragma unroll 1
        for (uint32_t k = 0; k < 32u / RPI; ++k) f(i, RPI * k + lane / LPR, lane % LPR);
    }
}

template <int CHUNKS>
__device__ __forceinline__ void staged8(const uint8_t* region, uint32_t row, uint32_t chunk, float (&v)[8]) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(region + stage_off<CHUNKS>(row, chunk));
    const f32x4 b = *reinterpret_cast<const f32x4*>(region + stage_off<CHUNKS>(row, chunk + 1));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}

// What the kernels ask of a type with an epilogue of its own, and most answer alike.
template <typename Base>
struct Own : Base {
    static constexpr bool kOwn = true;
    template <typename A>
    static __device__ __forceinline__ void tile(const A&, uint32_t tiles_m, uint32_t tiles_n, uint32_t group_m,
                                                uint32_t& tm, uint32_t& tn) {
        tile_of_workgroup(blockIdx.x, gridDim.x, tiles_m, tiles_n, group_m, tm, tn);
    }
    template <typename A>
    static __device__ __forceinline__ void batch(const A&, const uint16_t* __restrict__&, const uint16_t* __restrict__&,
                                                 uint16_t* __restrict__&) {}
};

// ---- Plain ------------------------------------------------------------------------

struct PlainArgs {};

template <typename Base>
struct Plain : Own<Base> {
    using Args = PlainArgs;

    template <bool EDGE, typename Acc>
    static __device__ __forceinline__ void store_tile(Acc& acc, uint8_t* region, uint32_t lane, uint16_t* C, int64_t ldc,
                                                      int64_t row0, int64_t col0, int64_t row_min, int64_t M, int64_t N,
                                                      const Args&) {
        constexpr int COLS = 32 * epi::AccTile<Acc>::FN;
        __syncthreads();
        by_rows<COLS>(acc, region, lane, [&](int i, uint32_t row, uint32_t c) {
            const int64_t m = row0 + 32 * i + row, n = col0 + 8 * c;
            if (EDGE && (m < row_min || m >= M)) return;
            float v[8];
            staged8<COLS / 4>(region, row, 2 * c, v);
            put8<EDGE>(C + m * ldc + n, round8<Base>(v), n, 0, N);
        });
    }

    template <int ROWS, int ON, int T, typename S, typename K, typename H>
    static __device__ __forceinline__ void store_block(S sum4, K, const H&, uint16_t* C, int64_t ldc, int64_t, int64_t M, int64_t N,
                                                       int64_t n0, int64_t n_own, const Args&) {
        for (uint32_t o = threadIdx.x; o < (uint32_t)(ROWS * ON / 4); o += T) {
            const uint32_t m = o / (ON / 4), c = 4 * (o % (ON / 4));
            if ((int64_t)m >= M) continue;
            const f32x4 s = sum4(m, c);
            const float v[4] = {s[0], s[1], s[2], s[3]};
            put4<Base>(C + (int64_t)m * ldc + n0 + c, v, n0 + c, n_own, N);
        }
    }
};

// ---- Two --------------------------------------------------------------------------

// One of two products in a launch, and the workgroups behind them for sums over rows: for
// small gradients, where a launch costs as much as a product.
struct Product {
    const uint16_t *A, *Bt;
    uint16_t* C;
    int64_t M, N, K, lda, ldb, ldc;
    uint32_t n_blocks, blocks;  // blocks (tiles) across the columns, and all of them
    uint32_t order;             // tile_of_workgroup's
    // K cut into `splits` ranges of k_per, whose fp32 sums go to part[split][m][n] for a second
    // pass (row-blocked stream only); part nullptr: whole
    uint32_t splits;
    int64_t k_per;
    float* part;
};
struct TwoArgs {
    Product product[2];
    // sums[r] = the sum of row r of sum_of (sum_k values, rows like a product's A), for r < sum_rows
    uint16_t* sums;
    const uint16_t* sum_of;
    int64_t sum_rows, sum_k;
};

// The sum of a row with a 16-byte start of `cols` (a multiple of 8) values over a wave, in
// fp32 and a fixed order.
template <typename E>
__device__ __forceinline__ float row_sum(const uint16_t* row, int64_t cols) {
    float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t c = 8 * (threadIdx.x % 64); c < cols; c += 512) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(row + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += widen8<E>(v, e);
    }
    return mx::wave_sum(((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7])));
}

template <typename Base>
struct Two : Own<Base> {
    static constexpr bool kTwo = true;
    using Args = TwoArgs;

    // Whether workgroup wg, of WAVES waves, is one for sums: then they are done.
    template <int WAVES>
    static __device__ __forceinline__ bool sums(const Args& ep, uint32_t wg) {
        const uint32_t products = ep.product[0].blocks * ep.product[0].splits + ep.product[1].blocks * ep.product[1].splits;
        if (wg < products) return false;
        const int64_t r = (int64_t)(wg - products) * WAVES + threadIdx.x / 64;
        if (r < ep.sum_rows) {
            const float s = row_sum<Base>(ep.sum_of + r * ep.sum_k, ep.sum_k);
            if (threadIdx.x % 64 == 0) ep.sums[r] = Base::round(s);
        }
        return true;
    }
    // Sets a workgroup's product and its number among that product's; returns where its sums go
    // (nullptr: rounded to C).
    static __device__ __forceinline__ float* select(const Args& ep, uint32_t& wg, uint32_t& n_wg, const uint16_t* __restrict__& A,
                                                  const uint16_t* __restrict__& B, uint16_t* __restrict__& C, int64_t& M,
                                                  int64_t& N, int64_t& K, int64_t& lda, int64_t& ldb, int64_t& ldc,
                                                  uint32_t& n_blocks, uint32_t& order) {
        const uint32_t first = ep.product[0].blocks * ep.product[0].splits;
        const bool second = wg >= first;
        if (second) wg -= first;
        const Product p = second ? ep.product[1] : ep.product[0];
        const uint32_t split = p.splits > 1 ? wg / p.blocks : 0;
        wg -= split * p.blocks;
        const int64_t k0 = split * p.k_per;
        A = p.A + k0;
        B = p.Bt + k0;
        C = p.C;
        M = p.M;
        N = p.N;
        K = p.K - k0 < p.k_per ? p.K - k0 : p.k_per;
        lda = p.lda;
        ldb = p.ldb;
        ldc = p.ldc;
        n_wg = p.blocks;
        n_blocks = p.n_blocks;
        order = p.order;
        return p.part != nullptr ? p.part + split * p.M * p.N : nullptr;
    }

    template <int N>
    struct Held : NothingHeld<N> {
        float* part;
    };

    template <bool EDGE, typename Acc>
    static __device__ __forceinline__ void store_tile(Acc& acc, uint8_t* region, uint32_t lane, uint16_t* C, int64_t ldc,
                                                      int64_t row0, int64_t col0, int64_t row_min, int64_t M, int64_t N,
                                                      const Args&) {
        Plain<Base>::template store_tile<EDGE>(acc, region, lane, C, ldc, row0, col0, row_min, M, N, PlainArgs{});
    }
    template <int ROWS, int ON, int T, typename S, typename K, typename H>
    static __device__ __forceinline__ void store_block(S sum4, K keep4, const H& held, uint16_t* C, int64_t ldc, int64_t row0,
                                                       int64_t M, int64_t N, int64_t n0, int64_t n_own, const Args&) {
        if (held.part == nullptr) {
            Plain<Base>::template store_block<ROWS, ON, T>(sum4, keep4, held, C, ldc, row0, M, N, n0, n_own, PlainArgs{});
            return;
        }
        typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
        for (uint32_t o = threadIdx.x; o < (uint32_t)(ROWS * ON / 4); o += T) {
            const uint32_t m = o / (ON / 4), c = 4 * (o % (ON / 4));
            if ((int64_t)m >= M) continue;
            const f32x4 s = sum4(m, c);
            float* const to = held.part + (row0 + m) * N + n0 + c;
            if (n0 + c >= n_own) {
                *reinterpret_cast<f32x4_any*>(to) = s;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n0 + c + e >= n_own) to[e] = s[e];
            }
        }
    }
};

// ---- Gated ------------------------------------------------------------------------

struct GatedArgs {
    const uint16_t* bias;  // 2 N values (those of the gates, then those of the ups), or nullptr
    uint16_t* kept;        // M x 2 N: g + b, then u + b', or nullptr
    int64_t ld_kept;
    int64_t half;          // rows of Bt from a gate's row to its up's
    int act;
};

template <typename Base>
struct Gated : Own<Base> {
    static constexpr bool kPairs = true;
    using Args = GatedArgs;

    // 4 or 8 consecutive columns from n of the bias, of the gates (at 0) or ups (at N).
    template <int C>
    static __device__ __forceinline__ void bias_of(const Args& ep, int64_t n, int64_t at, int64_t N, float (&b)[C]) {
#pragma unroll
        for (int i = 0; i < C; ++i) b[i] = ep.bias != nullptr && n + i < N ? Base::widen(ep.bias[at + n + i]) : 0.0f;
    }

    template <bool EDGE, typename Acc>
    static __device__ __forceinline__ void store_tile(Acc& acc, uint8_t* region, uint32_t lane, uint16_t* C, int64_t ldc,
                                                      int64_t row0, int64_t col0, int64_t row_min, int64_t M, int64_t N,
                                                      const Args& ep) {
        constexpr int COLS = 16 * epi::AccTile<Acc>::FN;  // of C
        constexpr int CHUNKS = COLS / 2;             // of the staged pairs: COLS gates, then COLS ups
        __syncthreads();
        float bg[8], bu[8];
        const int64_t n = col0 + 8 * (lane % (COLS / 8));
        bias_of(ep, n, 0, N, bg);
        bias_of(ep, n, N, N, bu);
        by_rows<COLS>(acc, region, lane, [&](int i, uint32_t row, uint32_t c) {
            const int64_t m = row0 + 32 * i + row;
            if (EDGE && (m < row_min || m >= M)) return;
            float g[8], u[8], h[8];
            staged8<CHUNKS>(region, row, 2 * c, g);
            staged8<CHUNKS>(region, row, CHUNKS / 2 + 2 * c, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                g[e] += bg[e];
                u[e] += bu[e];
            }
            act::dispatch(ep.act, [&](auto tag) {
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = act::apply<decltype(tag)::value>(g[e]) * u[e];
            });
            put8<EDGE>(C + m * ldc + n, round8<Base>(h), n, 0, N);
            if (ep.kept != nullptr) {
                uint16_t* const to = ep.kept + m * ep.ld_kept + n;
                put8<EDGE>(to, round8<Base>(g), n, 0, N);
                put8<EDGE>(to + N, round8<Base>(u), n, 0, N);
            }
        });
    }

    // Four columns of one row.
    static __device__ __forceinline__ void store4(const f32x4& gs, const f32x4& us, uint16_t* C, int64_t ldc, int64_t m,
                                                  int64_t n, int64_t N, const Args& ep, int64_t n_min = 0) {
        float g[4], u[4], h[4], bg[4], bu[4];
        bias_of(ep, n, 0, N, bg);
        bias_of(ep, n, N, N, bu);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            g[e] = gs[e] + bg[e];
            u[e] = us[e] + bu[e];
        }
        act::dispatch(ep.act, [&](auto tag) {
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = act::apply<decltype(tag)::value>(g[e]) * u[e];
        });
        put4<Base>(C + m * ldc + n, h, n, n_min, N);
        if (ep.kept != nullptr) {
            uint16_t* const to = ep.kept + m * ep.ld_kept + n;
            put4<Base>(to, g, n, n_min, N);
            put4<Base>(to + N, u, n, n_min, N);
        }
    }

    template <int ROWS, int ON, int T, typename S, typename K, typename H>
    static __device__ __forceinline__ void store_block(S sum4, K, const H&, uint16_t* C, int64_t ldc, int64_t row0, int64_t M,
                                                       int64_t N, int64_t n0, int64_t n_own, const Args& ep) {
        // C is at the block's first row already, what is kept is not
        Args at = ep;
        if (at.kept != nullptr) at.kept += row0 * at.ld_kept;
        for (uint32_t o = threadIdx.x; o < (uint32_t)(ROWS * ON / 4); o += T) {
            const uint32_t m = o / (ON / 4), c = 4 * (o % (ON / 4));
            if ((int64_t)m < M) store4(sum4(m, c), sum4(m, ON + c), C, ldc, m, n0 + c, N, at, n_own);
        }
    }
};

// ---- Poly -------------------------------------------------------------------------

struct PolyArgs {
    const uint16_t* d;  // beta's operand (pitch ldd), or nullptr
    uint16_t* ct;       // C transposed (pitch ldct), or nullptr
    int64_t ldd, ldct;
    float alpha, beta, diag;
    int64_t batch_a, batch_b, batch_c, batch_d, batch_ct;  // elements from one product of the batch to the next
};

// Tile (tm, tn) with tn <= tm of workgroup g of a triangle: g = tm (tm + 1) / 2 + tn.
__device__ __forceinline__ void tile_of_triangle(uint32_t g, uint32_t& tm, uint32_t& tn) {
    uint32_t r = (uint32_t)((__builtin_sqrtf(8.0f * (float)g + 1.0f) - 1.0f) * 0.5f);
    while (r * (r + 1) / 2 > g) --r;
    while ((r + 1) * (r + 2) / 2 <= g) ++r;
    tm = r;
    tn = g - r * (r + 1) / 2;
}

// Columns of the workgroup's tile: two waves side by side.
template <typename Acc>
constexpr int64_t TILE_COLS = 64 * epi::AccTile<Acc>::FN;

// In: the element type of the operands and of D; Out: that of C.  M, N: multiples of 32
// where C is written transposed.
template <typename In, typename Out, bool TRI>
struct Poly : Own<In> {
    using Args = PolyArgs;

    // D of a thread's groups of four columns: its latency passes beside the operands'.
    template <int N>
    struct Held {
        u32x2 d[N];
        __device__ __forceinline__ void fetch(const Args& ep, int on, int threads, int64_t row0, int64_t M, int64_t, int64_t n0) {
            const uint16_t* const src = ep.d != nullptr ? ep.d + blockIdx.y * ep.batch_d + row0 * ep.ldd + n0 : nullptr;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const uint32_t o = threadIdx.x + threads * k;
                const uint32_t m = o / (on / 4), c = 4 * (o % (on / 4));
                typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
                d[k] = u32x2{0u, 0u};
                if (src != nullptr && (int64_t)m < M) d[k] = *reinterpret_cast<const u32x2_any*>(src + (int64_t)m * ep.ldd + c);
            }
        }
    };

    static __device__ __forceinline__ void tile(const Args&, uint32_t tiles_m, uint32_t tiles_n, uint32_t group_m,
                                                uint32_t& tm, uint32_t& tn) {
        if constexpr (TRI) tile_of_triangle(blockIdx.x, tm, tn);
        else tile_of_workgroup(blockIdx.x, gridDim.x, tiles_m, tiles_n, group_m, tm, tn);
    }
    static __device__ __forceinline__ void batch(const Args& ep, const uint16_t* __restrict__& A,
                                                 const uint16_t* __restrict__& B, uint16_t* __restrict__& C) {
        A += blockIdx.y * ep.batch_a;
        B += blockIdx.y * ep.batch_b;
        C += blockIdx.y * ep.batch_c;
    }

    template <bool EDGE, typename Acc>
    static __device__ __forceinline__ void store_tile(Acc& acc, uint8_t* region, uint32_t lane, uint16_t* C, int64_t ldc,
                                                      int64_t row0, int64_t col0, int64_t row_min, int64_t M, int64_t N,
                                                      const Args& ep) {
        constexpr int COLS = 32 * epi::AccTile<Acc>::FN, CHUNKS = COLS / 4;
        constexpr uint32_t LPR = COLS / 8, RPI = 64 / LPR;
        const uint16_t* const d = ep.d != nullptr ? ep.d + blockIdx.y * ep.batch_d : nullptr;
        // (a tile on the diagonal holds its own transpose)
        const bool both = ep.ct != nullptr && !(TRI && row_min == col0 / TILE_COLS<Acc> * TILE_COLS<Acc>);
        uint16_t* const ct = both ? ep.ct + blockIdx.y * ep.batch_ct : nullptr;
        const uint32_t c = lane % LPR;
        const int64_t n = col0 + 8 * c;
        // D of 32 rows is fetched before the 32 rows in front of them are worked on: a load
        // where it is needed would cost every one of them its latency (4096 x 8192 x 4096:
        // 275 -> 239 us)
        constexpr int IT = 32 / RPI;
        u32x4 next[IT];
        auto fetch = [&](int i) {
#pragma unroll
            for (int k = 0; k < IT; ++k) {
                const int64_t m = row0 + 32 * i + RPI * k + lane / LPR;
                next[k] = u32x4{0u, 0u, 0u, 0u};
                if (EDGE && (m < row_min || m >= M || n >= N)) continue;
                const uint16_t* const src = d + m * ep.ldd + n;
                if (!EDGE || n + 8 <= N) {
                    next[k] = *reinterpret_cast<const u32x4_any*>(src);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (n + e < N) next[k][e / 2] |= (uint32_t)src[e] << (16 * (e % 2));
                }
            }
        };
        if (d != nullptr) fetch(0);
        __syncthreads();
#pragma unroll 1
        for (int i = 0; i < epi::AccTile<Acc>::FM; ++i) {
            epi::stage_fp32_rows(acc, region, lane,
                                 [](uint32_t row, uint32_t chunk) { return stage_off<CHUNKS>(row, chunk); });
            u32x4 now[IT];
#pragma unroll
            for (int k = 0; k < IT; ++k) now[k] = d != nullptr ? next[k] : u32x4{0u, 0u, 0u, 0u};
            if (d != nullptr && i + 1 < epi::AccTile<Acc>::FM) fetch(i + 1);
#pragma unroll
            for (int k = 0; k < IT; ++k) {
                const uint32_t row = RPI * k + lane / LPR;
                const int64_t m = row0 + 32 * i + row;
                float v[8];
                staged8<CHUNKS>(region, row, 2 * c, v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = __builtin_fmaf(ep.beta, widen8<In>(now[k], e),
                                          __builtin_fmaf(v[e], ep.alpha, m == n + e ? ep.diag : 0.0f));
                if (!EDGE || (m >= row_min && m < M)) put8<EDGE, false>(C + m * ldc + n, round8<Out>(v), n, 0, N);
                if (ct != nullptr) {
                    *reinterpret_cast<f32x4*>(region + stage_off<CHUNKS>(row, 2 * c)) = f32x4{v[0], v[1], v[2], v[3]};
                    *reinterpret_cast<f32x4*>(region + stage_off<CHUNKS>(row, 2 * c + 1)) = f32x4{v[4], v[5], v[6], v[7]};
                }
            }
            const int64_t mr = row0 + 32 * i;
            if (ct == nullptr || (EDGE && (mr < row_min || mr >= M))) continue;
            // columns of 8 rows each, four lanes to a column
#pragma unroll 1
            for (uint32_t k = 0; k < COLS / 16; ++k) {
                const uint32_t col = 16 * k + lane / 4, oct = lane % 4;
                float t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t[e] = *reinterpret_cast<const float*>(region + stage_off<CHUNKS>(8 * oct + e, col / 4) + 4 * (col % 4));
                if (!EDGE || col0 + col < N)
                    *reinterpret_cast<u32x4_any*>(ct + (col0 + col) * ep.ldct + mr + 8 * oct) = round8<Out>(t);
            }
        }
    }

    template <int ROWS, int ON, int T, typename S, typename K, typename H>
    static __device__ __forceinline__ void store_block(S sum4, K keep4, const H& held, uint16_t* C, int64_t ldc, int64_t row0, int64_t M,
                                                       int64_t N, int64_t n0, int64_t n_own, const Args& ep) {
        uint16_t* const ct = ep.ct != nullptr ? ep.ct + blockIdx.y * ep.batch_ct + row0 : nullptr;
#pragma unroll
        for (int k = 0; k < ROWS * ON / 4 / T; ++k) {
            const uint32_t o = threadIdx.x + T * k;
            const uint32_t m = o / (ON / 4), c = 4 * (o % (ON / 4));
            if ((int64_t)m >= M) continue;
            const f32x4 s = sum4(m, c);
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = __builtin_fmaf(ep.beta, In::widen((uint16_t)(held.d[k][e / 2] >> (16 * (e % 2)))),
                                      __builtin_fmaf(s[e], ep.alpha, row0 + m == n0 + c + e ? ep.diag : 0.0f));
            put4<Out>(C + (int64_t)m * ldc + n0 + c, v, n0 + c, n_own, N);
            if (ct != nullptr) *keep4(m, c) = f32x4{v[0], v[1], v[2], v[3]};
        }
        if (ct == nullptr) return;
        __syncthreads();
        // four rows of a column at a time
        for (uint32_t o = threadIdx.x; o < (uint32_t)(ROWS * ON / 4); o += T) {
            const uint32_t m = 4 * (o % (ROWS / 4)), c = o / (ROWS / 4);
            if ((int64_t)m >= M || n0 + c < n_own) continue;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = reinterpret_cast<const float*>(keep4(m + e, c & ~3u))[c & 3u];
            put4<Out>(ct + (n0 + c) * ep.ldct + m, v, m, 0, M);
        }
    }
};

}  // namespace own
}  // namespace gr
