// What the products of training have around them: operands copied with their rows
// transposed or padded, the gated activation's backward pass, sums over rows.
//
// The gradient of a weight, dW = dY^T X, sums over tokens, along which neither
// operand is contiguous.  Both are written transposed once (2 bytes read and
// written per element, nothing next to the product's 2 M operations per element), with
// the tokens padded by zeros to whole strips of 64, and the product is then the one of two
// k-contiguous operands.  All of these kernels are bound by memory: every element is
// read once and written once, in 16-byte pieces.
#pragma once

#include "norm_kernel.hpp"
#include "own_epilogue.hpp"
#include "transpose.hpp"

namespace gr {
namespace train {

constexpr int PAD = 64;  // tokens of a transposed operand: whole strips of this

// dst[c][r] = src[r][c] (transposed) or dst[r][c] = src[r][c], 0 outside src's rows x
// cols.  dst has 16-byte rows; it gets `pad` columns, a multiple of 8.
struct Job {
    const uint16_t* src;
    uint16_t* dst;
    int64_t rows, cols, lds, ldd;
    int64_t pad;
    uint32_t tiles_c;  // tiles across the columns
    uint32_t tiles;    // all of them; 0: nothing to do
    int transposed;
};

// Several jobs in one launch: a workgroup per tile, the first job's first.
constexpr int JOBS = 4;
struct Jobs {
    Job job[JOBS];
};

// The job of a workgroup, field by field: an array indexed by a variable would go through scratch
// memory.
__device__ __forceinline__ Job job_of(const Jobs jobs, uint32_t& tile) {
    Job j = jobs.job[0];
#pragma unroll
    for (int i = 1; i < JOBS; ++i) {
        const bool next = tile >= j.tiles;
        const Job& n = jobs.job[i];
        tile -= next ? j.tiles : 0;
        j.src = next ? n.src : j.src;
        j.dst = next ? n.dst : j.dst;
        j.rows = next ? n.rows : j.rows;
        j.cols = next ? n.cols : j.cols;
        j.lds = next ? n.lds : j.lds;
        j.ldd = next ? n.ldd : j.ldd;
        j.pad = next ? n.pad : j.pad;
        j.tiles_c = next ? n.tiles_c : j.tiles_c;
        j.transposed = next ? n.transposed : j.transposed;
        j.tiles = next ? n.tiles : j.tiles;
    }
    return j;
}

__device__ __forceinline__ void relayout(const Job j, uint32_t tile, uint8_t* lds) {
    const int64_t r0 = (int64_t)(tile / j.tiles_c) * TILE, c0 = (int64_t)(tile % j.tiles_c) * TILE;
    u32x4 v[2];
    uint32_t row[2], chunk[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t o = threadIdx.x + THREADS * i;
        row[i] = o / 8;
        chunk[i] = o % 8;
        const int64_t r = r0 + row[i], c = c0 + 8 * chunk[i];
        const int64_t left = j.cols - c;
        const int n = r < j.rows && left > 0 ? (left < 8 ? (int)left : 8) : 0;
        v[i] = n > 0 ? mx::load8(j.src + r * j.lds + c, n, j.cols >= 8) : u32x4{0u, 0u, 0u, 0u};
    }
    if (!j.transposed) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (r0 + row[i] < j.rows && c0 + 8 * chunk[i] < j.pad)
                *reinterpret_cast<u32x4*>(j.dst + (r0 + row[i]) * j.ldd + c0 + 8 * chunk[i]) = v[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<u32x4*>(lds + tile_off(row[i], chunk[i])) = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t o = threadIdx.x + THREADS * i;
        const uint32_t c = o / 8, oct = o % 8;
        if (c0 + c < j.cols && r0 + 8 * oct < j.pad)
            *reinterpret_cast<u32x4*>(j.dst + (c0 + c) * j.ldd + r0 + 8 * oct) = column8(lds, c, oct);
    }
}

__global__ void __launch_bounds__(THREADS) relayout_kernel(Jobs jobs) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[TILE * TILE * 2];
    uint32_t tile = blockIdx.x;
    const Job j = job_of(jobs, tile);
    relayout(j, tile, lds);
}

// ---- the gated activation's backward pass -----------------------------------------------

// An activation's value and derivative at a finite x.  Sigmoid's complement is taken as the
// sigmoid of -x, so that neither side of 0 cancels.
template <int A>
__device__ __forceinline__ void value_and_slope_within(float x, float& a, float& d) {
    if constexpr (A == kActRelu) {
        a = x > 0.0f ? x : 0.0f;
        d = x > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (A == kActGelu) {
        const float phi = 0.5f * erfcf(-0.70710678118654752f * x);
        a = x * phi;
        d = __builtin_fmaf(x, 0.39894228040143268f * act::ex(-0.5f * x * x), phi);
    } else if constexpr (A == kActGeluTanh) {
        const float x2 = __builtin_fminf(x * x, 1e30f);  // no infinity times the 0 that is left of the exponential
        const float z = 1.5957691216057308f * (x * __builtin_fmaf(0.044715f, x2, 1.0f));
        const float s = act::rcp(1.0f + act::ex(-z)), o = act::rcp(1.0f + act::ex(z));
        a = x * s;
        d = __builtin_fmaf(a, o * 1.5957691216057308f * __builtin_fmaf(3.0f * 0.044715f, x2, 1.0f), s);
    } else if constexpr (A == kActSilu) {
        const float s = act::rcp(1.0f + act::ex(-x)), o = act::rcp(1.0f + act::ex(x));
        a = x * s;
        d = __builtin_fmaf(a, o, s);
    } else if constexpr (A == kActSigmoid) {
        a = act::rcp(1.0f + act::ex(-x));
        d = a * act::rcp(1.0f + act::ex(x));
    } else if constexpr (A == kActTanh) {
        a = act::apply<kActTanh>(x);
        // 1 - tanh^2 = 4 e / (1 + e)^2 with e = exp(-2 |x|)
        const float e = act::ex(-2.0f * __builtin_fabsf(x)), r = act::rcp(1.0f + e);
        d = 4.0f * e * r * r;
    } else {
        a = x;
        d = 1.0f;
    }
}

// The same at any x, with the limits at an infinity (not 0 times infinity): a gate beyond the
// type's range is kept as one, where the forward pass had a finite sum.
template <int A>
__device__ __forceinline__ void value_and_slope(float x, float& a, float& d) {
    if constexpr (A == kActGelu || A == kActGeluTanh || A == kActSilu) {
        value_and_slope_within<A>(__builtin_isinf(x) ? __builtin_copysignf(__FLT_MAX__, x) : x, a, d);
        if (x == __builtin_inff()) a = x;
    } else {
        value_and_slope_within<A>(x, a, d);
    }
}

struct GatedBwdArgs {
    const uint16_t* dh;  // M x I
    const uint16_t* gu;  // M x 2 I: gates, then ups
    uint16_t* dgu;       // M x 2 I, zeros from there to the pitch
    uint16_t* dgu_t;     // 2 I x Mp, zeros for the tokens from M on; nullptr: not wanted
    int64_t M, I, ld_dh, ld_gu, ld_dgu, ld_t;
    int act;
};

// dg = dh u act'(g), du = dh act(g) of a tile of 64 tokens x 64 columns, written
// as they are and transposed.  The workgroups behind the tiles do `jobs`.
template <typename E>
__global__ void __launch_bounds__(THREADS) gated_backward_kernel(GatedBwdArgs a, uint32_t tiles_c, uint32_t tiles, Jobs jobs) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][TILE * TILE * 2];
    if (blockIdx.x >= tiles) {
        uint32_t tile = blockIdx.x - tiles;
        const Job j = job_of(jobs, tile);
        relayout(j, tile, lds[0]);
        return;
    }
    const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * TILE, c0 = (int64_t)(blockIdx.x % tiles_c) * TILE;
    u32x4 dh[2], g[2], u[2];
    int n[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t o = threadIdx.x + THREADS * i;
        const int64_t r = r0 + o / 8, c = c0 + 8 * (o % 8);
        const int64_t left = a.I - c;
        n[i] = r < a.M && left > 0 ? (left < 8 ? (int)left : 8) : 0;
        dh[i] = g[i] = u[i] = u32x4{0u, 0u, 0u, 0u};
        if (n[i] > 0) {
            dh[i] = mx::load8(a.dh + r * a.ld_dh + c, n[i], a.I >= 8);
            g[i] = mx::load8(a.gu + r * a.ld_gu + c, n[i], a.I >= 8);
            u[i] = mx::load8(a.gu + r * a.ld_gu + a.I + c, n[i], a.I >= 8);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t o = threadIdx.x + THREADS * i;
        u32x4 dg = u32x4{0u, 0u, 0u, 0u}, du = dg;
        if (n[i] > 0) {
            float vg[8], vu[8];
            act::dispatch(a.act, [&](auto tag) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float v, s;
                    value_and_slope<decltype(tag)::value>(own::widen8<E>(g[i], e), v, s);
                    const float d = own::widen8<E>(dh[i], e);
                    vg[e] = d * own::widen8<E>(u[i], e) * s;
                    vu[e] = d * v;
                }
            });
            dg = own::round8<E>(vg);
            du = own::round8<E>(vu);
            uint16_t* const to = a.dgu + (r0 + o / 8) * a.ld_dgu + c0 + 8 * (o % 8);
            own::put8<true, false>(to, dg, 0, 0, n[i]);
            own::put8<true, false>(to + a.I, du, 0, 0, n[i]);
        }
        *reinterpret_cast<u32x4*>(lds[0] + tile_off(o / 8, o % 8)) = dg;
        *reinterpret_cast<u32x4*>(lds[1] + tile_off(o / 8, o % 8)) = du;
    }
    if (c0 + TILE >= a.I) {
        const int64_t r = r0 + threadIdx.x / 4;
        if (r < a.M)
            for (int64_t c = 2 * a.I + threadIdx.x % 4; c < a.ld_dgu; c += 4) a.dgu[r * a.ld_dgu + c] = 0;
    }
    if (a.dgu_t == nullptr) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t o = threadIdx.x + THREADS * i;
        const uint32_t half = o / (TILE * 8), c = o / 8 % TILE, oct = o % 8;
        if (c0 + c < a.I)
            *reinterpret_cast<u32x4*>(a.dgu_t + (half * a.I + c0 + c) * a.ld_t + r0 + 8 * oct) = column8(lds[half], c, oct);
    }
}

// out[r] = the sum of row r of a matrix with 16-byte rows of `cols` (a multiple of 8)
// values: a bias's gradient from the transposed gradient.  A wave per row.
template <typename E>
__global__ void __launch_bounds__(THREADS) row_sums_kernel(const uint16_t* src, int64_t rows, int64_t cols, int64_t ld,
                                                           uint16_t* out) {
    for (int64_t r = (int64_t)blockIdx.x * (THREADS / 64) + threadIdx.x / 64; r < rows; r += (int64_t)gridDim.x * (THREADS / 64)) {
        const float s = own::row_sum<E>(src + r * ld, cols);
        if (threadIdx.x % 64 == 0) out[r] = E::round(s);
    }
}

// C[m][n] = round(the sum over the splits, in order, of part[split][m][n]): the second pass of a
// weight's gradient whose tokens were cut into ranges.  Four columns per thread where N allows.
template <typename E, int VEC>
__global__ void __launch_bounds__(THREADS) sum_splits_kernel(const float* part, int64_t splits, int64_t M, int64_t N, uint16_t* C,
                                                             int64_t ldc) {
    const int64_t total = M * N, step = (int64_t)gridDim.x * THREADS * VEC;
    for (int64_t o = ((int64_t)blockIdx.x * THREADS + threadIdx.x) * VEC; o < total; o += step) {
        float sum[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum[e] = 0.0f;
#pragma unroll 4
        for (int64_t s = 0; s < splits; ++s) {
            if constexpr (VEC == 4) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(part + s * total + o);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += v[e];
            } else {
                sum[0] += part[s * total + o];
            }
        }
        const int64_t m = o / N, n = o - m * N;
        if constexpr (VEC == 4) own::put4<E>(C + m * ldc + n, sum, n, 0, N);
        else C[m * ldc + n] = E::round(sum[0]);
    }
}

}  // namespace train
}  // namespace gr
