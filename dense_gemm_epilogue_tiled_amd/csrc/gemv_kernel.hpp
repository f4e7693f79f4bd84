// The gated linear layer for up to four tokens: a wave takes two columns of the result, that
// is two gate rows and two up rows of the weight, and reads them from end to end, 16 bytes per
// lane and four pieces of each row in flight; x comes from the caches.
//
// Bound by the weight's way from memory.  With so few tokens a matrix instruction's rows stay
// empty and the multiply-adds of ordinary lanes are few (a sixth of their rate at four
// tokens), so that nothing asks for the weight in pieces of 16 rows: 1 x 4096 x 14336
// (235 MB of weights) 43.5 us with the matrix instructions' stream, 37.2 here (6.3 TB/s; a
// plain read reaches 6.5).  Any K and any address: a ragged end is loaded element by element.
#pragma once

#include "norm_kernel.hpp"
#include "own_epilogue.hpp"

namespace gr {
namespace gemv {

constexpr int WAVES = 4, THREADS = 64 * WAVES;
constexpr int COLS = 2;    // columns of the result per wave

struct Args {
    const uint16_t *x, *w;
    uint16_t* c;
    int64_t M, I, K, ldx, ldw, ldc;
    own::GatedArgs ep;
};

// MT: tokens, of which the last stands for missing ones.
template <typename E, int MT>
__device__ __forceinline__ void columns(const Args& a, int64_t n0, int lane) {
    constexpr int ROWS = 2 * COLS;
    constexpr int UNROLL = MT == 4 ? 2 : 4;  // pieces of 512 values of each row in flight
    const uint16_t* row[ROWS];  // gate rows, then up rows
#pragma unroll
    for (int j = 0; j < COLS; ++j) {
        const int64_t n = n0 + j < a.I ? n0 + j : a.I - 1;
        row[j] = a.w + n * a.ldw;
        row[COLS + j] = row[j] + a.ep.half * a.ldw;
    }
    const uint16_t* x[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) x[m] = a.x + (m < a.M ? m : a.M - 1) * a.ldx;
    float sum[ROWS][MT];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) sum[r][m] = 0.0f;
    auto add = [&](const u32x4 (&w)[ROWS], const u32x4 (&v)[MT]) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const float xv = own::widen8<E>(v[m], e);
#pragma unroll
                for (int r = 0; r < ROWS; ++r) sum[r][m] = __builtin_fmaf(own::widen8<E>(w[r], e), xv, sum[r][m]);
            }
    };
    int64_t k = 8 * lane;
    for (; k - 8 * lane + 512 * UNROLL <= a.K; k += 512 * UNROLL) {
        u32x4 w[UNROLL][ROWS], v[UNROLL][MT];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                w[i][r] = __builtin_nontemporal_load(reinterpret_cast<const own::u32x4_any*>(row[r] + k + 512 * i));
#pragma unroll
            for (int m = 0; m < MT; ++m) v[i][m] = *reinterpret_cast<const own::u32x4_any*>(x[m] + k + 512 * i);
        }
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) add(w[i], v[i]);
    }
    for (; k < a.K; k += 512) {
        const int n = a.K - k < 8 ? (int)(a.K - k) : 8;
        u32x4 w[ROWS], v[MT];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) w[r] = mx::load8(row[r] + k, n);
#pragma unroll
        for (int m = 0; m < MT; ++m) v[m] = mx::load8(x[m] + k, n);
        add(w, v);
    }
    // lane 4 j + m stores column j of token m
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int j = 0; j < COLS; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float sg = mx::wave_sum(sum[j][m]), su = mx::wave_sum(sum[COLS + j][m]);
            g = lane == 4 * j + m ? sg : g;
            u = lane == 4 * j + m ? su : u;
        }
    const int64_t n = n0 + lane / 4, m = lane % 4;
    if (lane >= 4 * COLS || n >= a.I || m >= a.M || m >= MT) return;
    if (a.ep.bias != nullptr) {
        g += E::widen(a.ep.bias[n]);
        u += E::widen(a.ep.bias[a.I + n]);
    }
    const float h = activate(g, a.ep.act) * u;
    a.c[m * a.ldc + n] = (uint16_t)own::round2<E>(h, h);
    if (a.ep.kept != nullptr) {
        a.ep.kept[m * a.ep.ld_kept + n] = (uint16_t)own::round2<E>(g, g);
        a.ep.kept[m * a.ep.ld_kept + a.I + n] = (uint16_t)own::round2<E>(u, u);
    }
}

template <typename E, int MT>
__global__ void __launch_bounds__(THREADS) gated_gemv_kernel(Args a) {
    const int64_t step = (int64_t)gridDim.x * WAVES * COLS;
    for (int64_t n0 = ((int64_t)blockIdx.x * WAVES + threadIdx.x / 64) * COLS; n0 < a.I; n0 += step)
        columns<E, MT>(a, n0, threadIdx.x % 64);
}

}  // namespace gemv
}  // namespace gr
