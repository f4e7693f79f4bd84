// Around the products that make an update orthogonal: its Frobenius norm, and the
// fp16 operands X = update / (norm + eps) and X^T of the iteration
//
//   A = X X^T,  B = b A + c A A - (b + c) I,  X <- (a + b + c) X + B X
//
// which takes each singular value s of X to a s + b s^3 + c s^5 (five steps of the
// usual coefficients bring all but the smallest near 1).  The narrow side is X's rows,
// so that A and B are as small as they can be; both are symmetric.
//
// Operands are held in fp16 times a power of two, not in bfloat16, whose 8 bits would
// be seen in a bfloat16 result: every step rounds X, A and B once.  The multiple of I that
// is taken from B to X's factor is the polynomial's share at a singular value of 1: B's
// diagonal, and with it the rounding of what scales whole rows of X, is then small
// where the iteration ends (the result's error before its own rounding, 256 x 1024: 1.1e-3
// against 1.5e-3 with a X + (b A + c A A) X).  The elements
// are bounded by the singular values, and small by the matrix's size: X times
// 2^13 and A and B times 2^10 keep the elements of a random 8192 x 8192 matrix (1e-4 in X,
// 4e-6 in A) normal numbers.  Above, B's elements have to stay below 64 (with the usual
// coefficients: singular values below 2.6), and singular values below 8 for A, or below 4
// for the (A - I) X of the form with two launches.
//
// Rows and columns are padded by zeros to multiples of 64, which the iteration keeps:
// the products see whole strips whatever the matrix.
#pragma once

#include "norm_kernel.hpp"
#include "own_epilogue.hpp"
#include "transpose.hpp"

namespace gr {
namespace ortho {

constexpr float SCALE_X = 8192.0f, SCALE_A = 1024.0f;
constexpr int PARTS = 256;  // partial sums of the norm per matrix

struct ElemF32 {};

// 8 values of a row from column c, n of them there.
template <typename In>
__device__ __forceinline__ void load8(const void* row, int64_t c, int n, float (&v)[8]) {
    if constexpr (__is_same(In, ElemF32)) {
        typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
        const float* const p = static_cast<const float*>(row) + c;
        if (n >= 8) {
            const f32x4 a = *reinterpret_cast<const f32x4_any*>(p), b = *reinterpret_cast<const f32x4_any*>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
        }
    } else {
        const u32x4 w = n > 0 ? mx::load8(static_cast<const uint16_t*>(row) + c, n) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = own::widen8<In>(w, i);
    }
}
template <typename In>
constexpr int kBytes = __is_same(In, ElemF32) ? 4 : 2;

// What a value is multiplied by to become one of X: SCALE_X / (norm + eps), as a factor of about
// 1 and a power of two, since fp32 does not hold it where the norm is below 2.4e-35.  A zero
// matrix without an eps stays zero.
struct Factor {
    float f;
    int e;
    __device__ __forceinline__ Factor(double squares, float eps) : f(0.0f), e(0) {
        const double norm = __builtin_sqrt(squares) + (double)eps;
        if (norm != 0.0) f = (float)frexp((double)SCALE_X / norm, &e);
    }
    __device__ __forceinline__ float operator()(float v) const { return ldexpf(v, e) * f; }
};

struct PrepArgs {
    const void* src;
    int64_t rows, cols, ld, batch;  // of the update, batch: elements from one matrix to the next
    double* part;                   // PARTS per matrix
    uint16_t *x, *xt;               // like the update, and transposed: zeros up to rows_pad, cols_pad; one
                                    // may be nullptr
    int64_t rows_pad, cols_pad, batch_x;
    float eps;
};

// part[p] = the sum of squares of every PARTS-th group of 256 chunks.  In fp64: the
// squares of any fp32 value have their place.
template <typename In>
__global__ void __launch_bounds__(256) square_sum_kernel(PrepArgs a) {
    __shared__ double red[4];
    const uint8_t* const src = static_cast<const uint8_t*>(a.src) + blockIdx.y * a.batch * kBytes<In>;
    const int64_t per_row = (a.cols + 7) / 8, chunks = a.rows * per_row;
    double sum = 0.0;
    for (int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x; o < chunks; o += PARTS * 256) {
        const int64_t r = o / per_row, c = 8 * (o - r * per_row);
        float v[8];
        load8<In>(src + r * a.ld * kBytes<In>, c, a.cols - c < 8 ? (int)(a.cols - c) : 8, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)v[i], (double)v[i], sum);
    }
#pragma unroll
    for (int s = 1; s < 64; s *= 2) sum += __shfl_xor(sum, s);
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = sum;
    __syncthreads();
    if (threadIdx.x == 0) a.part[blockIdx.y * PARTS + blockIdx.x] = ((red[0] + red[1]) + red[2]) + red[3];
}

// A tile of 64 x 64 of X and of X^T.
template <typename In>
__global__ void __launch_bounds__(256) normalise_kernel(PrepArgs a, uint32_t tiles_c) {
    using train::TILE;
    __shared__ __attribute__((aligned(16))) uint8_t lds[TILE * TILE * 2];
    __shared__ double red[4];
    const uint8_t* const src = static_cast<const uint8_t*>(a.src) + blockIdx.y * a.batch * kBytes<In>;
    const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * TILE, c0 = (int64_t)(blockIdx.x % tiles_c) * TILE;
    float v[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t o = threadIdx.x + 256 * i;
        const int64_t r = r0 + o / 8, c = c0 + 8 * (o % 8), left = a.cols - c;
        const int n = r < a.rows && left > 0 ? (left < 8 ? (int)left : 8) : 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
        if (n > 0) load8<In>(src + r * a.ld * kBytes<In>, c, n, v[i]);
    }
    double sum = a.part[blockIdx.y * PARTS + threadIdx.x];
    static_assert(PARTS == 256, "a partial sum per thread");
#pragma unroll
    for (int s = 1; s < 64; s *= 2) sum += __shfl_xor(sum, s);
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = sum;
    __syncthreads();
    sum = ((red[0] + red[1]) + red[2]) + red[3];
    const Factor scaled(sum, a.eps);
    uint16_t* const x = a.x + blockIdx.y * a.batch_x;  // (not used where there is none)
    uint16_t* const xt = a.xt + blockIdx.y * a.batch_x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t o = threadIdx.x + 256 * i;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = scaled(v[i][e]);
        const u32x4 w = own::round8<ElemF16>(v[i]);
        if (a.x != nullptr) *reinterpret_cast<u32x4*>(x + (r0 + o / 8) * a.cols_pad + c0 + 8 * (o % 8)) = w;
        *reinterpret_cast<u32x4*>(lds + train::tile_off(o / 8, o % 8)) = w;
    }
    if (a.xt == nullptr) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t o = threadIdx.x + 256 * i;
        *reinterpret_cast<u32x4*>(xt + (c0 + o / 8) * a.rows_pad + r0 + 8 * (o % 8)) = train::column8(lds, o / 8, o % 8);
    }
}

}  // namespace ortho
}  // namespace gr
