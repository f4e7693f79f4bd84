// The whole orthogonalisation of a small matrix in one workgroup: X (r x c, fp16) and A (r x
// r) stay in its LDS for all steps, where a step is otherwise two launches of a few
// microseconds each.  r and c are padded by zeros to multiples of 64, r to 64 or 128, and 2 r (c + r)
// bytes have to fit 160 KiB: the border is what fits.  Five steps in us, bfloat16, replayed in a
// graph, as two launches a step and here:
//
//                64 x 64     64 x 640    128 x 128   128 x 256   128 x 512
//   1 matrix     33   15     41   41     49   31     44   41     48   67
//   8                        45   42                 48   41     55   68
//   300          105  28                             196  82     295  147
//
// (1000 of 128 x 512: 757 and 309.)  So one workgroup a matrix is the faster form but for a few
// matrices of the longest, whose columns one CU works off alone.
//
//   A = X X^T       32 x 32 tiles on and below the diagonal, a wave each; both operands are
//                   rows of X, which the matrix instruction wants as they lie; a tile
//                   below the diagonal is written a second time transposed
//   B = b A + c A A - (b + c) I    32 x 32 tiles, a wave each, held in registers until all
//                   waves have read A, then written over it
//   X <- (a + b + c) X + B X       columns of X by 16 or 32, which one wave reads whole
//                   (transposing reads) before it writes them over
//
// Scales and roundings are those of the products' path.  What bounds it is LDS: B is read once for each group of columns.
#pragma once

#include "ortho_kernel.hpp"

namespace gr {
namespace ortho {

constexpr int SMALL_LDS = 160 * 1024;
constexpr int SMALL_WAVES = 16;
constexpr int SMALL_THREADS = 64 * SMALL_WAVES;
constexpr int SMALL_R = 128;  // widest narrow side
static_assert((SMALL_R / 32) * (SMALL_R / 32) <= SMALL_WAVES, "a tile of B per wave");

struct SmallArgs {
    const void* src;
    uint16_t* out;
    int64_t rows, cols, ld, batch, ldo, batch_o;  // batch: elements from one matrix to the next
    uint32_t cp;                                  // padded wide side
    int tall, steps;
    float k1, k2, all, scale, eps;                // b, c, a + b + c
};

#define GR_LDS __attribute__((address_space(3)))

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Where the 16-byte chunks of a matrix with rows of `pitch` values lie, a multiple of 64: those
// of 16 rows at one chunk cover all 64 banks, with rows that begin at the same bank (an even
// multiple) as with rows that begin at two by turns.
struct Place {
    uint32_t pitch, shift, mask;
    __device__ __forceinline__ explicit Place(uint32_t p) : pitch(p), shift(p / 64 % 2), mask(p / 64 % 2 ? 7u : 15u) {}
    __device__ __forceinline__ uint32_t chunk(uint32_t row, uint32_t c) const {
        return row * pitch * 2 + ((c ^ ((row >> shift) & mask)) << 4);
    }
    // Value `col` of row `row`; 4 values from a multiple of 4 on are consecutive.
    __device__ __forceinline__ uint32_t value(uint32_t row, uint32_t col) const { return chunk(row, col >> 3) + 2 * (col & 7u); }
};

__device__ __forceinline__ f16x8 rows_of(const GR_LDS uint8_t* m, const Place& p, uint32_t row, uint32_t chunk) {
    return *(const GR_LDS f16x8*)(m + p.chunk(row, chunk));
}

// The lane's index, as if new: addresses made from it are computed where they are used, not
// kept (and spilled) over the steps.
__device__ __forceinline__ uint32_t fresh(uint32_t lane) {
    asm volatile("" : "+v"(lane));
    return lane;
}

__device__ __forceinline__ u32x2 round4(const float (&v)[4]) {
    return u32x2{own::round2<ElemF16>(v[0], v[1]), own::round2<ElemF16>(v[2], v[3])};
}

// acc[i][j] += rows r0 + 16 i of m times rows c0 + 16 j of m, over k values.
__device__ __forceinline__ void row_products(const GR_LDS uint8_t* m, const Place& p, uint32_t r0, uint32_t c0, uint32_t k,
                                             uint32_t lane, f32x4 (&acc)[2][2]) {
    const uint32_t li = lane & 15u, lg = lane >> 4;
#pragma unroll 4
    for (uint32_t s = 0; s < k / 32; ++s) {
        f16x8 a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            a[i] = rows_of(m, p, r0 + 16 * i + li, 4 * s + lg);
            b[i] = rows_of(m, p, c0 + 16 * i + li, 4 * s + lg);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = ElemF16::mfma16(b[j], a[i], acc[i][j]);
    }
}

// X <- all X + B X for P groups of 16 columns from c0: read() takes them, update() the rows
// [16 first, 16 end) of the result; `out` gets the last step's.
template <int RP, int P>
struct ColumnGroups {
    f16x8 f[P][RP / 32];

    __device__ __forceinline__ void read(GR_LDS uint8_t* x, const Place& xp, uint32_t c0, uint32_t lane) {
        const uint32_t li = lane & 15u, lg = lane >> 4;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (uint32_t s = 0; s < RP / 32; ++s) {
                const uint32_t row = 32 * s + 8 * lg + (li >> 2), col = c0 + 16 * p + 4 * (li & 3u);
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((GR_LDS s16x4*)(x + xp.value(row, col)));
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((GR_LDS s16x4*)(x + xp.value(row + 4, col)));
                f[p][s] = __builtin_bit_cast(f16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
    }
    template <typename Out>
    __device__ __forceinline__ void update(GR_LDS uint8_t* x, const Place& xp, const GR_LDS uint8_t* b, uint32_t c0,
                                           uint32_t first, uint32_t end, uint32_t lane, float all, Out out) const {
        const uint32_t li = lane & 15u, lg = lane >> 4;
        const Place bp(RP);
#pragma unroll 2
        for (uint32_t i = first; i < end; ++i) {
            f32x4 acc[P];
#pragma unroll
            for (int p = 0; p < P; ++p) acc[p] = f32x4{};
#pragma unroll
            for (uint32_t s = 0; s < RP / 32; ++s) {
                const f16x8 a = rows_of(b, bp, 16 * i + li, 4 * s + lg);
#pragma unroll
                for (int p = 0; p < P; ++p) acc[p] = ElemF16::mfma16(f[p][s], a, acc[p]);
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const uint32_t row = 16 * i + li, col = c0 + 16 * p + 4 * lg;
                GR_LDS u32x2* const at = (GR_LDS u32x2*)(x + xp.value(row, col));
                const u32x2 old = *at;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = __builtin_fmaf(all, ElemF16::widen((uint16_t)(old[e / 2] >> (16 * (e % 2)))), acc[p][e] * (1.0f / SCALE_A));
                if (!out(row, col, v)) *at = round4(v);
            }
        }
    }
};

template <typename In, int RP>
__global__ void __launch_bounds__(SMALL_THREADS) small_kernel(SmallArgs a) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[SMALL_LDS];
    const uint32_t tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr uint32_t rp = RP, t = RP / 32;
    const uint32_t cp = a.cp;
    const Place xp(cp), mp(rp);
    GR_LDS uint8_t* const x = (GR_LDS uint8_t*)lds;
    GR_LDS uint8_t* const m = x + 2 * rp * cp;  // A, then B
    const uint8_t* const src = static_cast<const uint8_t*>(a.src) + blockIdx.x * a.batch * kBytes<In>;

    // The norm, then X = the matrix (or its transpose) times SCALE_X / (norm + eps).
    const uint32_t per_row = (uint32_t)((a.cols + 7) / 8), chunks = (uint32_t)a.rows * per_row;
    // f(row, column, columns, values) of every chunk of 8 columns, four loads in flight
    auto each = [&](auto f) {
        for (uint32_t o0 = tid; o0 < chunks; o0 += 4 * SMALL_THREADS) {
            float v[4][8];
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                const uint32_t o = o0 + i * SMALL_THREADS, r = o / per_row, c = 8 * (o - r * per_row);
                if (o < chunks)
                    load8<In>(src + r * a.ld * kBytes<In>, c, a.cols - c < 8 ? (int)(a.cols - c) : 8, v[i]);
            }
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                const uint32_t o = o0 + i * SMALL_THREADS, r = o / per_row, c = 8 * (o - r * per_row);
                if (o < chunks) f(r, c, a.cols - c < 8 ? (int)(a.cols - c) : 8, v[i]);
            }
        }
    };
    double sum = 0.0;
    each([&](uint32_t, uint32_t, int, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)v[i], (double)v[i], sum);
    });
#pragma unroll
    for (int s = 1; s < 64; s *= 2) sum += __shfl_xor(sum, s);
    GR_LDS double* const red = (GR_LDS double*)m;
    if (tid % 64 == 0) red[wave] = sum;
    for (uint32_t o = tid; o < rp * cp / 8; o += SMALL_THREADS) *(GR_LDS u32x4*)(x + 16 * o) = u32x4{0u, 0u, 0u, 0u};
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < SMALL_WAVES; ++i) sum += red[i];
    const Factor scaled(sum, a.eps);
    each([&](uint32_t r, uint32_t c, int n, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = scaled(v[i]);
        const u32x4 w = own::round8<ElemF16>(v);  // zeros behind the row's end
        if (!a.tall) {
            *(GR_LDS u32x4*)(x + xp.chunk(r, c >> 3)) = w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) *(GR_LDS uint16_t*)(x + xp.value(c + i, r)) = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
        }
    });
    __syncthreads();

    uint32_t tr, tc;
    own::tile_of_triangle(wave, tr, tc);
    tr = __builtin_amdgcn_readfirstlane(tr);
    tc = __builtin_amdgcn_readfirstlane(tc);
    static_assert(t * (t + 1) / 2 <= SMALL_WAVES, "a tile of A per wave");
#pragma unroll 1
    for (int step = 0; step < a.steps; ++step) {
        if (tr < t) {
            const uint32_t lane = fresh(tid & 63u), li = lane & 15u, lg = lane >> 4;
            f32x4 acc[2][2] = {};
            row_products(x, xp, 32 * tr, 32 * tc, cp, lane, acc);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t row = 32 * tr + 16 * i + li, col = 32 * tc + 16 * j + 4 * lg;
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e] * (SCALE_A / (SCALE_X * SCALE_X));
                    const u32x2 w = round4(v);
                    *(GR_LDS u32x2*)(m + mp.value(row, col)) = w;
                    if (tr != tc) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *(GR_LDS uint16_t*)(m + mp.value(col + e, row)) = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
                    }
                }
        }
        __syncthreads();
        u32x2 held[2][2];
        const uint32_t r0 = 32 * (wave / t), c0 = 32 * (wave % t);
        const uint32_t lane = fresh(tid & 63u), li = lane & 15u, lg = lane >> 4;
        if (wave < t * t) {
            f32x4 acc[2][2] = {};
            row_products(m, mp, r0, c0, rp, lane, acc);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t row = r0 + 16 * i + li, col = c0 + 16 * j + 4 * lg;
                    const u32x2 w = *(const GR_LDS u32x2*)(m + mp.value(row, col));
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float d = row == col + e ? -SCALE_A * (a.k1 + a.k2) : 0.0f;
                        v[e] = __builtin_fmaf(a.k1, ElemF16::widen((uint16_t)(w[e / 2] >> (16 * (e % 2)))),
                                              __builtin_fmaf(acc[i][j][e], a.k2 / SCALE_A, d));
                    }
                    held[i][j] = round4(v);
                }
        }
        __syncthreads();
        if (wave < t * t) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    *(GR_LDS u32x2*)(m + mp.value(r0 + 16 * i + li, c0 + 16 * j + 4 * lg)) = held[i][j];
        }
        __syncthreads();
        const bool last = step + 1 == a.steps;
        uint16_t* const to = a.out + blockIdx.x * a.batch_o;
        auto out = [&](uint32_t row, uint32_t col, const float (&v)[4]) {
            if (!last) return false;
            float s[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = v[e] * (a.scale / SCALE_X);
            if (!a.tall) {
                if ((int64_t)row < a.rows) own::put4<ElemBF16>(to + row * a.ldo + col, s, col, 0, a.cols);
            } else if ((int64_t)row < a.cols) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if ((int64_t)col + e < a.rows) to[(col + e) * a.ldo + row] = (uint16_t)own::round2<ElemBF16>(s[e], s[e]);
            }
            return true;
        };
        if (cp >= 32 * SMALL_WAVES) {
            // two groups of columns at a time where every wave has as many: B is read half as often
            for (uint32_t s = wave; s < cp / 32; s += SMALL_WAVES) {
                ColumnGroups<RP, 2> g;
                g.read(x, xp, 32 * s, lane);
                g.update(x, xp, m, 32 * s, 0, RP / 16, lane, a.all, out);
            }
        } else {
            // two waves to a group of columns where there are few, each for half of its rows:
            // both have read the group before either writes
            const bool two = cp <= 8 * SMALL_WAVES;
            const uint32_t c0 = 16 * (two ? wave / 2 : wave);
            const uint32_t half = two ? RP / 32 : RP / 16, first = two ? wave % 2 * half : 0;
            ColumnGroups<RP, 1> g;
            if (c0 < cp) g.read(x, xp, c0, lane);
            if (two) __syncthreads();
            if (c0 < cp) g.update(x, xp, m, c0, first, first + half, lane, a.all, out);
            for (uint32_t s = c0 + 16 * SMALL_WAVES; s < cp; s += 16 * SMALL_WAVES) {  // (none where two share a group)
                g.read(x, xp, s, lane);
                g.update(x, xp, m, s, 0, RP / 16, lane, a.all, out);
            }
        }
        __syncthreads();
    }
}

#undef GR_LDS

}  // namespace ortho
}  // namespace gr
