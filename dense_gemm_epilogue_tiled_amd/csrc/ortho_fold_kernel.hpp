// A step of the orthogonalisation, behind A's product, where the narrow side is at most 256
// (padded): with D = A - I, which one workgroup's registers hold,
//
//   Y  = D X
//   X <- (a + b + c) X + (b + 2 c) Y + c D Y
//
// which is a X + (b A + c A A) X.  B is never formed: two launches a step, not three (8 x
// 256 x 1024, five steps: 87 us against 126), and X is kept in one layout, not in two.  D and Y,
// both small where the iteration ends, are rounded to fp16 (D times SCALE_A, Y times SCALE_Y);
// Y's own multiple is added before its rounding.
//
// A wave holds 32 rows of D, and the workgroup walks over blocks of 32 columns of X: the
// block is staged in LDS, every wave reads all of it transposed (the matrix instruction wants
// 8 values of a column) and gets its rows of Y, which take the same way.  A lane's results are
// 4 columns of a row.  What bounds it is LDS, from which each product reads its block once
// per wave, and D's way into the registers where there are few blocks.
#pragma once

#include "ortho_kernel.hpp"

namespace gr {
namespace ortho {

constexpr int64_t FOLD_R = 256;  // widest narrow side
constexpr int FOLD_COLS = 32;
constexpr float SCALE_Y = 1024.0f;

struct FoldArgs {
    const uint16_t *x, *d;  // rp x cp, rp x rp
    uint16_t* next;         // rp x cp, or the result: rows x cols bfloat16 (tall: transposed)
    int64_t rows, cols, ldo, batch_o;
    uint32_t cp;
    float k2, y, all, scale;  // c, b + 2 c, a + b + c; scale: of the result
};

enum FoldTo { kNextX, kResult, kResultTall };

#define GR_LDS __attribute__((address_space(3)))

// The 16-byte chunk c of row `row` in a block of 32 columns: the four rows that 16 lanes read
// transposed cover half of the banks, those of the next 16 lanes the other half.
__device__ __forceinline__ uint32_t fold_chunk(uint32_t row, uint32_t c) { return row * 64 + ((c ^ (row >> 2 & 2u)) << 4); }
__device__ __forceinline__ uint32_t fold_value(uint32_t row, uint32_t col) { return fold_chunk(row, col >> 3) + 2 * (col & 7u); }

// acc[i][p] += rows 16 i of D (d) times columns 16 p of the block m.
template <int RP>
__device__ __forceinline__ void fold_product(const GR_LDS uint8_t* m, const f16x8 (&d)[2][RP / 32], uint32_t lane, f32x4 (&acc)[2][2]) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    const uint32_t li = lane & 15u, lg = lane >> 4;
#pragma unroll
    for (int s = 0; s < RP / 32; ++s)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t row = 32 * s + 8 * lg + (li >> 2), col = 16 * p + 4 * (li & 3u);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((GR_LDS s16x4*)(m + fold_value(row, col)));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((GR_LDS s16x4*)(m + fold_value(row + 4, col)));
            const f16x8 f = __builtin_bit_cast(f16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
            for (int i = 0; i < 2; ++i) acc[i][p] = ElemF16::mfma16(f, d[i][s], acc[i][p]);
        }
}

template <int RP, FoldTo TO>
__global__ void __launch_bounds__(2 * RP) fold_kernel(FoldArgs a) {
    constexpr int THREADS = 2 * RP;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * RP * FOLD_COLS * 2];
    GR_LDS uint8_t* const xs = (GR_LDS uint8_t*)lds;
    GR_LDS uint8_t* const ys = xs + RP * FOLD_COLS * 2;
    const uint32_t lane = threadIdx.x & 63u, r0 = 32 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t li = lane & 15u, lg = lane >> 4, blocks = a.cp / FOLD_COLS;
    const uint16_t* const x = a.x + (int64_t)blockIdx.y * RP * a.cp;
    const uint16_t* const dm = a.d + (int64_t)blockIdx.y * RP * RP;
    // chunks threadIdx.x and threadIdx.x + THREADS of a block (4 to a row); a block's are loaded
    // while the one in front of it is worked on
    u32x4 ahead[2];
    auto load = [&](uint32_t block) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t o = threadIdx.x + THREADS * k;
            ahead[k] = *reinterpret_cast<const u32x4*>(x + (int64_t)(o / 4) * a.cp + block * FOLD_COLS + 8 * (o % 4));
        }
    };
    load(blockIdx.x);
    f16x8 d[2][RP / 32];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int s = 0; s < RP / 32; ++s)
            d[i][s] = *reinterpret_cast<const f16x8*>(dm + (r0 + 16 * i + li) * RP + 32 * s + 8 * lg);
    for (uint32_t block = blockIdx.x; block < blocks; block += gridDim.x) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t o = threadIdx.x + THREADS * k;
            *(GR_LDS u32x4*)(xs + fold_chunk(o / 4, o % 4)) = ahead[k];
        }
        __syncthreads();  // (the block before it: its Y has been read by all that are here, too)
        if (block + gridDim.x < blocks) load(block + gridDim.x);
        f32x4 acc[2][2] = {}, keep[2][2];
        fold_product<RP>(xs, d, lane, acc);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t at = fold_value(r0 + 16 * i + li, 16 * p + 4 * lg);
                const u32x2 old = *(const GR_LDS u32x2*)(xs + at);
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    keep[i][p][e] = __builtin_fmaf(a.all, ElemF16::widen((uint16_t)(old[e / 2] >> (16 * (e % 2)))),
                                                   acc[i][p][e] * (a.y * (1.0f / SCALE_A)));
                    v[e] = acc[i][p][e] * (SCALE_Y / (SCALE_A * SCALE_X));
                }
                *(GR_LDS u32x2*)(ys + at) = u32x2{own::round2<ElemF16>(v[0], v[1]), own::round2<ElemF16>(v[2], v[3])};
                acc[i][p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
        __syncthreads();  // (all have read the block of X: the next may be written)
        fold_product<RP>(ys, d, lane, acc);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t row = r0 + 16 * i + li, col = block * FOLD_COLS + 16 * p + 4 * lg;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = __builtin_fmaf(acc[i][p][e], a.k2 * (SCALE_X / (SCALE_A * SCALE_Y)), keep[i][p][e]);
                if constexpr (TO == kNextX) {
                    *reinterpret_cast<u32x2*>(a.next + (int64_t)blockIdx.y * RP * a.cp + (int64_t)row * a.cp + col) =
                        u32x2{own::round2<ElemF16>(v[0], v[1]), own::round2<ElemF16>(v[2], v[3])};
                } else {
                    uint16_t* const to = a.next + blockIdx.y * a.batch_o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] *= a.scale * (1.0f / SCALE_X);
                    if constexpr (TO == kResult) {
                        if (row < a.rows) own::put4<ElemBF16>(to + row * a.ldo + col, v, col, 0, a.cols);
                    } else if (row < a.cols) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (col + e < a.rows) to[(col + e) * a.ldo + row] = (uint16_t)own::round2<ElemBF16>(v[e], v[e]);
                    }
                }
            }
    }
}

#undef GR_LDS

}  // namespace ortho
}  // namespace gr
