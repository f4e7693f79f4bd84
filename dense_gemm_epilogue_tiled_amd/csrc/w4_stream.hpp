// The core of the products with MX fp4 weights for few rows: weights stream past
// rows of X that stay in registers.
//
//   v[m][n] = sum_k X[m][k] * W[n][k] * 2^(S[n][k/32] - 127)
//
// W (E2M1 pairs, K/2 bytes a row) and S (one E8M0 code per 32 k) are read once;
// with few rows the time is that of streaming them.  So that nothing else
// moves in the loop, a wave owns a range of 128 * ST k and holds those columns of
// X (16 * MT rows, 64 * ST * MT registers' bytes a lane) for the whole kernel.  It
// takes the W rows in units of 16, one after the other, D units in flight,
// and the waves of a workgroup that share a K add their partial sums in LDS.
//
// MFMA 16 x 16 x 32: a lane holds row lane % 16 and 8 k of its group lane / 16.
// Which k those are is free as long as X and W agree: group g takes the blocks
// of 32 k with number 4s + g, so that a lane's 16-byte load of W is one whole block
// with one scale, and the conversion to 16 bits applies that scale on the way,
// at no cost.  In bfloat16 this is exact for scale codes 2 .. 252.  In fp16 the
// scale is taken relative to the first one of the row in the wave's range,
// which multiplies the fp32 sum afterwards; it is exact within 2^+-13 of that.
// Units with other codes take multiply_any, which multiplies each block's fp32 sum by its
// scale: exact for all codes; code 255 gives NaN.
#pragma once

#include "common.hpp"
#include "norm_kernel.hpp"

namespace gr {
namespace w4 {

using mx::u32_any;
using mx::u32x2_any;
using mx::u32x4_any;

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

// The widened weights of one dword times 2^k (scale holds 2^k): 8 values, k order.
template <typename E>
__device__ __forceinline__ f16x8 widen8(uint32_t d, float scale) {
    u32x4 r;
    if constexpr (E::kIsF16) {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, scale, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, scale, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, scale, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, scale, 3));
    } else {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3));
    }
    return __builtin_bit_cast(f16x8, r);
}

// A unit of W in registers: step s holds the lane's block 4s + g, and byte g of
// c[s] its scale code (byte 0 of c[0]: the code of block 0 in every lane).
template <int ST>
struct Weights {
    u32x4 w[ST];
    uint32_t c[ST];
};

// `blocks` whole blocks of the row from w and s on are in the wave's range (at
// least 1, the same in all lanes).  Absent ones repeat block 0; X is 0 there.
template <int ST>
__device__ __forceinline__ void load_weights(Weights<ST>& b, const uint8_t* w, const uint8_t* s, int g, int blocks) {
    if (blocks >= 4 * ST) {
#pragma unroll
        for (int i = 0; i < ST; ++i) b.w[i] = *(const u32x4_any*)(w + 16 * g + 64 * i);
        if constexpr (ST == 1) {
            b.c[0] = *(const u32_any*)s;
        } else if constexpr (ST == 2) {
            const u32x2 c = *(const u32x2_any*)s;
            b.c[0] = c[0];
            b.c[1] = c[1];
        } else {
#pragma unroll
            for (int i = 0; i < ST; i += 4) {
                const u32x4 c = *(const u32x4_any*)(s + 4 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) b.c[i + j] = c[j];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < ST; ++i) {
            const int at = 4 * i + g < blocks ? 4 * i + g : 0;
            b.w[i] = *(const u32x4_any*)(w + 16 * at);
            b.c[i] = (uint32_t)s[at] << (8 * g);
        }
        if (g != 0) b.c[0] |= s[0];
    }
}

// The columns of X in the wave's range, PL planes (2: a value in two parts).
template <int MT, int PL, int ST>
struct Rows {
    u32x4 x[PL][MT][ST][4];
};

// x: this lane's row of each plane and tile from the range's first column on;
// nullptr for a row that does not exist.
template <int MT, int PL, int ST>
__device__ __forceinline__ void load_rows(Rows<MT, PL, ST>& r, const uint16_t* const (&x)[PL][MT], int g, int blocks) {
#pragma unroll
    for (int p = 0; p < PL; ++p)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < ST; ++i) {
                const bool there = x[p][mt] != nullptr && 4 * i + g < blocks;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    r.x[p][mt][i][j] = there ? *(const u32x4_any*)(x[p][mt] + 128 * i + 32 * g + 8 * j)
                                             : u32x4{0u, 0u, 0u, 0u};
            }
}

// acc[mt] += sum over the unit's blocks, any scale codes, in units of 2^(ref - 127).
// Block by block: the groups that hold the other blocks put zeros on both sides.
template <typename E, int MT, int PL, int ST>
__device__ __forceinline__ void multiply_any(const Weights<ST>& b, const Rows<MT, PL, ST>& r, f32x4 (&acc)[MT], int g,
                                             int ref) {
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < ST; ++i) {
        const int own = (int)((b.c[i] >> (8 * g)) & 255u);
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
            const bool mine = g == q;
            const int code = __shfl(own, 16 * q + (int)(threadIdx.x % 16));
            f32x4 t[MT] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f16x8 w = widen8<E>(mine ? b.w[i][j] : 0u, 1.0f);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int p = 0; p < PL; ++p)
                        t[mt] = E::mfma16(__builtin_bit_cast(f16x8, mine ? r.x[p][mt][i][j] : zero), w, t[mt]);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc[mt][k] += code == 255 ? __builtin_nanf("") : __builtin_amdgcn_ldexpf(t[mt][k], code - ref);
        }
    }
}

// acc[mt] = the unit's product.  D[i][j] of the MFMA has row i of X in (lane /
// 16) * 4 + register and row j of W in lane % 16, so that a lane's own code 0 is
// that of its column.
template <typename E, int MT, int PL, int ST>
__device__ __forceinline__ void multiply(const Weights<ST>& b, const Rows<MT, PL, ST>& r, f32x4 (&acc)[MT], int g) {
    int ref = 127;
    if constexpr (E::kIsF16) {
        ref = (int)(b.c[0] & 255u);
        // far enough for any weights; the fp32 sum keeps its range
        ref = ref < 127 - 24 ? 127 - 24 : (ref > 127 + 24 ? 127 + 24 : ref);
    }
    const uint32_t low = E::kIsF16 ? (uint32_t)(ref - 13) : 2u;
    constexpr uint32_t kSpan = E::kIsF16 ? 26u : 250u;
    uint32_t code[ST], worst = 0;
#pragma unroll
    for (int i = 0; i < ST; ++i) {
        code[i] = (b.c[i] >> (8 * g)) & 255u;
        worst = code[i] - low > worst ? code[i] - low : worst;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (__builtin_expect(__ballot(worst > kSpan) == 0, 1)) {
#pragma unroll
        for (int i = 0; i < ST; ++i) {
            const float scale = __builtin_bit_cast(float, (code[i] + (uint32_t)(127 - ref)) << 23);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f16x8 w = widen8<E>(b.w[i][j], scale);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int p = 0; p < PL; ++p)
                        acc[mt] = E::mfma16(__builtin_bit_cast(f16x8, r.x[p][mt][i][j]), w, acc[mt]);
            }
        }
    } else {
        multiply_any<E, MT, PL, ST>(b, r, acc, g, ref);
    }
    if constexpr (E::kIsF16) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[mt][k] = __builtin_amdgcn_ldexpf(acc[mt][k], ref - 127);
    }
}

// Workgroup barrier that orders LDS only: loads in flight stay in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// LDS of a workgroup: the partial sums of two batches of TB units per wave (one
// is written while the other is read), and for a K of several passes the sums
// so far of at most kSumTiles 16 x 16 tiles.
constexpr int kSumTiles = 16;
template <int MT, int TB, bool PASSES>
struct Lds {
    float part[2][TB * MT][kWaves][256];
    float sum[PASSES ? kSumTiles * 256 : 1];
};

// Units [u0, u1) of policy P by one workgroup.  kw of its waves share a unit's
// K, 128 * ST each; with PASSES the X of the next kw * 128 * ST k is loaded and the
// units are gone through again, at most kSumTiles / MT of them.
// P gives
//   key(u)                    units with the same key have the same rows of X
//   x(u, plane, m)            row m of X, or nullptr
//   row(u, r)                 the index of row r of unit u in W and S
//   w, s, ldw, lds, K
//   kPair                     units 2i and 2i + 1 are finished together
//   finish(u, m, n, v[, v2])  column n of the unit, row m
template <typename E, int MT, int PL, int ST, int TB, bool PASSES, typename P>
__device__ __forceinline__ void stream_units(const P& p, Lds<MT, TB, PASSES>& lds, int u0, int u1, int kw) {
    constexpr int D = 2;
    constexpr int kPer = P::kPair ? 2 : 1;
    const int lane = threadIdx.x % 64, g = lane / 16, r16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int groups = kWaves / kw, group = wave / kw, part_of = wave % kw;
    const int units = u1 - u0;
    if (units <= 0) return;  // (nothing below may ask P for a unit that does not exist)
    const int turns = (units + TB * groups - 1) / (TB * groups);
    const int64_t span = (int64_t)kw * (128 * ST);
    // the i-th unit of this wave, relative to u0; finished pairs stay together
    const auto unit_of = [&](int i) { return (i / kPer * groups + group) * kPer + i % kPer; };
    int parity = 0;
    for (int64_t pass = 0; pass * span < p.K || pass == 0; ++pass) {
        const int64_t k0 = pass * span + part_of * (128 * ST);
        const int64_t left = (p.K - k0) / 32;
        const bool active = left > 0;
        const int blocks = active ? (int)(left < 4 * ST ? left : 4 * ST) : 1;
        const int64_t kw0 = active ? k0 / 2 : 0, ks0 = active ? k0 / 32 : 0;
        // waves that hold a part of this pass
        const int64_t rest = (p.K - pass * span + 128 * ST - 1) / (128 * ST);
        const int parts = rest < kw ? (int)rest : kw;
        const bool last_pass = (pass + 1) * span >= p.K;
        Weights<ST> buf[D];
        Rows<MT, PL, ST> rows;
        int key = -1;
        const auto load = [&](Weights<ST>& b, int i) {
            const int u = unit_of(i);
            const bool there = u < units;
            // (absent units: one line of the last one)
            const int64_t at = p.row(u0 + (there ? u : units - 1), there ? r16 : 0);
            load_weights<ST>(b, p.w + at * p.ldw + kw0, p.s + at * p.lds + ks0, g, blocks);
        };
        if (active) {
#pragma unroll
            for (int d = 0; d < D; ++d) load(buf[d], d);
        }
        for (int turn = 0; turn < turns; ++turn) {
            if (active) {
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    const int i = turn * TB + t, u = unit_of(i);
                    if (u < units) {
                        const int k = p.key(u0 + u);
                        if (k != key) {
                            key = k;
                            const uint16_t* x[PL][MT];
#pragma unroll
                            for (int pl = 0; pl < PL; ++pl)
#pragma unroll
                                for (int mt = 0; mt < MT; ++mt) {
                                    x[pl][mt] = p.x(u0 + u, pl, mt * 16 + r16);
                                    if (x[pl][mt] != nullptr) x[pl][mt] += k0;
                                }
                            load_rows<MT, PL, ST>(rows, x, g, blocks);
                            // a wait here, so that none is needed where the X of an
                            // earlier unit is still there
                            __builtin_amdgcn_s_waitcnt(0x0F70);
                        }
                        f32x4 acc[MT];
                        multiply<E, MT, PL, ST>(buf[t % D], rows, acc, g);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) *(f32x4*)&lds.part[parity][t * MT + mt][wave][lane * 4] = acc[mt];
                    }
                    load(buf[t % D], i + D);
                }
            }
            lds_barrier();
            const int total = TB / kPer * groups * MT * 256;
            for (int at = threadIdx.x; at < total; at += kThreads) {
                const int e = at % 256, q = at / 256, mt = q % MT, t = q / MT % (TB / kPer), gi = q / MT / (TB / kPer);
                const int m = mt * 16 + e / 64 * 4 + e % 4, n = e / 4 % 16;
                const int u = ((turn * (TB / kPer) + t) * groups + gi) * kPer;
                if (u < units && p.wanted(u0 + u, m, n)) {
                    float v[kPer];
#pragma unroll
                    for (int h = 0; h < kPer; ++h) {
                        v[h] = 0.0f;
                        for (int w = 0; w < parts; ++w)
                            v[h] += lds.part[parity][(t * kPer + h) * MT + mt][gi * kw + w][e];
                        if constexpr (PASSES) {
                            float& sum = lds.sum[((u + h) * MT + mt) * 256 + e];
                            if (pass > 0) v[h] += sum;
                            if (!last_pass) sum = v[h];
                        }
                    }
                    if (!PASSES || last_pass) {
                        if constexpr (P::kPair)
                            p.finish(u0 + u, m, n, v[0], v[1]);
                        else
                            p.finish(u0 + u, m, n, v[0]);
                    }
                }
            }
            parity ^= 1;
        }
    }
}

}  // namespace w4
}  // namespace gr
