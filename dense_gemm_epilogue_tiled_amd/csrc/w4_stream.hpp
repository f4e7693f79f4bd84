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
//
// Measured: 16x28672x8192 (126 MB) 35 us with new weights, 30 when they are cached; a
// plain read of the weights takes 23 to 25.  Matrix cores and conversions would allow
// 14 TB/s (16 conversions of 1.9 ns and 4 MFMA of 7 ns per KB and SIMD); X, 256 KB per CU
// here, and the 25 to 34 KB a microsecond that a CU has in flight do not.
//
// A workgroup that meets other codes goes over its units again with multiply_any, which
// multiplies each block's fp32 sum by its scale: exact for all codes; code 255 gives
// NaN.  (In the loop itself that form cost 20 registers, which spilled.  What spills still:
// 15 to 25 registers of the MX fp4 x MX fp4 kernel with 64 rows and 4 steps, some read
// again for each unit; 4 to 15 of kernels with several passes and of the experts' first
// product, before and after their loops over units or in the second go.)
#pragma once

#include <type_traits>

#include "common.hpp"
#include "norm_kernel.hpp"

namespace gr {
namespace w4 {

using mx::u32x2_any;
using mx::u32x4_any;

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

// A matrix tile of up to 16 rows as a buffer: loads beyond its `bytes` give 0 and
// move nothing.  The pointer and size are the same in all lanes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t* p, uint32_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    const uint64_t low = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)at);
    const uint64_t high = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(low | high << 32), 0,
                                             __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}

// A unit: up to 16 rows of W and S from some k on.
struct Tile {
    const uint8_t *w, *s;
    uint32_t w_bytes, s_bytes;
};

// `rows` rows of K k with the pitches ldw and lds, from k on.
__device__ __forceinline__ Tile tile_at(const uint8_t* w, int64_t ldw, const uint8_t* s, int64_t lds, int64_t rows,
                                        int64_t K, int64_t k) {
    return {w + k / 2, s + k / 32, (uint32_t)((rows - 1) * ldw + (K - k) / 2),
            (uint32_t)((rows - 1) * lds + (K - k) / 32)};
}

// The usual range of a wave: the k from k on, of K.
struct Range {
    int64_t k, left;
};

// The scale codes of a unit, `blocks` whole blocks of whose rows are in the wave's
// range (at least 1, the same in all lanes): the code of the lane's block 4i + g in
// byte g of c[i], or in byte 0 if the range is not whole.  Blocks beyond it, where
// X is 0, repeat the code of block 0.
template <int ST>
__device__ __forceinline__ void load_codes(uint32_t (&c)[ST], __amdgpu_buffer_rsrc_t s, int at, int g, int blocks) {
    if (blocks >= 4 * ST) {
        if constexpr (ST == 1) {
            c[0] = __builtin_amdgcn_raw_buffer_load_b32(s, at, 0, 0);
        } else if constexpr (ST == 2) {
            const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(s, at, 0, 0);
            c[0] = v[0];
            c[1] = v[1];
        } else {
            static_assert(ST == 4, "steps per wave");
            const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(s, at, 0, 0);
#pragma unroll
            for (int i = 0; i < ST; ++i) c[i] = v[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < ST; ++i)
            c[i] = __builtin_amdgcn_raw_buffer_load_b8(s, at + (4 * i + g < blocks ? 4 * i + g : 0), 0, 0);
    }
}

// X in MX fp4 itself: the scaled MFMA 16 x 16 x 128 takes both operands as they are, a
// block and its scale per lane and operand.
struct ElemFp4 {
    static constexpr bool kIsF16 = false;
};
template <typename E>
inline constexpr bool is_fp4 = std::is_same_v<E, ElemFp4>;

typedef int i32x8 __attribute__((ext_vector_type(8)));

// The columns of X in the wave's range, PL planes (2: a value in two parts).
template <typename E, int MT, int PL, int ST>
struct Rows {
    u32x4 x[PL][MT][ST][4];
};
template <int MT, int PL, int ST>
struct Rows<ElemFp4, MT, PL, ST> {
    u32x4 x[MT][ST];
    uint32_t scale[MT];  // byte i: the code of step i
};

// x: this lane's row of each plane and tile from the range's first column on;
// nullptr for a row that does not exist.
template <typename E, int MT, int PL, int ST>
__device__ __forceinline__ void load_rows(Rows<E, MT, PL, ST>& r, const uint16_t* const (&x)[PL][MT], int g, int blocks) {
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

// The same for MX fp4: x the lane's row of each tile from its range on, scale its
// codes.  Blocks that are not there are 0 with the scale 1.
template <int MT, int PL, int ST>
__device__ __forceinline__ void load_rows(Rows<ElemFp4, MT, PL, ST>& r, const uint8_t* const (&x)[MT],
                                          const uint8_t* const (&scale)[MT], int g, int blocks) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        uint32_t code[ST];
#pragma unroll
        for (int i = 0; i < ST; ++i) {
            const bool there = x[mt] != nullptr && 4 * i + g < blocks;
            r.x[mt][i] = there ? *(const u32x4_any*)(x[mt] + 64 * i + 16 * g) : u32x4{0u, 0u, 0u, 0u};
            code[i] = there ? scale[mt][4 * i + g] : 127u;
        }
        r.scale[mt] = 0;
#pragma unroll
        for (int i = 0; i < ST; ++i) r.scale[mt] |= code[i] << (8 * i);
    }
}

// The value that lane % 16 holds, in all four lane groups.
__device__ __forceinline__ uint32_t from_group_0(uint32_t x) {
    const auto a = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false)[0];
}

// What multiplies a unit: the lane's scale codes, relative to ref, and whether there is
// one among the rows that are there that the conversion cannot apply.  The row of W whose code a lane holds is also its column
// of the result (D[i][j] of the MFMA has row i of X in lane / 16 * 4 + register and
// row j of W in lane % 16).
template <typename E, int ST>
struct Scales {
    int ref;
    uint32_t code[ST];
    bool any;

    __device__ __forceinline__ Scales(const uint32_t (&c)[ST], int shift, bool there) {
        ref = 127;
        if constexpr (E::kIsF16) {
            ref = (int)(from_group_0(c[0]) & 255u);
            // far enough for any weights; the fp32 sum keeps its range
            ref = ref < 127 - 24 ? 127 - 24 : (ref > 127 + 24 ? 127 + 24 : ref);
        }
        const uint32_t low = E::kIsF16 ? (uint32_t)(ref - 13) : 2u;
        constexpr uint32_t kSpan = E::kIsF16 ? 26u : 250u;
        uint32_t worst = 0;
#pragma unroll
        for (int i = 0; i < ST; ++i) {
            code[i] = (c[i] >> shift) & 255u;
            worst = code[i] - low > worst ? code[i] - low : worst;
        }
        // (the scaled MFMA takes every code)
        any = !is_fp4<E> && __ballot(there && worst > kSpan) != 0;
    }
};

// acc[mt] += the product of one step: 16 rows of W, 128 k, in units of 2^(ref - 127),
// with codes that the conversion can apply.
template <typename E, int MT, int PL, int ST>
__device__ __forceinline__ void multiply(const u32x4& wi, const Scales<E, ST>& s, int i,
                                         const Rows<E, MT, PL, ST>& r, f32x4 (&acc)[MT]) {
    const float scale = __builtin_bit_cast(float, (s.code[i] + (uint32_t)(127 - s.ref)) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f16x8 w = widen8<E>(wi[j], scale);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int p = 0; p < PL; ++p)
                acc[mt] = E::mfma16(__builtin_bit_cast(f16x8, r.x[p][mt][i][j]), w, acc[mt]);
    }
}

// (I: the step, which selects the byte of X's scales)
template <int I, int MT, int PL, int ST>
__device__ __forceinline__ void multiply_fp4(const u32x4& wi, const Scales<ElemFp4, ST>& s,
                                             const Rows<ElemFp4, MT, PL, ST>& r, f32x4 (&acc)[MT]) {
    const i32x8 w = {(int)wi[0], (int)wi[1], (int)wi[2], (int)wi[3], 0, 0, 0, 0};
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const u32x4& q = r.x[mt][I];
        const i32x8 x = {(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0};
        acc[mt] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, w, acc[mt], 4, 4, I, (int)r.scale[mt], 0,
                                                                   (int)s.code[I]);
    }
}

// The same for any codes, block by block: the groups that hold the other blocks put
// zeros on both sides.  acc is in units of 1 here: next to a small ref a large block would
// pass fp32's range.  takes(m): whether row m of X takes part in the range; a NaN scale
// stays away from rows that only have zeros there because it does not.
template <typename E, int MT, int PL, int ST, typename F>
__device__ __forceinline__ void multiply_any(const u32x4& wi, const Scales<E, ST>& s, int i,
                                             const Rows<E, MT, PL, ST>& r, f32x4 (&acc)[MT], int g, F takes) {
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        const bool mine = g == q;
        const int code = __shfl((int)s.code[i], 16 * q + (int)(threadIdx.x % 16));
        f32x4 t[MT] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f16x8 w = widen8<E>(mine ? wi[j] : 0u, 1.0f);
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
                acc[mt][k] += code == 255 && takes(mt * 16 + 4 * g + k) ? __builtin_nanf("")
                                                                     : __builtin_amdgcn_ldexpf(t[mt][k], code - 127);
    }
}

// Workgroup barrier that orders LDS only: loads in flight stay in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// LDS of a workgroup of NW waves: the partial sums of a batch of TB units per wave,
// twice (one is written while the other is read) or once, and for a K of several
// passes the sums so far of at most kSumTiles 16 x 16 tiles.
constexpr int kSumTiles = 16;
template <int NW, int MT, int TB, int BUFS, bool PASSES>
struct Lds {
    float part[BUFS][TB * MT][NW][256];
    float sum[PASSES ? kSumTiles * 256 : 1];
    int again[NW];  // of each wave: it met codes that the conversion cannot apply
};

// A few rows of one column of a result.  One per thread for 16 rows of X: more would
// take registers that X has, and leave threads idle; four for more rows, in a
// quarter of the instructions (64x8192x8192: 31 -> 27 us).
template <int R>
struct Column {
    float v[R];
};
constexpr int rows_at_once(int MT) { return MT == 1 ? 1 : 4; }

// Units [u0, u1) of policy P by one workgroup of NW waves.  kw of them share a
// unit's K, 128 * ST each; with PASSES the X of the next kw * 128 * ST k is loaded
// and the units are gone through again, at most kSumTiles / MT of them.
// P gives
//   run(u)                    what the units from u on share: their X and more; run.end
//                             is the first unit with other rows of X
//   range(k)                  where the k from k on are: range.left of them from there
//   x(run, plane, m, range)   row m of X from the range on, or nullptr
//   takes(range, m)           whether row m of X, if there is one, has a part in the range
//   tile(run, i, range)       the run's i-th unit from the range on
//   rows(run, i)              the number of its rows
//   K, ldw, lds               in k and bytes
//   kPair                     a run's units 2i and 2i + 1 are finished together
//   early(u0, u1), late(u0, value)   a load that goes out before all others, and what is
//                             done with its value once they are under way
//   wanted(run, i, m, n), finish(run, i, m, n, v[, v2])   column n of unit i, rows m ..
// ANY: for any scale codes; otherwise returns whether there were some that need it, in
// which case the results are not right.
template <bool ANY, typename E, int PL, int ST, int NW, int MT, int TB, int BUFS, bool PASSES, typename P>
__device__ __forceinline__ bool stream_units_by(const P& p, Lds<NW, MT, TB, BUFS, PASSES>& lds, int u0, int u1,
                                                int kw) {
    // units in flight: 4 steps where a batch has as many units
    constexpr int D = 4 / ST < TB ? 4 / ST : TB;
    static_assert(TB % D == 0, "a batch is a whole number of turns of the ring");
    constexpr int kPer = P::kPair ? 2 : 1;
    const int lane = threadIdx.x % 64, g = lane / 16, r16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int groups = NW / kw, group = wave / kw, part_of = wave % kw;  // powers of two
    const int64_t span = (int64_t)kw * (128 * ST);
    const auto ahead = p.early(u0, u1);
    bool bad = false;
    int parity = 0;
    for (int64_t pass = 0; pass == 0 || (PASSES && pass * span < p.K); ++pass) {
        const int64_t k0 = pass * span + part_of * (128 * ST);
        const auto range = p.range(k0);
        const int64_t left = range.left / 32;
        const bool active = left > 0;
        const int blocks = (int)(left < 4 * ST ? left : 4 * ST), shift = blocks < 4 * ST ? 0 : 8 * g;
        const int w_at = r16 * (int)p.ldw + 16 * g, s_at = r16 * (int)p.lds;
        const bool last_pass = !PASSES || (pass + 1) * span >= p.K;
        // runs of units with the same X
        for (int from = u0, to = 0; from < u1; from = to) {
            const auto run = p.run(from);
            to = run.end < u1 ? run.end : u1;
            const int units = to - from;
            const int turns = (units + TB * groups - 1) / (TB * groups);
            // the i-th unit of this wave; units that are finished together stay together
            const auto unit_of = [&](int i) { return (i / kPer * groups + group) * kPer + i % kPer; };
            const auto tile_of = [&](int i) {
                const int u = unit_of(i);
                Tile t = p.tile(run, u < units ? u : units - 1, range);
                if (u >= units) t.w_bytes = t.s_bytes = 0;
                return t;
            };
            u32x4 w[D][ST];
            uint32_t c[D][ST];
            Rows<E, MT, PL, ST> rows;
            if (active) {
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    const Tile t = tile_of(d);
                    load_codes<ST>(c[d], buffer_of(t.s, t.s_bytes), s_at, g, blocks);
#pragma unroll
                    for (int i = 0; i < ST; ++i)
                        w[d][i] = __builtin_amdgcn_raw_buffer_load_b128(buffer_of(t.w, t.w_bytes), w_at + 64 * i, 0, 0);
                }
                if constexpr (is_fp4<E>) {
                    const uint8_t *x[MT], *scale[MT];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        x[mt] = p.x(mt * 16 + r16, range);
                        scale[mt] = p.x_scale(mt * 16 + r16, range);
                    }
                    load_rows<MT, PL, ST>(rows, x, scale, g, blocks);
                } else {
                    const uint16_t* x[PL][MT];
#pragma unroll
                    for (int pl = 0; pl < PL; ++pl)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) x[pl][mt] = p.x(run, pl, mt * 16 + r16, range);
                    load_rows<E, MT, PL, ST>(rows, x, g, blocks);
                }
            }
            if (pass == 0 && from == u0) p.late(u0, ahead);
            for (int turn = 0; turn < turns; ++turn) {
#pragma unroll 1
                for (int t0 = 0; t0 < TB; t0 += D) {
#pragma unroll
                    for (int d = 0; d < D; ++d) {
                        const int t = t0 + d;
                        if (unit_of(turn * TB + t) >= units) break;
                        f32x4 acc[MT];
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) acc[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                        if (active) {
                            const Scales<E, ST> scales(c[d], shift, r16 < p.rows(run, unit_of(turn * TB + t)));
                            bad = bad || scales.any;
                            const Tile next = tile_of(turn * TB + t + D);
                            load_codes<ST>(c[d], buffer_of(next.s, next.s_bytes), s_at, g, blocks);
                            const auto more = [&](int i) {
                                w[d][i] = __builtin_amdgcn_raw_buffer_load_b128(buffer_of(next.w, next.w_bytes),
                                                                                w_at + 64 * i, 0, 0);
                            };
                            if constexpr (is_fp4<E>) {
                                multiply_fp4<0, MT, PL, ST>(w[d][0], scales, rows, acc);
                                more(0);
                                if constexpr (ST > 1) {
                                    multiply_fp4<1, MT, PL, ST>(w[d][1], scales, rows, acc);
                                    more(1);
                                }
                                if constexpr (ST > 2) {
                                    multiply_fp4<2, MT, PL, ST>(w[d][2], scales, rows, acc);
                                    more(2);
                                    multiply_fp4<3, MT, PL, ST>(w[d][3], scales, rows, acc);
                                    more(3);
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < ST; ++i) {
                                    if constexpr (ANY)
                                        multiply_any<E, MT, PL, ST>(w[d][i], scales, i, rows, acc, g,
                                                                    [&](int m) { return p.takes(range, m); });
                                    else
                                        multiply<E, MT, PL, ST>(w[d][i], scales, i, rows, acc);
                                    more(i);
                                }
                            }
                            if constexpr (E::kIsF16 && !ANY) {
#pragma unroll
                                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        acc[mt][k] = __builtin_amdgcn_ldexpf(acc[mt][k], scales.ref - 127);
                            }
                        }
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            *(f32x4*)&lds.part[parity][t * MT + mt][wave][lane * 4] = acc[mt];
                    }
                }
                // (a word for each wave, which it alone writes: nothing orders the waves before this barrier)
                if (!ANY && !is_fp4<E> && lane == 0) lds.again[wave] = bad;
                lds_barrier();
                constexpr int R = rows_at_once(MT);
                // what this turn finishes, pairs counted once
                const int all = TB / kPer * groups, rest = units / kPer - turn * all;
                const int total = (rest < all ? rest : all) * MT * (256 / R);
                // (a thread number that the compiler takes for new in each turn: what follows
                // from it is not kept in registers through the loop above)
                int first = threadIdx.x;
                asm volatile("" : "+v"(first));
                for (int at = first; at < total; at += 64 * NW) {
                    // R rows of one column of one unit: register e % 4 of lane e / 4
                    const int e = at % (256 / R) * R, mt = at / (256 / R) % MT, q = at / (256 / R) / MT;
                    const int m = mt * 16 + e / 64 * 4 + e % 4, n = e / 4 % 16, gi = q & (groups - 1), t = q / groups;
                    const int u = (turn * all + q) * kPer;
                    if (p.wanted(run, u, m, n)) {
                        typedef float Floats __attribute__((ext_vector_type(R)));
                        Column<R> v[kPer];
#pragma unroll
                        for (int h = 0; h < kPer; ++h) {
                            const auto& part = lds.part[parity][(t * kPer + h) * MT + mt];
                            const auto of = [&](int i) { return *(const Floats*)&part[gi * kw + i][e]; };
                            Floats x = of(0);
                            if (kw >= 4) {
                                const Floats b = of(1), y = of(2), z = of(3);
                                x = x + b + y + z;
#pragma unroll 1
                                for (int i = 4; i < kw; i += 4) {
                                    const Floats a = of(i), b = of(i + 1), y = of(i + 2), z = of(i + 3);
                                    x = x + a + b + y + z;
                                }
                            } else if (kw == 2) {
                                x = x + of(1);
                            }
                            if constexpr (PASSES) {
                                Floats& sum = *(Floats*)&lds.sum[((from - u0 + u + h) * MT + mt) * 256 + e];
                                if (pass > 0) x = x + sum;
                                if (!last_pass) sum = x;
                            }
#pragma unroll
                            for (int j = 0; j < R; ++j) v[h].v[j] = x[j];
                        }
                        if (last_pass) {
                            if constexpr (P::kPair)
                                p.finish(run, u, m, n, v[0], v[1]);
                            else
                                p.finish(run, u, m, n, v[0]);
                        }
                    }
                }
                if constexpr (BUFS == 2)
                    parity ^= 1;
                else if (PASSES || turn + 1 < turns || to < u1)
                    lds_barrier();
            }
        }
    }
    if constexpr (ANY || is_fp4<E>) return false;
    // (every wave's word was written before the last barrier; without units there was none)
    return u0 < u1 && __ballot(lds.again[lane % NW] != 0) != 0;
}

template <typename E, int PL, int ST, int NW, int MT, int TB, int BUFS, bool PASSES, typename P>
__device__ __forceinline__ void stream_units(const P& p, Lds<NW, MT, TB, BUFS, PASSES>& lds, int u0, int u1, int kw) {
    const bool again = stream_units_by<false, E, PL, ST>(p, lds, u0, u1, kw);
    if constexpr (!is_fp4<E>) {
        if (__builtin_expect(again, 0)) {
            __syncthreads();
            stream_units_by<true, E, PL, ST>(p, lds, u0, u1, kw);
        }
    }
}

}  // namespace w4
}  // namespace gr
