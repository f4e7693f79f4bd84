// Products of 16-bit activations with MX fp4 weights for few rows, and the
// experts of a mixture-of-experts layer built on them.
//
//   C = act(X * W~^T + bias),  W~[n][k] = W[n][k] * 2^(S[n][k/32] - 127)
//
// W (E2M1 pairs, K/2 bytes a row) and S (one E8M0 code per 32 k) are read once
// per 16 * MT rows of X: with few rows the time is that of streaming W.
//
// One wave multiplies a step of 128 k of 16 rows of W: each lane loads 16
// bytes, i.e. one scale block of 32 weights (lane = row n, lane / 16 = block).
// Two permlane swaps transpose the 4 x 4 dwords between the four lane groups and
// four registers, after which register j holds block j in the operand layout
// of a 16 x 16 x 32 MFMA, whose k run is exactly that block.  The weights are
// widened unscaled (exact in fp16 and bfloat16), and the block's scale, one per
// lane because a lane owns one column n of the result, multiplies the
// MFMA's fp32 sum: every scale code 0..254 is exact in both formats, and no
// scaled weight is ever rounded.  Code 255 makes the row's results NaN.
//
// K is split between the waves of a workgroup, each with a ring of steps in
// registers and no barrier until the end; the partial sums are added in LDS in
// wave order, so the results do not depend on timing.
#pragma once

#include "common.hpp"
#include "norm_kernel.hpp"

namespace gr {
namespace w4 {

using mx::u32_any;
using mx::u32x4_any;

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

// The widened weights of one dword: 8 values, k order.
template <typename E>
__device__ __forceinline__ f16x8 widen8(uint32_t d) {
    u32x4 r;
    if constexpr (E::kIsF16) {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 3));
    } else {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 3));
    }
    return __builtin_bit_cast(f16x8, r);
}

// Register j, lane group g  <->  register g, lane group j.
__device__ __forceinline__ void transpose_groups(u32x4& d) {
    auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto e = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    d[0] = c[0];
    d[1] = c[1];
    d[2] = e[0];
    d[3] = e[1];
}

// One step of 128 k in registers: W of NT x 16 rows, X of MT x 16 rows in PL
// planes (2: a value in two parts, high and low).
template <int MT, int NT, int PL>
struct Step {
    u32x4 w[NT];
    uint32_t s[NT];
    u32x4 x[PL][MT][4];
};

// Where a lane reads: rows of W, S and X.  Rows beyond the matrix are clamped
// to its last one; their results are never stored.
template <int MT, int NT, int PL>
struct Rows {
    const uint8_t* w[NT];
    const uint8_t* s[NT];
    const uint16_t* x[PL][MT];
};

// Load step `k` (a multiple of 128, k < K).  The last step may hold fewer than
// four blocks; loads of the blocks it lacks are sent to its first one, and
// the scales' dword is moved back to end at the row's last scale (SHORT, for
// K < 128: read bytewise), so nothing outside the rows is read.
template <bool SHORT, int MT, int NT, int PL>
__device__ __forceinline__ void load_step(Step<MT, NT, PL>& st, const Rows<MT, NT, PL>& rows, int64_t k, int64_t K) {
    const int g = (threadIdx.x % 64) / 16;
    const int left = (int)((K - k) / 32);
    const int64_t wg = k / 2 + (g < left ? g * 16 : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        st.w[nt] = *(const u32x4_any*)(rows.w[nt] + wg);
        if constexpr (SHORT) {
            uint32_t v = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) v |= (uint32_t)rows.s[nt][j < left ? j : 0] << (8 * j);
            st.s[nt] = v;
        } else {
            const int back = left < 4 ? 4 - left : 0;
            st.s[nt] = *(const u32_any*)(rows.s[nt] + k / 32 - back) >> (8 * back);
        }
    }
#pragma unroll
    for (int p = 0; p < PL; ++p)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                st.x[p][mt][j] = *(const u32x4_any*)(rows.x[p][mt] + k + (j < left ? 32 * j : 0) + 8 * g);
}

// acc[mt][nt] += the step's product; D[i][j] of the MFMA has row i of X in (lane /
// 16) * 4 + register and row j of W in lane % 16.
template <typename E, int MT, int NT, int PL>
__device__ __forceinline__ void multiply(Step<MT, NT, PL>& st, f32x4 (&acc)[MT][NT], int64_t k, int64_t K) {
    const int left = (int)((K - k) / 32);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        uint32_t codes = st.s[nt];
        const uint32_t nans = (~codes - 0x01010101u) & codes & 0x80808080u;  // bytes equal to 255 (lowest one exact)
        transpose_groups(st.w[nt]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j < left) {
                const f16x8 w = widen8<E>(st.w[nt][j]);
                // 2^(code - 127): code 0 is the subnormal 2^-127
                const uint32_t bits = ((codes >> (8 * j)) & 255u) << 23;
                float scale = __builtin_bit_cast(float, bits > 0x00400000u ? bits : 0x00400000u);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int p = 0; p < PL; ++p) t = E::mfma16(__builtin_bit_cast(f16x8, st.x[p][mt][j]), w, t);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[mt][nt][i] = __builtin_fmaf(t[i], scale, acc[mt][nt][i]);
                }
            }
        }
        // The scale above was infinite for code 255, and infinity times a sum is
        // infinite or NaN; the definition says NaN.
        if (nans != 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < left && ((codes >> (8 * j)) & 255u) == 255u) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[mt][nt][i] = __builtin_nanf("");
                }
        }
    }
}

// Steps [first, last) through a ring of D steps in registers: load(buffer, i)
// runs D - 1 steps ahead of use(buffer, i).  Loads past the end repeat the last
// step, so that the number of loads in flight is the same in every turn.
template <int D, typename S, typename Load, typename Use>
__device__ __forceinline__ void ring(int first, int last, Load&& load, Use&& use) {
    if (first >= last) return;
    S buf[D];
#pragma unroll
    for (int d = 0; d < D - 1; ++d) load(buf[d], first + d < last ? first + d : last - 1);
    for (int i = first; i < last; i += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int ahead = i + d + D - 1;
            load(buf[(d + D - 1) % D], ahead < last ? ahead : last - 1);
            if (i + d < last) use(buf[d], i + d);
        }
    }
}

// The partial sums of the kw waves that share an item, lane by lane.
template <int REGS>
struct Partials {
    float v[kWaves][REGS][64];
};

// ---- C = act(X W~^T + bias) -------------------------------------------------------

struct LinearArgs {
    const uint16_t* x;
    const uint8_t* w;
    const uint8_t* s;
    const uint16_t* bias;  // nullptr for none
    uint16_t* c;
    int64_t M, N, K, ldx, ldw, lds, ldc;
    int64_t n_tiles, items;  // items: n_tiles * m_tiles, the tiles of one column of C next to each other
    int act;
    int kw;  // waves that share an item's K: 1, 2, 4 or 8
};

template <typename E, int MT, int NT, int D, bool SHORT>
__global__ void __launch_bounds__(kThreads) linear_w4_kernel(LinearArgs a) {
    __shared__ Partials<MT * NT * 4> part;
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int kw = a.kw;
    const int64_t item = (int64_t)blockIdx.x * (kWaves / kw) + wave / kw;
    const int64_t m_tiles = a.items / a.n_tiles;
    const bool valid = item < a.items;
    const int64_t m0 = valid ? item % m_tiles * (16 * MT) : 0;
    const int64_t n0 = valid ? item / m_tiles * (16 * NT) : 0;
    f32x4 acc[MT][NT] = {};
    if (valid) {
        Rows<MT, NT, 1> rows;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int64_t n = n0 + nt * 16 + lane % 16;
            const int64_t at = n < a.N ? n : a.N - 1;
            rows.w[nt] = a.w + at * a.ldw;
            rows.s[nt] = a.s + at * a.lds;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int64_t m = m0 + mt * 16 + lane % 16;
            rows.x[0][mt] = a.x + (m < a.M ? m : a.M - 1) * a.ldx;
        }
        const int steps = (int)((a.K + 127) / 128);
        const int w = wave % kw;
        const int first = (int)((int64_t)steps * w / kw), last = (int)((int64_t)steps * (w + 1) / kw);
        using S = Step<MT, NT, 1>;
        ring<D, S>(
            first, last, [&](S& st, int i) { load_step<SHORT>(st, rows, (int64_t)i * 128, a.K); },
            [&](S& st, int i) { multiply<E>(st, acc, (int64_t)i * 128, a.K); });
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) part.v[wave][(mt * NT + nt) * 4 + i][lane] = acc[mt][nt][i];
    __syncthreads();
    if (!valid) return;
    // the item's waves share its MT * NT * 4 registers of 64 lanes
    const int w0 = wave / kw * kw;
#pragma unroll 1
    for (int r = wave % kw; r < MT * NT * 4; r += kw) {
        float v = 0.0f;
        for (int w = 0; w < kw; ++w) v += part.v[w0 + w][r][lane];
        const int i = r % 4, nt = r / 4 % NT, mt = r / 4 / NT;
        const int64_t m = m0 + mt * 16 + lane / 16 * 4 + i, n = n0 + nt * 16 + lane % 16;
        if (m < a.M && n < a.N) {
            if (a.bias != nullptr) v += E::widen(a.bias[n]);
            a.c[m * a.ldc + n] = E::round(mx::exact_activate(v, a.act));
        }
    }
}

// ---- mixture of experts -----------------------------------------------------------
//
//   out[t] = sum_j weight[t][j] * (W2[e] * h + b2[e]),  h = act(g) * u,
//   (g, u) = W13[e] * x[t] + b13[e],  e = id[t][j]
//
// Two kernels.  The first makes h for every (expert, token) pair, the second
// multiplies by W2 and adds a token's experts.  Both work on the experts that
// at least one token chose, so each of their weights is read once, and on chunks
// of 64 tokens (a bit each in an expert's 64-bit set).  Pairs are numbered by
// expert, then token: the number is the row of h.  h holds weight * act(g) * u
// in two bfloat16 parts (high and the rest's high: 16 bits and fp32's
// range), so that the second product starts from nearly fp32 values.

constexpr int kChunk = 64;         // tokens per chunk
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
// sum over the experts of ceil(pairs / 16) < experts + pairs / 16
constexpr int kMaxTiles = kMaxExperts + kChunk * kMaxTopK / 16;

// Which tokens chose which expert, for one chunk (LDS).
struct Routing {
    unsigned long long tokens[kMaxExperts];
    uint16_t expert[kMaxExperts + 1];  // the chosen experts, ascending
    uint16_t row[kMaxExperts + 1];     // first pair of each; [count]: pairs in all
    uint16_t tile[kMaxTiles];          // tiles of 16 pairs: slot in `expert` * 4 + tile of that expert
    int count, tiles;
};

// Fill r from the chunk's ids (n tokens x topk); called by the whole
// workgroup.  Ids outside [0, E) choose nothing, and a token that names an
// expert twice is one pair.
__device__ __forceinline__ void route(Routing& r, const int32_t* ids, int n, int topk, int E) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) r.tokens[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n * topk; i += blockDim.x) {
        const uint32_t e = (uint32_t)ids[i];
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
                r.expert[at] = (uint16_t)e;
                r.row[at] = (uint16_t)(rows + ((upto - mine) & 0xFFFF));
                const int first = tiles + ((upto - mine) >> 16);
                for (int i = 0; i * 16 < pairs; ++i) r.tile[first + i] = (uint16_t)(at * 4 + i);
            }
            const int all = __shfl(upto, 63);
            count += __popcll(chosen);
            rows += all & 0xFFFF;
            tiles += all >> 16;
        }
        if (lane == 0) {
            r.count = count;
            r.tiles = tiles;
            r.row[count] = (uint16_t)rows;
        }
    }
    __syncthreads();
}

struct MoeArgs {
    const uint16_t* x;
    const int32_t* ids;
    const float* weights;
    const uint8_t *w13, *s13, *w2, *s2;
    const uint16_t *b13, *b2;  // nullptr for none
    uint16_t* h;               // two planes of T * topk rows of I (bfloat16)
    uint16_t* c;
    int64_t T, H, I, ldx, ldc;
    int E, topk, act, kw;
};

// The r-th token of a set, for r < its size.
__device__ __forceinline__ int nth_token(unsigned long long set, int r) {
    for (int i = 0; i < r; ++i) set &= set - 1;
    return __ffsll(set) - 1;
}

// h.  An item is 16 columns of h for 16 pairs of one expert: the 16 rows of
// gate weights and the 16 of up weights.  The grid is at most a few
// workgroups per CU, each taking items in turn, so the routing is read once per
// workgroup.
template <typename E, int D, bool SHORT>
__global__ void __launch_bounds__(kThreads) moe_gate_up_kernel(MoeArgs a) {
    __shared__ Routing r;
    __shared__ Partials<8> part;
    const int64_t t0 = (int64_t)blockIdx.y * kChunk;
    const int n_tok = (int)(a.T - t0 < kChunk ? a.T - t0 : kChunk);
    route(r, a.ids + t0 * a.topk, n_tok, a.topk, a.E);
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int kw = a.kw, groups = kWaves / kw;
    const int n_tiles = (int)((a.I + 15) / 16);
    const int steps = (int)((a.H + 127) / 128);
    const int64_t items = (int64_t)r.tiles * n_tiles;
    const int64_t turns = (items + (int64_t)gridDim.x * groups - 1) / ((int64_t)gridDim.x * groups);
    for (int64_t turn = 0; turn < turns; ++turn) {
        const int64_t item = (turn * gridDim.x + blockIdx.x) * groups + wave / kw;
        const bool valid = item < items;
        const int at_tile = valid ? r.tile[item / n_tiles] : 0;
        const int slot = __builtin_amdgcn_readfirstlane(at_tile / 4), rt = __builtin_amdgcn_readfirstlane(at_tile % 4);
        const int n0 = valid ? (int)(item % n_tiles) * 16 : 0;
        const int e = r.expert[slot];
        const unsigned long long set = r.tokens[e];
        const int pairs = __popcll(set);
        f32x4 acc[1][2] = {};
        if (valid) {
            Rows<1, 2, 1> rows;
            const int64_t n = n0 + lane % 16 < a.I ? n0 + lane % 16 : a.I - 1;
            const int64_t at = (int64_t)e * 2 * a.I + n;
            rows.w[0] = a.w13 + at * (a.H / 2);
            rows.w[1] = a.w13 + (at + a.I) * (a.H / 2);
            rows.s[0] = a.s13 + at * (a.H / 32);
            rows.s[1] = a.s13 + (at + a.I) * (a.H / 32);
            const int p = rt * 16 + lane % 16;
            rows.x[0][0] = a.x + (t0 + nth_token(set, p < pairs ? p : pairs - 1)) * a.ldx;
            const int w = wave % kw;
            const int first = steps * w / kw, last = steps * (w + 1) / kw;
            using S = Step<1, 2, 1>;
            ring<D, S>(
                first, last, [&](S& st, int i) { load_step<SHORT>(st, rows, (int64_t)i * 128, a.H); },
                [&](S& st, int i) { multiply<E>(st, acc, (int64_t)i * 128, a.H); });
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) part.v[wave][nt * 4 + i][lane] = acc[0][nt][i];
        __syncthreads();
        if (valid) {
            const int w0 = wave / kw * kw;
#pragma unroll 1
            for (int i = wave % kw; i < 4; i += kw) {
                float g = 0.0f, u = 0.0f;
                for (int w = 0; w < kw; ++w) {
                    g += part.v[w0 + w][i][lane];
                    u += part.v[w0 + w][4 + i][lane];
                }
                const int p = rt * 16 + lane / 16 * 4 + i;
                const int64_t n = n0 + lane % 16;
                if (p < pairs && n < a.I) {
                    const int64_t t = t0 + nth_token(set, p);
                    if (a.b13 != nullptr) {
                        g += E::widen(a.b13[(int64_t)e * 2 * a.I + n]);
                        u += E::widen(a.b13[(int64_t)e * 2 * a.I + a.I + n]);
                    }
                    float weight = 0.0f;
                    for (int j = 0; j < a.topk; ++j)
                        if (a.ids[t * a.topk + j] == e) weight += a.weights[t * a.topk + j];
                    const float v = mx::exact_activate(g, a.act) * u * weight;
                    const uint16_t high = to_bf16(v);
                    const uint16_t low = to_bf16(v - ElemBF16::widen(high));
                    const int64_t at = (t0 * a.topk + r.row[slot] + p) * a.I + n;
                    a.h[at] = high;
                    a.h[a.T * a.topk * a.I + at] = low;
                }
            }
        }
        __syncthreads();
    }
}

// out.  A workgroup makes 16 columns of out for its chunk's tokens; its waves
// share the (expert, step) units of the whole sum, each adding what it finished of
// an expert into an LDS tile of its own, token by token.
template <typename E, int D, bool SHORT>
__global__ void __launch_bounds__(kThreads) moe_down_kernel(MoeArgs a) {
    __shared__ Routing r;
    __shared__ float tile[kWaves][kChunk][16];
    const int64_t t0 = (int64_t)blockIdx.y * kChunk;
    const int n_tok = (int)(a.T - t0 < kChunk ? a.T - t0 : kChunk);
    for (int i = threadIdx.x; i < kWaves * kChunk * 16; i += kThreads) (&tile[0][0][0])[i] = 0.0f;
    route(r, a.ids + t0 * a.topk, n_tok, a.topk, a.E);
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t n = n0 + lane % 16 < a.H ? n0 + lane % 16 : a.H - 1;
    const int steps = (int)((a.I + 127) / 128);
    const int units = r.tiles * steps;
    const int first = (int)((int64_t)units * wave / kWaves), last = (int)((int64_t)units * (wave + 1) / kWaves);
    f32x4 acc[1][1] = {};
    using S = Step<1, 1, 2>;
    const int64_t plane = a.T * a.topk * a.I;
    // add a tile's sums to the tokens they belong to
    auto flush = [&](int tile_index) {
        const int slot = r.tile[tile_index] / 4, rt = r.tile[tile_index] % 4;
        const unsigned long long set = r.tokens[r.expert[slot]];
        const int pairs = __popcll(set);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = rt * 16 + lane / 16 * 4 + i;
            if (p < pairs) tile[wave][nth_token(set, p)][lane % 16] += acc[0][0][i];
            acc[0][0][i] = 0.0f;
        }
    };
    ring<D, S>(
        first, last,
        [&](S& st, int i) {
            const int at_tile = r.tile[i / steps], slot = at_tile / 4, rt = at_tile % 4;
            const int e = r.expert[slot], base = r.row[slot], pairs = r.row[slot + 1] - base;
            Rows<1, 1, 2> rows;
            rows.w[0] = a.w2 + ((int64_t)e * a.H + n) * (a.I / 2);
            rows.s[0] = a.s2 + ((int64_t)e * a.H + n) * (a.I / 32);
            const int p = rt * 16 + lane % 16;
            const uint16_t* const h = a.h + (t0 * a.topk + base + (p < pairs ? p : pairs - 1)) * a.I;
            rows.x[0][0] = h;
            rows.x[1][0] = h + plane;
            load_step<SHORT>(st, rows, (int64_t)(i % steps) * 128, a.I);
        },
        [&](S& st, int i) {
            multiply<ElemBF16>(st, acc, (int64_t)(i % steps) * 128, a.I);
            if (i + 1 == last || (i + 1) % steps == 0) flush(i / steps);
        });
    __syncthreads();
    for (int i = threadIdx.x; i < n_tok * 16; i += kThreads) {
        const int t = i / 16;
        const int64_t col = n0 + i % 16;
        if (col < a.H) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v += tile[w][t][i % 16];
            if (a.b2 != nullptr) {
                for (int j = 0; j < a.topk; ++j) {
                    const uint32_t e = (uint32_t)a.ids[(t0 + t) * a.topk + j];
                    if (e < (uint32_t)a.E)
                        v += a.weights[(t0 + t) * a.topk + j] * E::widen(a.b2[(int64_t)e * a.H + col]);
                }
            }
            a.c[(t0 + t) * a.ldc + col] = E::round(v);
        }
    }
}

// ---- router ------------------------------------------------------------------------
//
//   logit[t][e] = sum_k x[t][k] * Wr[e][k] + bias[e], fp32
//   the topk largest, in order (ties: lower index first; NaN above infinity),
//   weight[j] = exp(logit_j - max) / sum over the chosen (renorm) or over all E
//
// A workgroup takes 16 tokens and every expert: its waves share the tiles of
// 16 experts and their K, the logits meet in LDS, and each wave then
// picks for whole tokens.

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
    uint32_t o = mx::dpp<mx::kQuadXor1>(x);
    x = o > x ? o : x;
    o = mx::dpp<mx::kQuadXor2>(x);
    x = o > x ? o : x;
    o = mx::dpp<mx::kRowHalfMirror>(x);
    x = o > x ? o : x;
    o = mx::dpp<mx::kRowMirror>(x);
    x = o > x ? o : x;
    o = __shfl_xor(x, 16);
    x = o > x ? o : x;
    o = __shfl_xor(x, 32);
    return o > x ? o : x;
}

// The topk of one token's E logits, by one wave; PER logits per lane (expert
// = lane + 64 * i).
template <int PER>
__device__ __forceinline__ void pick(const float* logits, int E, int topk, int renorm, int32_t* ids, float* weights) {
    const int lane = threadIdx.x % 64;
    float v[PER];
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        v[i] = e < E ? logits[e] : 0.0f;
        key[i] = e < E ? order_bits(v[i]) : 0u;
    }
    int my_id = 0;
    float my_logit = 0.0f, top = 0.0f;
    for (int j = 0; j < topk; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) m = key[i] > m ? key[i] : m;
        m = wave_max(m);
        int id = 0, owner = -1;
        float logit = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const unsigned long long has = __ballot(key[i] == m);
            if (owner < 0 && has != 0) {
                owner = __ffsll(has) - 1;
                id = owner + 64 * i;
                logit = __shfl(v[i], owner);
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

template <typename E, int PER>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(RouteArgs a) {
    __shared__ float part[kRouteWaves][4][64];
    __shared__ float logits[16][64 * PER];
    const int lane = threadIdx.x % 64, g = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t t0 = (int64_t)blockIdx.x * 16;
    const int n_tiles = (a.E + 15) / 16;
    // waves per tile of 16 experts: a power of two, all 16 for one tile
    int kw = kRouteWaves;
    while (kw > 1 && kw * n_tiles > kRouteWaves) kw /= 2;
    const int per_turn = kRouteWaves / kw;
    const int64_t t = t0 + lane % 16 < a.T ? t0 + lane % 16 : a.T - 1;
    const uint16_t* const x = a.x + t * a.ldx;
    const int64_t steps = (a.H + 31) / 32;
    const int64_t first = steps * (wave % kw) / kw, last = steps * (wave % kw + 1) / kw;
    const int turns = (n_tiles + per_turn - 1) / per_turn;
    for (int turn = 0; turn < turns; ++turn) {
        const int nt = turn * per_turn + wave / kw;
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
        if (nt < n_tiles) {
            const int e = nt * 16 + lane % 16 < a.E ? nt * 16 + lane % 16 : a.E - 1;
            const uint16_t* const w = a.w + (int64_t)e * a.ldw;
            const int64_t whole = a.H / 32 < last ? a.H / 32 : last;
            int64_t k = first;
#pragma unroll 8
            for (; k < whole; ++k) {
                const u32x4 xv = *(const u32x4_any*)(x + k * 32 + g * 8);
                const u32x4 wv = *(const u32x4_any*)(w + k * 32 + g * 8);
                acc = E::mfma16(__builtin_bit_cast(f16x8, xv), __builtin_bit_cast(f16x8, wv), acc);
            }
            if (k < last) {  // the tail of H: absent values are 0 on both sides
                const int64_t left = a.H - (k * 32 + g * 8);
                u32x4 xv = {0u, 0u, 0u, 0u}, wv = {0u, 0u, 0u, 0u};
                if (left > 0) {
                    xv = mx::load8(x + k * 32 + g * 8, left < 8 ? (int)left : 8);
                    wv = mx::load8(w + k * 32 + g * 8, left < 8 ? (int)left : 8);
                }
                acc = E::mfma16(__builtin_bit_cast(f16x8, xv), __builtin_bit_cast(f16x8, wv), acc);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][i][lane] = acc[i];
        __syncthreads();
        // 256 sums per tile
        for (int i = threadIdx.x; i < per_turn * 256; i += kRouteThreads) {
            const int tile = i / 256, reg = i / 64 % 4, l = i % 64;
            float v = 0.0f;
            for (int w = 0; w < kw; ++w) v += part[tile * kw + w][reg][l];
            const int e = (turn * per_turn + tile) * 16 + l % 16;
            if (e < a.E) {
                if (a.bias != nullptr) v += a.bias[e];
                logits[l / 16 * 4 + reg][e] = v;
            }
        }
        __syncthreads();
    }
    const int64_t mine = t0 + wave;
    if (mine < a.T) pick<PER>(logits[wave], a.E, a.topk, a.renorm, a.ids + mine * a.topk, a.weights + mine * a.topk);
}

}  // namespace w4
}  // namespace gr
