// The end of a residual block and the beginning of the next in one pass, and back:
//
//   p = y r(y),  r(v) = 1 / sqrt(mean(v^2) + eps)
//   total  = round(residual + scale * gate * (p * w))
//   normed = round(total r(total) * w_next)
//
// with a gate of N values for each group of consecutive rows.  Backward, with q =
// total r(total) and the row means over the columns:
//
//   dq = dnormed * w_next
//   d  = dtotal + r(total) (dq - q mean(dq q))             (= dresidual)
//   dp = d * scale * gate * w
//   dy = r(y) (dp - p mean(dp p))
//   dw = sum over rows of d scale gate p,  dgate = sum over its rows of d scale p w,
//   dw_next = sum over rows of dnormed q
//
// in fp32 from the 16-bit inputs, each output rounded once.  Both passes are bound by
// memory: a row is held in registers, every input is read once and every output
// written once (forward 4, backward 6 matrices of M x N).  TPR threads hold a row, at
// most C chunks of 8 columns each.  Backward, a thread keeps its columns' sums in
// registers over the rows of its workgroup (one chunk per thread up to 8192 columns: with two, half
// as many waves find room, 8192 x 8192 201 us against 190; beyond that the sums do not all
// fit and some are spilled: of the same bytes 4096 x 16384 takes 384 us and 2048 x 32768 894, and
// rows that are no multiples of 8, which load with branches, half as much again or more), so that only one partial sum per workgroup (or wave,
// where a wave holds a row) and column goes through memory; a second kernel adds
// those in a fixed order.
#pragma once

#include "norm_kernel.hpp"
#include "own_epilogue.hpp"

namespace gr {
namespace sandwich {

constexpr int64_t MAX_N = 32768;

// Rows that the threads of a workgroup hold at once (a wave each, or all of them one), and
// the threads.
constexpr int rows_at_once(int tpr) { return tpr == 64 ? 4 : 1; }
constexpr int threads_for(int tpr) { return tpr == 64 ? 256 : tpr; }

struct Args {
    const uint16_t *y, *residual, *w, *next_w, *gate;  // w, next_w, gate: nullptr for ones
    uint16_t *total, *normed;                          // normed: nullptr if not wanted
    int64_t M, N, ldy, ldr, ldt, ldn, ld_gate;
    int64_t group;                                     // rows per gate
    float scale, eps;
    int64_t first;                                     // row of the launch's first workgroup
};

// The chunks of 8 columns that thread t of TPR has of rows of N: how many columns each
// holds.  WHOLE: N is a multiple of 8, so that a chunk holds 8 or none; a thread then loads
// without a branch (where it has none, the row's last chunk, for zeros), and all of its loads
// are in flight at once.
template <int TPR, int C, bool WHOLE>
struct Columns {
    int n[C];
    bool more;  // 8 columns or more: a short chunk has 8 - n before it
    uint32_t at[C];
    __device__ __forceinline__ Columns(int t, int64_t N) : more(N > 8) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const uint32_t first = 8u * (uint32_t)(t + c * TPR);
            n[c] = first < N ? (N - first < 8 ? (int)(N - first) : 8) : 0;
            at[c] = WHOLE && n[c] == 0 ? (uint32_t)N - 8u : first;
        }
    }
    __device__ __forceinline__ void load(const uint16_t* row, u32x4 (&v)[C]) const {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if constexpr (WHOLE) v[c] = *reinterpret_cast<const own::u32x4_any*>(row + at[c]);
            else v[c] = n[c] > 0 ? mx::load8(row + at[c], n[c], more) : u32x4{0u, 0u, 0u, 0u};
        }
    }
    // Zeros where there are no columns.
    __device__ __forceinline__ void clear(u32x4 (&v)[C]) const {
        if constexpr (WHOLE) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) v[c][i] = n[c] > 0 ? v[c][i] : 0u;
        }
    }
    __device__ __forceinline__ void store(uint16_t* row, int c, const u32x4& v) const {
        if (n[c] == 0) return;
        if constexpr (WHOLE) *reinterpret_cast<own::u32x4_any*>(row + at[c]) = v;
        else own::put8<true, false>(row + at[c], v, 0, 0, n[c]);
    }
};

__device__ __forceinline__ float half_up(float sum, int64_t N, float eps) { return mx::inv_sqrt(sum / (float)N + eps); }

// Sums of K values over the TPR threads of a row, the same bits in each of them.  red:
// K * TPR / 64 floats of this call's own.
template <int TPR, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float* red) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = mx::wave_sum(v[k]);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        if (threadIdx.x % 64 == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) red[k * W + threadIdx.x / 64] = v[k];
        }
        __syncthreads();
        const int lane = threadIdx.x % 64;
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = mx::wave_sum(lane < W ? red[k * W + lane] : 0.0f);
    }
}

template <typename E, int TPR, int C, bool WHOLE>
__global__ void __launch_bounds__(threads_for(TPR)) forward_kernel(Args a) {
    constexpr int kRows = rows_at_once(TPR);
    __shared__ float red[2][TPR > 64 ? TPR / 64 : 1];
    const int64_t row = a.first + (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    if (row >= a.M) return;  // whole waves, and no barrier where TPR is 64
    const Columns<TPR, C, WHOLE> col(threadIdx.x % TPR, a.N);
    u32x4 y[C], s[C], w[C], g[C], w2[C];
    col.load(a.y + row * a.ldy, y);
    col.load(a.residual + row * a.ldr, s);
    if (a.w != nullptr) col.load(a.w, w);
    if (a.gate != nullptr) col.load(a.gate + row / a.group * a.ld_gate, g);
    if (a.next_w != nullptr) col.load(a.next_w, w2);
    col.clear(y);
    float sum[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = own::widen8<E>(y[c], i);
            sum[0] = __builtin_fmaf(v, v, sum[0]);
        }
    row_sums<TPR>(sum, red[0]);
    const float r = half_up(sum[0], a.N, a.eps) * a.scale;
    sum[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float b = own::widen8<E>(y[c], i) * r;
            if (a.w != nullptr) b *= own::widen8<E>(w[c], i);
            if (a.gate != nullptr) b *= own::widen8<E>(g[c], i);
            v[i] = own::widen8<E>(s[c], i) + b;
        }
        s[c] = own::round8<E>(v);
        if (col.n[c] > 0) {
            col.store(a.total + row * a.ldt, c, s[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float z = i < col.n[c] ? own::widen8<E>(s[c], i) : 0.0f;
                sum[0] = __builtin_fmaf(z, z, sum[0]);
            }
        }
    }
    if (a.normed == nullptr) return;
    row_sums<TPR>(sum, red[1]);
    const float r2 = half_up(sum[0], a.N, a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (col.n[c] == 0) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = own::widen8<E>(s[c], i) * r2;
            if (a.next_w != nullptr) v[i] *= own::widen8<E>(w2[c], i);
        }
        col.store(a.normed + row * a.ldn, c, own::round8<E>(v));
    }
}

struct BwdArgs {
    const uint16_t *dtotal, *dnormed, *y, *total, *w, *next_w, *gate;  // dtotal, dnormed: nullptr for zeros
    uint16_t *dy, *dresidual, *dw, *dnext_w, *dgate;                   // dw, dnext_w, dgate: nullptr if not wanted
    float* part;         // slots x 2 x N partial sums
    int64_t M, N, ld_dt, ld_dn, ldy, ldt, ld_dy, ld_dr, ld_gate, ld_dgate;
    int64_t group;       // rows per gate
    int64_t groups;      // gates (1 without a gate)
    int64_t split;       // slots per gate where that is at least 1, else 0
    int64_t slots;       // partial sums of a column
    float scale, eps;
};

// The rows [first, end) of a slot, which belong to one gate, or to whole gates
// where there are fewer slots than gates (split 0).
struct Rows {
    int64_t first, end;
};
__device__ __forceinline__ Rows rows_of(const BwdArgs& a, int64_t slot) {
    if (a.split > 0) {
        const int64_t g = slot / a.split, s = slot % a.split;
        return {g * a.group + a.group * s / a.split, g * a.group + a.group * (s + 1) / a.split};
    }
    return {a.groups * slot / a.slots * a.group, a.groups * (slot + 1) / a.slots * a.group};
}

template <int C>
__device__ __forceinline__ void packed(u32x4 (&v)[C]) {
#pragma unroll
    for (int c = 0; c < C; ++c) asm volatile("" : "+v"(v[c]));
}

// SPLIT: a slot's rows have one gate, and its first partial sum is that of d scale
// p; else that times the gate, and dgate is written here.
template <typename E, int TPR, int C, bool SPLIT, bool WHOLE>
__global__ void __launch_bounds__(threads_for(TPR)) backward_kernel(BwdArgs a) {
    constexpr int kRows = rows_at_once(TPR);
    constexpr int W = TPR > 64 ? TPR / 64 : 1;
    __shared__ float red[2][4 * W];
    const int64_t slot = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    if (slot >= a.slots) return;  // whole waves, and no barrier where TPR is 64
    const Columns<TPR, C, WHOLE> col(threadIdx.x % TPR, a.N);
    const Rows rows = rows_of(a, slot);
    // what is absent counts as ones, and as zeros among the gradients
    u32x4 w[C], w2[C], g[C], y[C], z[C], dt[C], dn[C], next[4][C];
    constexpr uint32_t one = E::kIsF16 ? 0x3C003C00u : 0x3F803F80u;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        w[c] = w2[c] = g[c] = u32x4{one, one, one, one};
        next[0][c] = next[1][c] = next[2][c] = next[3][c] = u32x4{0u, 0u, 0u, 0u};
    }
    if (a.w != nullptr) col.load(a.w, w);
    if (a.next_w != nullptr) col.load(a.next_w, w2);
    if (SPLIT && a.gate != nullptr) col.load(a.gate + rows.first / a.group * a.ld_gate, g);
    float s1[C][8], s2[C][8], sw[SPLIT ? 1 : C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s1[c][i] = s2[c][i] = 0.0f;
            if constexpr (!SPLIT) sw[c][i] = 0.0f;
        }
    // A row is fetched while the one in front of it is worked on, where the registers are
    // there (8192 x 8192: 190 -> 185 us).
    constexpr bool kAhead = C == 1;
    auto fetch = [&](int64_t row) {
        col.load(a.y + row * a.ldy, next[0]);
        col.load(a.total + row * a.ldt, next[1]);
        if (a.dtotal != nullptr) col.load(a.dtotal + row * a.ld_dt, next[2]);
        if (a.dnormed != nullptr) col.load(a.dnormed + row * a.ld_dn, next[3]);
    };
    if (kAhead && rows.first < rows.end) fetch(rows.first);
    for (int64_t row = rows.first; row < rows.end; ++row) {
        if (!kAhead) fetch(row);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            y[c] = next[0][c];
            z[c] = next[1][c];
            dt[c] = next[2][c];
            dn[c] = next[3][c];
        }
        if (kAhead && row + 1 < rows.end) fetch(row + 1);
        if (!SPLIT && row % a.group == 0) col.load(a.gate + row / a.group * a.ld_gate, g);
        col.clear(y);
        col.clear(z);
        col.clear(dn);
        col.clear(dt);
        // packed(): values wait for their next use in 16 bits, not widened
        packed(w2);
        float sum[3] = {0.0f, 0.0f, 0.0f};  // of y^2, total^2, dq total
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float yv = own::widen8<E>(y[c], i), zv = own::widen8<E>(z[c], i);
                sum[0] = __builtin_fmaf(yv, yv, sum[0]);
                sum[1] = __builtin_fmaf(zv, zv, sum[1]);
                sum[2] = __builtin_fmaf(own::widen8<E>(dn[c], i) * own::widen8<E>(w2[c], i), zv, sum[2]);
            }
        row_sums<TPR>(sum, red[0]);
        packed(y);
        packed(z);
        packed(dn);
        packed(w2);
        packed(w);
        packed(g);
        const float r1 = half_up(sum[0], a.N, a.eps), r2 = half_up(sum[1], a.N, a.eps);
        const float mean2 = sum[2] * r2 / (float)a.N;
        float d[C][8], dot[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float dnv = own::widen8<E>(dn[c], i), q = own::widen8<E>(z[c], i) * r2;
                const float dq = dnv * own::widen8<E>(w2[c], i);
                d[c][i] = __builtin_fmaf(r2, __builtin_fmaf(-q, mean2, dq), own::widen8<E>(dt[c], i));
                s2[c][i] = __builtin_fmaf(dnv, q, s2[c][i]);
            }
            col.store(a.dresidual + row * a.ld_dr, c, own::round8<E>(d[c]));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = own::widen8<E>(y[c], i) * r1, v = d[c][i] * a.scale;
                s1[c][i] = __builtin_fmaf(v, p, s1[c][i]);
                d[c][i] = v * own::widen8<E>(g[c], i) * own::widen8<E>(w[c], i);  // dp from here on
                dot[0] = __builtin_fmaf(d[c][i], p, dot[0]);
            }
        }
        row_sums<TPR>(dot, red[1]);
        packed(y);
        const float mean1 = dot[0] / (float)a.N;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = r1 * __builtin_fmaf(-(own::widen8<E>(y[c], i) * r1), mean1, d[c][i]);
            col.store(a.dy + row * a.ld_dy, c, own::round8<E>(v));
        }
        if constexpr (!SPLIT) {
            if ((row + 1) % a.group == 0) {  // the gate's last row
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        v[i] = s1[c][i] * own::widen8<E>(w[c], i);
                        sw[c][i] = __builtin_fmaf(own::widen8<E>(g[c], i), s1[c][i], sw[c][i]);
                        s1[c][i] = 0.0f;
                    }
                    if (a.dgate != nullptr) col.store(a.dgate + row / a.group * a.ld_dgate, c, own::round8<E>(v));
                }
            }
        }
    }
    if (a.part == nullptr) return;
    float* const to = a.part + slot * 2 * a.N;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < col.n[c]) {
                to[col.at[c] + i] = SPLIT ? s1[c][i] : sw[SPLIT ? 0 : c][i];
                to[a.N + col.at[c] + i] = s2[c][i];
            }
}

// The sums of the slots' partial sums: a workgroup of 256 threads for 32 columns, 32 threads
// for each 4 of them, which take every 32nd slot and meet in LDS in order.  blockIdx.y 0: the
// first sums, 1: the second.
constexpr int REDUCE_COLS = 32, REDUCE_PARTS = 32;
template <typename E>
__global__ void __launch_bounds__(256) reduce_kernel(BwdArgs a) {
    __shared__ __attribute__((aligned(16))) float red[REDUCE_PARTS][REDUCE_COLS];
    const int lane = threadIdx.x % 8, part = threadIdx.x / 8;
    const int64_t n0 = (int64_t)blockIdx.x * REDUCE_COLS, n = n0 + threadIdx.x;
    const bool second = blockIdx.y != 0, mine = threadIdx.x < REDUCE_COLS && n < a.N;
    if (second ? a.dnext_w == nullptr : (a.dw == nullptr && (a.split == 0 || a.dgate == nullptr))) return;
    typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
    const int64_t c = n0 + 4 * lane;
    const float* const src = a.part + (second ? a.N : 0) + c;
    // The sum over the slots [first, end) of column n, for the first 32 threads.
    auto total = [&](int64_t first, int64_t end) {
        if (end > a.slots) end = a.slots;  // no rows: no slots
        f32x4 s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (c + 4 <= a.N) {
#pragma unroll 4
            for (int64_t k = first + part; k < end; k += REDUCE_PARTS) {
                const f32x4 v = *reinterpret_cast<const f32x4_any*>(src + k * 2 * a.N);
                s = f32x4{s[0] + v[0], s[1] + v[1], s[2] + v[2], s[3] + v[3]};
            }
        } else {
            for (int64_t k = first + part; k < end; k += REDUCE_PARTS)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < a.N) s[i] += src[k * 2 * a.N + i];
        }
        __syncthreads();
        *reinterpret_cast<f32x4*>(&red[part][4 * lane]) = s;
        __syncthreads();
        float t = 0.0f;
        if (threadIdx.x < REDUCE_COLS) {
#pragma unroll
            for (int i = 0; i < REDUCE_PARTS; ++i) t += red[i][threadIdx.x];
        }
        return t;
    };
    if (second || a.split == 0) {
        const float s = total(0, a.slots);
        if (mine) (second ? a.dnext_w : a.dw)[n] = E::round(s);
        return;
    }
    const float w = mine && a.w != nullptr ? E::widen(a.w[n]) : 1.0f;
    float dw = 0.0f;
    for (int64_t g = 0; g < a.groups; ++g) {
        const float s = total(g * a.split, (g + 1) * a.split);
        dw = __builtin_fmaf(mine && a.gate != nullptr ? E::widen(a.gate[g * a.ld_gate + n]) : 1.0f, s, dw);
        if (a.dgate != nullptr && mine) a.dgate[g * a.ld_dgate + n] = E::round(s * w);
    }
    if (a.dw != nullptr && mine) a.dw[n] = E::round(dw);
}

}  // namespace sandwich
}  // namespace gr
