// RMS norm with the residual's addition, gated activation, and their write-out
// in 16 bits or in an OCP MX format (elements with one E8M0 scale per 32
// consecutive columns of a row).
//
//   norm   s = round16(x + r);  y = s * w / sqrt(mean(s^2) + eps)
//   gated  y = act(g) * u       (u absent: y = act(g))
//   MX     of a block of 32 values with largest magnitude a:
//          e = floor(log2 a) - emax (emax: 8 for E4M3, 2 for E2M1), held to
//          [-127, 127], e = -127 for a = 0; scale code e + 127; element =
//          y * 2^-e rounded to nearest even, held to +-448 (+-6).  A block with an
//          infinity or NaN gets the scale code 255 (NaN) and zero elements.
//
// Everything between the 16-bit inputs and the output is fp32, rounded once.
// Both kernels are bound by memory: each input is read once into registers
// and each output written once.  A thread handles chunks of 8 consecutive
// columns (one 16-byte load), so a block of 32 lies in 4 neighbouring lanes
// and its largest magnitude takes two DPP steps.  8192x8192 bfloat16 with a residual
// to MX fp8: 87 us, 5.4 TB/s (a copy of 1 GiB reaches 5.0); gated SiLU 4100x14336: 58
// us, 5.1 TB/s.  Small calls are one trip to memory beyond an empty launch: 1x4096
// 3.0 us against 2.8.
#pragma once

#include "common.hpp"

namespace gr {
namespace mx {

// Output formats (equal to the GR_OUT_* values of the C ABI).
enum : int { kOut16 = 0, kOutMx8 = 1, kOutMx4 = 2 };

constexpr uint32_t kInfBits = 0x7F800000u;
constexpr uint32_t kAbsMask = 0x7FFFFFFFu;

// Vectors at any address (the memory system splits a misaligned access
// itself).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));

// 8 consecutive 16-bit values; only the first n (1 to 8) are used, the others are 0.
// Where `before` says that there are 8 - n more in front of p in the same row, those are
// read along in one load and shifted out (their values do not matter: another
// thread may be writing them); else one by one.
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int n, bool before = false) {
    if (n >= 8) return *(const u32x4_any*)p;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (before) {
        v = *(const u32x4_any*)(p - (8 - n));
        const int shift = 16 * (8 - n);  // 16 .. 112 bits
        const uint64_t low = v[0] | (uint64_t)v[1] << 32, high = v[2] | (uint64_t)v[3] << 32;
        const uint64_t l = shift < 64 ? low >> shift | high << (64 - shift) : high >> (shift - 64);
        const uint64_t h = shift < 64 ? high >> shift : 0;
        return u32x4{(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)h, (uint32_t)(h >> 32)};
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) v[i / 2] |= (uint32_t)p[i] << (16 * (i % 2));
    return v;
}

__device__ __forceinline__ void store8(uint16_t* p, u32x4 v, int n) {
    if (n >= 8) {
        *(u32x4_any*)p = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint16_t)(v[i / 2] >> (16 * (i % 2)));
}

template <typename E>
__device__ __forceinline__ float value_of(const u32x4& v, int i) {
    return E::widen((uint16_t)(v[i / 2] >> (16 * (i % 2))));
}

template <typename E>
__device__ __forceinline__ u32x4 round8(const float (&v)[8]) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (uint32_t)E::round(v[2 * i]) | ((uint32_t)E::round(v[2 * i + 1]) << 16);
    return r;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dppf(float x) {
    return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(uint32_t, x)));
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kRowHalfMirror = 0x141, kRowMirror = 0x140;

// f over x of this lane and of the lane 16 (32) further, the same in all lanes: the
// swap of a register with itself gives both halves to every lane.
template <typename F>
__device__ __forceinline__ uint32_t over_16(uint32_t x, F f) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return f(r[0], r[1]);
}
template <typename F>
__device__ __forceinline__ uint32_t over_32(uint32_t x, F f) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return f(r[0], r[1]);
}

// The sum over the 64 lanes, the same bits in each (a fixed tree).
__device__ __forceinline__ float wave_sum(float x) {
    x += dppf<kQuadXor1>(x);
    x += dppf<kQuadXor2>(x);
    x += dppf<kRowHalfMirror>(x);
    x += dppf<kRowMirror>(x);
    const auto add = [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    };
    return __builtin_bit_cast(float, over_32(over_16(__builtin_bit_cast(uint32_t, x), add), add));
}

// Write 8 values of one row: column c8 * 8 on, n of them (n < 8 only for the
// 16-bit output).  For the MX outputs the 4 lanes of a quad hold the 4 chunks of
// one block, so all four call this together.  y points at the row's first
// byte, e at its first scale.
template <typename E, int OUT>
__device__ __forceinline__ void emit(const float (&v)[8], uint8_t* y, uint8_t* e, int64_t c8, int n) {
    if constexpr (OUT == kOut16) {
        store8((uint16_t*)y + c8 * 8, round8<E>(v), n);
    } else {
        // largest magnitude as a bit pattern: infinities and NaN order above
        // every finite value
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __builtin_bit_cast(uint32_t, v[i]) & kAbsMask;
            top = b > top ? b : top;
        }
        uint32_t o = dpp<kQuadXor1>(top);
        top = o > top ? o : top;
        o = dpp<kQuadXor2>(top);
        top = o > top ? o : top;
        constexpr uint32_t emax = OUT == kOutMx8 ? 8 : 2;
        const uint32_t ex = top >> 23;  // floor(log2 top) + 127 for a normal value
        const bool bad = top >= kInfBits;
        const uint32_t code = bad ? 255u : (ex > emax ? ex - emax : 0u);
        // 2^-e = 2^(127 - code); code <= 252 where it is used
        const float inv = bad ? 0.0f : __builtin_bit_cast(float, (254u - code) << 23);
        constexpr float most = OUT == kOutMx8 ? 448.0f : 6.0f;
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = bad ? 0.0f : __builtin_amdgcn_fmed3f(v[i] * inv, -most, most);
        if constexpr (OUT == kOutMx8) {
            u32x2 w;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                int p = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
                p = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], p, true);
                w[i] = (uint32_t)p;
            }
            *(u32x2_any*)(y + c8 * 8) = w;
        } else {
            uint32_t w = 0;
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[0], q[1], 1.0f, 0);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[2], q[3], 1.0f, 1);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[4], q[5], 1.0f, 2);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[6], q[7], 1.0f, 3);
            *(u32_any*)(y + c8 * 4) = w;
        }
        if (c8 % 4 == 0) e[c8 / 4] = (uint8_t)code;
    }
}

// ---- RMS norm -------------------------------------------------------------------

struct NormArgs {
    const uint16_t* x;
    const uint16_t* r;  // nullptr: no residual
    const uint16_t* w;  // nullptr: all ones
    uint16_t* s;        // the rounded sum; nullptr: not stored
    uint8_t* y;
    uint8_t* e;         // scales (MX outputs)
    int64_t M, N, ldx, ldr, lds, ldy_bytes, lde;
    float eps;
};

template <typename E>
__device__ __forceinline__ u32x4 add8(const u32x4& a, const u32x4& b) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = value_of<E>(a, i) + value_of<E>(b, i);
    return round8<E>(v);
}

// 1 / sqrt(v) to the last bit or so: the hardware's estimate (1 ulp) and one
// Newton step.  The step is NaN for v = 0 and v = inf, where the estimate is exact.
__device__ __forceinline__ float inv_sqrt(float v) {
    const float r = __builtin_amdgcn_rsqf(v);
    const float e = __builtin_fmaf(-v * r, r, 1.0f);
    const float n = __builtin_fmaf(0.5f * r, e, r);
    return n == n ? n : r;
}

// Sum over the TPR threads of a row, the same bits in each of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* red) {
    x = wave_sum(x);
    if constexpr (TPR > 64) {
        if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = x;
        __syncthreads();
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) t += red[i];
        x = t;
    }
    return x;
}

// TPR threads (64: a wave of 4 in a workgroup) hold a row in registers, at
// most C chunks of 8 columns each: one read of x and r, one write of s and y.
template <typename E, int OUT, int TPR, int C>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) rms_norm_kernel(NormArgs a) {
    __shared__ float red[TPR > 64 ? TPR / 64 : 1];
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    if (row >= a.M) return;  // whole waves, and no barrier where TPR is 64
    const int64_t chunks = (a.N + 7) / 8;
    const uint16_t* const x = a.x + row * a.ldx;
    u32x4 s[C];
    int n[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t at = t + (int64_t)c * TPR;
        const int64_t left = a.N - at * 8;
        n[c] = at < chunks ? (left < 8 ? (int)left : 8) : 0;
        s[c] = n[c] > 0 ? load8(x + at * 8, n[c], at > 0) : u32x4{0u, 0u, 0u, 0u};
    }
    if (a.r != nullptr) {
        const uint16_t* const r = a.r + row * a.ldr;
        u32x4 b[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
            b[c] = n[c] > 0 ? load8(r + (t + (int64_t)c * TPR) * 8, n[c], a.N > 8) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int c = 0; c < C; ++c) s[c] = add8<E>(s[c], b[c]);
    }
    u32x4 w[C];
    if (a.w != nullptr) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            w[c] = n[c] > 0 ? load8(a.w + (t + (int64_t)c * TPR) * 8, n[c], a.N > 8) : u32x4{0u, 0u, 0u, 0u};
    }
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = value_of<E>(s[c], i);
            sum = __builtin_fmaf(v, v, sum);
        }
    const float scale = inv_sqrt(row_sum<TPR>(sum, red) / (float)a.N + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (n[c] > 0) {
            const int64_t at = t + (int64_t)c * TPR;
            if (a.s != nullptr) store8(a.s + row * a.lds + at * 8, s[c], n[c]);
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = value_of<E>(s[c], i) * scale;
                if (a.w != nullptr) v[i] *= value_of<E>(w[c], i);
            }
            emit<E, OUT>(v, a.y + row * a.ldy_bytes, a.e + row * a.lde, at, n[c]);
        }
    }
}

// Rows longer than the registers hold: one workgroup of 1024 threads reads
// the row twice.  The second time each thread reads again only what it read
// (or, for the sum, wrote) itself.
template <typename E, int OUT>
__global__ void __launch_bounds__(1024) rms_norm_long_kernel(NormArgs a) {
    __shared__ float red[16];
    const int64_t row = blockIdx.x;
    const int64_t chunks = (a.N + 7) / 8;
    const uint16_t* const x = a.x + row * a.ldx;
    const uint16_t* const r = a.r != nullptr ? a.r + row * a.ldr : nullptr;
    float sum = 0.0f;
    for (int64_t at = threadIdx.x; at < chunks; at += 1024) {
        const int n = a.N - at * 8 < 8 ? (int)(a.N - at * 8) : 8;
        u32x4 s = load8(x + at * 8, n, at > 0);
        if (r != nullptr) s = add8<E>(s, load8(r + at * 8, n, at > 0));
        if (a.s != nullptr) store8(a.s + row * a.lds + at * 8, s, n);
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = value_of<E>(s, i);
            part = __builtin_fmaf(v, v, part);
        }
        sum += part;
    }
    const float scale = inv_sqrt(row_sum<1024>(sum, red) / (float)a.N + a.eps);
    for (int64_t at = threadIdx.x; at < chunks; at += 1024) {
        const int n = a.N - at * 8 < 8 ? (int)(a.N - at * 8) : 8;
        u32x4 s;
        if (a.s != nullptr) {
            s = load8(a.s + row * a.lds + at * 8, n);
        } else {
            s = load8(x + at * 8, n, at > 0);
            if (r != nullptr) s = add8<E>(s, load8(r + at * 8, n, at > 0));
        }
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = value_of<E>(s, i) * scale;
        if (a.w != nullptr) {
            const u32x4 w = load8(a.w + at * 8, n, at > 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= value_of<E>(w, i);
        }
        emit<E, OUT>(v, a.y + row * a.ldy_bytes, a.e + row * a.lde, at, n);
    }
}

// ---- gated activation ------------------------------------------------------------

// v / (1 + e^-z) within about an ulp: the exponent's argument in two parts,
// and the quotient mended by its remainder.  Above z = -126 ln 2 the divisor
// stays finite; below it the 1 is nothing next to e^-z, and v e^z is taken in
// two halves, since e^z itself is subnormal, the second with the argument's second part.
__device__ __forceinline__ float over_1p_exp(float v, float z) {
    constexpr float kLog2e = 1.44269504088896341f, kLog2eLow = 1.925963033500e-8f, kLn2 = 0.693147180559945309f;
    const float t = -z * kLog2e;
    // (an infinite t has no second part)
    const float low = __builtin_fabsf(t) < 3.0e38f
                          ? __builtin_fmaf(-z, kLog2eLow, __builtin_fmaf(-z, kLog2e, -t))
                          : 0.0f;
    const float p = __builtin_amdgcn_exp2f(t);
    const float d = 1.0f + __builtin_fmaf(p * kLn2, low, p);
    const float r = __builtin_amdgcn_rcpf(d);
    const float q = v * r;
    const float m = __builtin_fmaf(__builtin_fmaf(-q, d, v), r, q);
    const float half = __builtin_amdgcn_exp2f(-0.5f * t);
    return t > 126.0f ? v * half * __builtin_fmaf(-half * kLn2, low, half) : (m == m ? m : q);
}

// The activations of the C ABI with small relative errors, tails included: an MX
// element is rounded relative to its block, not to 1.  SiLU, sigmoid and tanh are within
// a few fp32 ulp; the argument that GELU's erfc and the tanh form's exponential take is
// rounded before, which costs some x^2 half steps more in their tails.
template <int A>
__device__ __forceinline__ float exact_act(float x) {
    if constexpr (A == kActRelu) {
        return x > 0.0f ? x : 0.0f;
    } else if constexpr (A == kActGelu) {
        return 0.5f * x * erfcf(-0.70710678118654752f * x);
    } else if constexpr (A == kActGeluTanh) {
        return over_1p_exp(x, 1.5957691216057308f * (x * __builtin_fmaf(0.044715f * x, x, 1.0f)));
    } else if constexpr (A == kActSilu) {
        return over_1p_exp(x, x);
    } else if constexpr (A == kActSigmoid) {
        return over_1p_exp(1.0f, x);
    } else if constexpr (A == kActTanh) {
        return tanhf(x);
    } else {
        return x;
    }
}

__device__ __forceinline__ float exact_activate(float x, int a) {
    float y = x;
    act::dispatch(a, [&](auto tag) { y = exact_act<decltype(tag)::value>(x); });
    return y;
}

struct GatedArgs {
    const uint16_t* g;
    const uint16_t* u;  // nullptr: no product
    uint8_t* y;
    uint8_t* e;
    int64_t M, N, ldg, ldu, ldy_bytes, lde;
    int act;
};

// A workgroup of THREADS handles THREADS * CHUNKS chunks of one row (CHUNKS 16-byte
// loads of each input in flight per thread), and rows blockIdx.y, blockIdx.y +
// gridDim.y, ...; rows without padding come as one long row.
template <typename E, int OUT, int THREADS, int CHUNKS>
__global__ void __launch_bounds__(THREADS) gated_act_kernel(GatedArgs a) {
    const int64_t chunks = (a.N + 7) / 8;
    const int64_t first = (int64_t)blockIdx.x * (THREADS * CHUNKS) + threadIdx.x;
    for (int64_t row = blockIdx.y; row < a.M; row += gridDim.y) {
        u32x4 g[CHUNKS], u[CHUNKS];
        int n[CHUNKS];
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const int64_t at = first + c * THREADS;
            const int64_t left = a.N - at * 8;
            n[c] = at < chunks ? (left < 8 ? (int)left : 8) : 0;
            if (n[c] > 0) {
                g[c] = load8(a.g + row * a.ldg + at * 8, n[c], at > 0);
                if (a.u != nullptr) u[c] = load8(a.u + row * a.ldu + at * 8, n[c], at > 0);
            }
        }
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            if (n[c] > 0) {
                float v[8];
                act::dispatch(a.act, [&](auto tag) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = exact_act<decltype(tag)::value>(value_of<E>(g[c], i));
                });
                if (a.u != nullptr) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] *= value_of<E>(u[c], i);
                }
                emit<E, OUT>(v, a.y + row * a.ldy_bytes, a.e + row * a.lde, first + c * THREADS, n[c]);
            }
        }
    }
}

}  // namespace mx
}  // namespace gr
