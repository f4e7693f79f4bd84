// Host side of the operators around the MX products: RMS norm and gated
// activation with MX outputs, 16-bit activations times MX fp4 weights, the router
// and the experts of a mixture-of-experts layer.  See include/gemm_relu.h.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/gemm_relu.h"
#include "host.hpp"
#include "norm_kernel.hpp"
#include "w4_kernel.hpp"

namespace {

static_assert(GR_OUT_16 == gr::mx::kOut16 && GR_OUT_MXFP8 == gr::mx::kOutMx8 && GR_OUT_MXFP4 == gr::mx::kOutMx4,
              "output format codes");

constexpr int64_t kCus = 256;

bool known_fmt(int fmt) { return fmt == GR_FMT_F16 || fmt == GR_FMT_BF16; }
bool known_act(int act) { return act >= 0 && act < gr::kActCount; }
bool known_out(int out) { return out == GR_OUT_16 || out == GR_OUT_MXFP8 || out == GR_OUT_MXFP4; }

int64_t aligned(int64_t bytes) { return (bytes + kWorkspaceAlign - 1) / kWorkspaceAlign * kWorkspaceAlign; }

struct Region {
    uintptr_t at;
    int64_t bytes;
};

bool overlaps(const Region& a, const Region& b) { return overlaps(a.at, a.bytes, b.at, b.bytes); }

// A rows x cols matrix of 16-bit elements (bytes < 0: too large).
Region matrix16(const void* p, int64_t rows, int64_t cols, int64_t ld) {
    return {reinterpret_cast<uintptr_t>(p), p ? span_bytes(rows, cols, ld) : 0};
}
Region matrix8(const void* p, int64_t rows, int64_t cols, int64_t ld) {
    return {reinterpret_cast<uintptr_t>(p), p ? span_bytes8(rows, cols, ld) : 0};
}

// Columns of one row of an output in `out_fmt`, in the units of its pitch
// (16-bit elements, or bytes).
int64_t out_cols(int64_t N, int out_fmt) { return out_fmt == GR_OUT_MXFP4 ? N / 2 : N; }

// Checks shared by rms_norm_mx and gated_act_mx on the output and its scales.
int validate_out(int64_t M, int64_t N, const void* Y, int64_t ldy, const uint8_t* SY, int64_t ld_sy, int out_fmt,
                 Region* y, Region* e) {
    if (!known_out(out_fmt)) return GR_ERR_INVALID_ARG;
    const bool mx = out_fmt != GR_OUT_16;
    if (mx && N % 32 != 0) return GR_ERR_INVALID_DIM;
    const int64_t cols = out_cols(N, out_fmt), blocks = N / 32;
    if (ldy < (cols > 1 ? cols : 1)) return GR_ERR_INVALID_LD;
    if (mx && ld_sy < (blocks > 1 ? blocks : 1)) return GR_ERR_INVALID_LD;
    const bool used = M > 0 && N > 0;
    if (used && (!Y || (mx && !SY))) return GR_ERR_NULL_PTR;
    *y = mx ? matrix8(Y, M, cols, ldy) : matrix16(Y, M, cols, ldy);
    *e = mx ? matrix8(SY, M, blocks, ld_sy) : Region{0, 0};
    if (y->bytes < 0 || e->bytes < 0) return GR_ERR_TOO_LARGE;
    return overlaps(*y, *e) ? GR_ERR_ALIAS : GR_OK;
}

// ---- RMS norm ----------------------------------------------------------------------

// Rows in registers: 64, 256 or 1024 threads with up to 4 chunks of 8 columns.
template <typename E, int OUT, int TPR>
int launch_norm_tpr(const gr::mx::NormArgs& a, int64_t chunks, hipStream_t stream) {
    const int threads = TPR < 256 ? 256 : TPR, rows = threads / TPR;
    const int64_t grid = (a.M + rows - 1) / rows;
    if (chunks <= TPR) return launch(gr::mx::rms_norm_kernel<E, OUT, TPR, 1>, grid, threads, stream, a);
    if (chunks <= 2 * TPR) return launch(gr::mx::rms_norm_kernel<E, OUT, TPR, 2>, grid, threads, stream, a);
    return launch(gr::mx::rms_norm_kernel<E, OUT, TPR, 4>, grid, threads, stream, a);
}

// The fewest threads that hold the row; where the rows do not fill the chip, as many
// as give each one chunk, so that nothing waits twice (77x1501: 5.1 us with 64
// threads per row, 3.2 with 256).
template <typename E, int OUT>
int launch_norm(const gr::mx::NormArgs& a, hipStream_t stream) {
    const int64_t chunks = (a.N + 7) / 8, per = a.M < 2 * kCus ? 1 : 4;
    if (chunks <= per * 64) return launch_norm_tpr<E, OUT, 64>(a, chunks, stream);
    if (chunks <= per * 256) return launch_norm_tpr<E, OUT, 256>(a, chunks, stream);
    if (chunks <= 4 * 1024) return launch_norm_tpr<E, OUT, 1024>(a, chunks, stream);
    return launch(gr::mx::rms_norm_long_kernel<E, OUT>, a.M, 1024, stream, a);
}

template <typename E>
int run_norm(const gr::mx::NormArgs& a, int out_fmt, hipStream_t stream) {
    // rows beyond what one grid counts (2^32 threads) go in further launches
    const int64_t most = int64_t(1) << 21;
    for (int64_t row = 0; row < a.M; row += most) {
        gr::mx::NormArgs b = a;
        b.M = a.M - row < most ? a.M - row : most;
        b.x += row * a.ldx;
        if (b.r) b.r += row * a.ldr;
        if (b.s) b.s += row * a.lds;
        b.y += row * a.ldy_bytes;
        if (b.e) b.e += row * a.lde;
        const int st = out_fmt == GR_OUT_MXFP8   ? launch_norm<E, gr::mx::kOutMx8>(b, stream)
                       : out_fmt == GR_OUT_MXFP4 ? launch_norm<E, gr::mx::kOutMx4>(b, stream)
                                                 : launch_norm<E, gr::mx::kOut16>(b, stream);
        if (st != GR_OK) return st;
    }
    return GR_OK;
}

// ---- gated activation ------------------------------------------------------------

template <typename E, int OUT>
int launch_gated(const gr::mx::GatedArgs& a, hipStream_t stream) {
    const int64_t chunks = (a.N + 7) / 8;
    const auto grid = [&](int64_t per) {
        // (the kernel goes through further rows by itself)
        return dim3((uint32_t)((chunks + per - 1) / per), (uint32_t)(a.M < 65535 ? a.M : 65535));
    };
    // few chunks: one per thread and small workgroups, to reach every CU
    // (8x8192: 4.1 us with 256 threads and two, 3.3 so)
    if (chunks * a.M <= 4 * 64 * kCus) return launch_grid(gr::mx::gated_act_kernel<E, OUT, 64, 1>, grid(64), 64, stream, a);
    return launch_grid(gr::mx::gated_act_kernel<E, OUT, 256, 2>, grid(512), 256, stream, a);
}

template <typename E>
int run_gated(const gr::mx::GatedArgs& a, int out_fmt, hipStream_t stream) {
    if (out_fmt == GR_OUT_MXFP8) return launch_gated<E, gr::mx::kOutMx8>(a, stream);
    if (out_fmt == GR_OUT_MXFP4) return launch_gated<E, gr::mx::kOutMx4>(a, stream);
    return launch_gated<E, gr::mx::kOut16>(a, stream);
}

// ---- 16-bit activations, MX fp4 weights ------------------------------------------

constexpr int64_t kW4MaxPitch = int64_t(1) << 26;

int validate_w4(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* Bt, int64_t ldbt,
                const void* SB, int64_t ld_sb, const void* bias, int act, const void* C, int64_t ldc, int fmt,
                bool with_a = true) {
    if (M < 0 || N < 0 || K < 0 || K % 32 != 0) return GR_ERR_INVALID_DIM;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return GR_ERR_TOO_LARGE;
    if (lda < (K > 1 ? K : 1) || ldbt < (K > 1 ? K / 2 : 1) || ld_sb < (K > 1 ? K / 32 : 1) || ldc < (N > 1 ? N : 1))
        return GR_ERR_INVALID_LD;
    // (the kernels count a tile of 16 rows of the weights in 32 bits)
    if (ldbt > kW4MaxPitch || ld_sb > kW4MaxPitch) return GR_ERR_TOO_LARGE;
    if (!known_act(act) || !known_fmt(fmt)) return GR_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return GR_OK;
    if (!C || (K > 0 && ((with_a && !A) || !Bt || !SB))) return GR_ERR_NULL_PTR;
    const Region c = matrix16(C, M, N, ldc), a = matrix16(A, M, K, lda), b = matrix8(Bt, N, K / 2, ldbt),
                 s = matrix8(SB, N, K / 32, ld_sb), v = matrix16(bias, 1, N, N);
    if (c.bytes < 0 || a.bytes < 0 || b.bytes < 0 || s.bytes < 0) return GR_ERR_TOO_LARGE;
    if (overlaps(c, a) || overlaps(c, b) || overlaps(c, s) || overlaps(c, v)) return GR_ERR_ALIAS;
    return GR_OK;
}

// How a K is divided: steps of 128 per wave (a power of two, at most `most`), the
// waves of a workgroup, those of them that share a unit, and whether they pass
// over the units more than once.  Workgroups of 8 waves, two per CU; of 16 where
// 8 waves do not hold the K at once.
struct Division {
    int steps, waves, kw;
    bool passes;
};

Division divide(int64_t K, int most, bool wide) {
    const int64_t steps = (K + 127) / 128;
    Division d{1, wide && most * 8 < steps ? 16 : 8, 1, false};
    while (d.steps < most && d.steps * d.waves < steps) d.steps *= 2;
    while (d.kw < d.waves && d.steps * d.kw < steps) d.kw *= 2;
    d.passes = (int64_t)d.steps * d.kw < steps;
    return d;
}

template <typename E, int NW, int MT, int ST, bool PASSES>
int launch_w4(const gr::w4::LinearArgs& a, dim3 grid, hipStream_t stream) {
    return launch_grid(gr::w4::linear_w4_kernel<E, NW, MT, ST, PASSES>, grid, 64 * NW, stream, a);
}

template <typename E, int MT>
int launch_w4_rows(const gr::w4::LinearArgs& a, const Division& d, dim3 grid, hipStream_t stream) {
    constexpr int most = MT == 1 ? 4 : 8 / MT;
    if (d.passes) return launch_w4<E, MT == 1 ? 16 : 8, MT, most, true>(a, grid, stream);
    if constexpr (MT == 1)
        if (d.waves == 16) return launch_w4<E, 16, 1, 4, false>(a, grid, stream);
    if (d.steps == most) return launch_w4<E, 8, MT, most, false>(a, grid, stream);
    if constexpr (MT < 4)
        if (d.steps == 2) return launch_w4<E, 8, MT, 2, false>(a, grid, stream);
    return launch_w4<E, 8, MT, 1, false>(a, grid, stream);
}

// Rows of X per workgroup (16 * MT), units of 16 rows of W that one takes, and whether K
// goes to several workgroups (`splits` of `span` k, sums in a workspace with rows of ldp)
// instead of several passes of one.
struct W4Plan {
    int MT;
    Division d;
    int64_t units, splits, span, ldp;
};

// (M and N at least 1.)  What a CU reads (26 KB a microsecond, from L2 or farther) and the units' sums make the
// time of the streaming kernels; the split's second kernel takes 4.5 more.  More
// rows of X per workgroup read W less often, fewer read X less often: 64x1000x2048 takes
// 11.4 us with 64 rows and 6.1 with 16, 64x8192x8192 is fastest with 64.  Two workgroups
// per CU, where they fit, share the units but read X twice.
W4Plan w4_plan(int64_t M, int64_t N, int64_t K, bool split) {
    W4Plan best{};
    double least = -1;
    const int64_t all = (N + 15) / 16, steps = K > 0 ? (K + 127) / 128 : 1;
    for (int MT = 1; MT <= (M <= 16 ? 1 : (M <= 32 ? 2 : 4)); MT *= 2) {
        const int most = MT == 1 ? 4 : 8 / MT;
        const int64_t held = most * (MT == 1 ? 16 : 8);  // steps of 128 that a workgroup holds
        const int64_t needed = (steps + held - 1) / held, tiles = (M + 16 * MT - 1) / (16 * MT);
        const int64_t rows = M < 16 * MT ? M : 16 * MT;
        // as many splits as X needs, or more where the units are too few for the chip
        for (int64_t want = split && M <= 64 && needed <= 64 ? needed : 1;; want *= 2) {
            W4Plan p{MT, {}, 1, 1, steps * 128, (N + 3) / 4 * 4};
            if (want > 1) {
                p.span = (steps + want - 1) / want * 128;
                p.splits = (steps * 128 + p.span - 1) / p.span;
            }
            p.d = divide(p.span, most, MT == 1);
            for (int wgs = 1; wgs <= (MT == 1 && p.d.waves == 8 ? 2 : 1); ++wgs) {
                p.units = (tiles * p.splits * all + kCus * wgs - 1) / (kCus * wgs);
                if (p.units > all) p.units = all;
                const int64_t grid = tiles * p.splits * ((all + p.units - 1) / p.units);
                const int64_t rounds = (grid + kCus * wgs - 1) / (kCus * wgs);
                const double kb = wgs * (2.0 * rows + 8.5 * p.units) * (double)p.span / 1024;
                const double us = rounds * (kb / 26 + (0.4 + 0.27 * MT) * p.units) + (p.splits > 1 ? 4.5 : 0);
                if (least < 0 || us < least) {
                    least = us;
                    best = p;
                }
            }
            if (!split || M > 64 || want * 2 > 64 || p.span <= 512 || tiles * p.splits * all >= kCus) break;
        }
    }
    return best;
}

int64_t w4_workspace(int64_t M, int64_t N, int64_t K) {
    if (M == 0 || N == 0) return 0;
    const W4Plan p = w4_plan(M, N, K, true);
    return p.splits > 1 ? aligned(p.splits * M * p.ldp * 4) : 0;
}

template <typename E, int MT>
int run_w4_rows(gr::w4::LinearArgs a, const W4Plan& p, hipStream_t stream) {
    const Division& d = p.d;
    a.kw = d.kw;
    a.span = p.span;
    a.ldp = p.ldp;
    const int64_t all = (a.N + 15) / 16, room = gr::w4::kSumTiles / MT;
    int64_t gx = (all + p.units - 1) / p.units;
    if (d.passes && gx * room < all) gx = (all + room - 1) / room;
    const int64_t gy = (a.M + 16 * MT - 1) / (16 * MT);
    // rows beyond the grid's y limit go in further launches
    for (int64_t y = 0; y < gy; y += 65535) {
        gr::w4::LinearArgs b = a;
        b.x += y * 16 * MT * a.ldx;
        b.c += y * 16 * MT * a.ldc;
        b.M -= y * 16 * MT;
        const dim3 grid((uint32_t)gx, (uint32_t)(gy - y < 65535 ? gy - y : 65535), (uint32_t)p.splits);
        const int st = launch_w4_rows<E, MT>(b, d, grid, stream);
        if (st != GR_OK) return st;
    }
    if (p.splits == 1) return GR_OK;
    const int64_t per = 4 * gr::w4::kSumThreads;
    return launch_grid(gr::w4::linear_w4_sum_kernel<E>, dim3((uint32_t)((a.N + per - 1) / per), (uint32_t)a.M),
                       gr::w4::kSumThreads, stream, a);
}

template <typename E>
int run_w4(const gr::w4::LinearArgs& a, const W4Plan& p, hipStream_t stream) {
    if (p.MT == 1) return run_w4_rows<E, 1>(a, p, stream);
    if (p.MT == 2) return run_w4_rows<E, 2>(a, p, stream);
    return run_w4_rows<E, 4>(a, p, stream);
}

// ---- both operands in MX fp4 -------------------------------------------------------

// The streaming kernel's time goes with what a CU has to read, some 32 KB a
// microsecond whether from L2 or farther (its L1 holds 32 KB of misses): with tiles of
// 16 * MT rows a CU reads those rows once and takes `units` tiles of 16 rows of Bt.
struct Fp4Plan {
    int MT;
    int64_t units, rounds;
};

Fp4Plan fp4_plan(int64_t M, int64_t N) {
    Fp4Plan best{1, 0, 0};
    int64_t least = 0;
    for (int MT = 1; MT <= 4; MT *= 2) {
        const int64_t tiles = (M + 16 * MT - 1) / (16 * MT), all = (N + 15) / 16;
        int64_t units = (tiles * all + kCus - 1) / kCus;
        if (units > all) units = all;
        const int64_t rounds = (tiles * ((all + units - 1) / units) + kCus - 1) / kCus, rows = rounds * (MT + units);
        if (least == 0 || rows < least) {
            least = rows;
            best = {MT, units, rounds};
        }
    }
    return best;
}

// Whether the streaming kernel is the faster one.  Where gemm_mxfp4_bt has only its guarded
// kernel (K % 128 != 0, rows at odd addresses), 128 x 128 at a time: by what both were
// seen to take over 486 sizes, to which the choice below comes within 1% on average.
// Streaming wins with few tiles and a long K (200x4000x2080 13 against 24 us,
// 4096x4096x4000 119 against 207), the guarded kernel with many and a short one
// (4096x4096x544 26 against 79 us, 8192x8192x1056 169 against 302).
// Against the 128 x 128 tiles without guards, one per CU, where it reads less (4x4096x4096:
// 4.9 against 10.0 us, 512x4096x4096: 29.9 against 17.3, 512x2048x8192 30.7 against 22.1: the
// fewer tiles, the more each reads a microsecond); not where those tiles fill the chip.
bool fp4_streams(int64_t M, int64_t N, int64_t K, int64_t ldbt, int64_t ld_sb, int path) {
    if (ldbt > kW4MaxPitch || ld_sb > kW4MaxPitch || K < 32) return false;
    const int64_t tiles = (M + 127) / 128 * ((N + 127) / 128);
    const Fp4Plan p = fp4_plan(M, N);
    // (fitted: microseconds to start, KB per microsecond, and the sums of a unit)
    const double row = (double)K * 17 / 32 / 1024;  // KB
    if (path == GR_PATH_TILE_EDGE) {
        // (the waves that share a unit's K make its sums; the guarded kernel's tiles leave L2 with a long K)
        const double sums = 0.22 + 0.02 * divide(K, 4, false).kw * p.MT, k = K <= 2304 ? 0.0105 : 0.0135;
        return 4.5 + p.rounds * (16 * (p.MT + p.units) * row / 31 + sums * p.units) <
               5.0 + (tiles + kCus - 1) / kCus * (1 + k * K);
    }
    if (tiles > kCus) return false;
    const double stream = 1.5 + 16 * (p.MT + p.units) * row / 26 + (0.4 + 0.27 * p.MT) * p.units;
    const double tile = 4.5 + 256 * row / (tiles <= 64 ? 52 : (tiles <= 128 ? 42 : 33));
    return stream < tile;
}

template <typename E, int MT>
int run_fp4_rows(gr::w4::Fp4Args a, int64_t units, hipStream_t stream) {
    using namespace gr::w4;
    const Division d = divide(a.K, 4, false);
    a.kw = d.kw;
    const int64_t gy = (a.M + 16 * MT - 1) / (16 * MT);
    const int64_t all = (a.N + 15) / 16;
    int64_t gx = (all + units - 1) / units;
    const int64_t room = kSumTiles / MT;
    if (d.passes && gx * room < all) gx = (all + room - 1) / room;
    for (int64_t y = 0; y < gy; y += 65535) {
        Fp4Args b = a;
        b.x += y * 16 * MT * a.ldx;
        b.sx += y * 16 * MT * a.ldsx;
        b.c += y * 16 * MT * a.ldc;
        b.M -= y * 16 * MT;
        const dim3 grid((uint32_t)gx, (uint32_t)(gy - y < 65535 ? gy - y : 65535));
        const int st = d.passes       ? launch_grid(fp4_stream_kernel<E, MT, 4, true>, grid, 512, stream, b)
                       : d.steps == 4 ? launch_grid(fp4_stream_kernel<E, MT, 4, false>, grid, 512, stream, b)
                       : d.steps == 2 ? launch_grid(fp4_stream_kernel<E, MT, 2, false>, grid, 512, stream, b)
                                      : launch_grid(fp4_stream_kernel<E, MT, 1, false>, grid, 512, stream, b);
        if (st != GR_OK) return st;
    }
    return GR_OK;
}

template <typename E>
int run_fp4(const gr::w4::Fp4Args& a, hipStream_t stream) {
    const Fp4Plan p = fp4_plan(a.M, a.N);
    if (p.MT == 1) return run_fp4_rows<E, 1>(a, p.units, stream);
    if (p.MT == 2) return run_fp4_rows<E, 2>(a, p.units, stream);
    return run_fp4_rows<E, 4>(a, p.units, stream);
}

// ---- mixture of experts ------------------------------------------------------------

constexpr int64_t kMoeMaxDim = int64_t(1) << 20;  // H and I: the kernels count steps of 128 in 32 bits

// The workspace: h (two bfloat16 planes), y (fp32), the pairs' rows.
int64_t moe_h_bytes(int64_t T, int64_t I, int64_t topk) { return aligned(T * topk * I * 4); }
int64_t moe_y_bytes(int64_t T, int64_t H, int64_t topk) { return aligned(T * topk * H * 4); }
int64_t moe_workspace(int64_t T, int64_t H, int64_t I, int64_t topk) {
    return I > 0 ? moe_h_bytes(T, I, topk) + moe_y_bytes(T, H, topk) + aligned(T * topk * 4) : 0;
}

int validate_moe_dims(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk) {
    if (T < 0 || H < 0 || I < 0 || E < 1 || H % 32 != 0 || I % 32 != 0) return GR_ERR_INVALID_DIM;
    if (topk < 1) return GR_ERR_INVALID_ARG;
    if (T > 64 * 65535 || H > kMoeMaxDim || I > kMoeMaxDim || E > gr::w4::kMaxExperts || topk > gr::w4::kMaxTopK)
        return GR_ERR_TOO_LARGE;
    return GR_OK;
}

template <typename E>
int run_moe(gr::w4::MoeArgs a, hipStream_t stream) {
    using namespace gr::w4;
    const uint32_t chunks = (uint32_t)((a.T + kChunk - 1) / kChunk);
    if (a.I > 0) {
        // at most this many tiles of 16 pairs of one expert are in a chunk
        const int64_t n_tok = a.T < kChunk ? a.T : kChunk, pairs = n_tok * a.topk;
        const int64_t tiles = (pairs < a.E ? pairs : a.E) + (n_tok > 16 ? pairs / 16 : 0);
        const Division d13 = divide(a.H, 4, true), d2 = divide(a.I, 2, true);
        a.kw13 = d13.kw;
        a.kw2 = d2.kw;
        // workgroups for every tile of pairs; with several passes no more units each
        // than their sums have room for, whichever tiles there are (an item of the first
        // product is two units)
        const auto grid = [&](int64_t each, const Division& d, int64_t room) {
            int64_t wgs = tiles * each;
            const int64_t most = kCus * (16 / d.waves);
            if (wgs > most) wgs = most;
            const int64_t least = tiles * ((each + room - 1) / room);
            if (d.passes && wgs < least) wgs = least;
            return dim3((uint32_t)wgs, chunks);
        };
        const dim3 g13 = grid(a.I / 16, d13, kSumTiles / 2), g2 = grid(a.H / 16, d2, kSumTiles);
        const int lds = routing_bytes(a.E, a.topk);
        int st = d13.passes        ? launch_lds(moe_gate_up_kernel<E, 16, 4, true>, g13, 1024, lds, stream, a)
                 : d13.waves == 16 ? launch_lds(moe_gate_up_kernel<E, 16, 4, false>, g13, 1024, lds, stream, a)
                 : d13.steps == 4  ? launch_lds(moe_gate_up_kernel<E, 8, 4, false>, g13, 512, lds, stream, a)
                 : d13.steps == 2  ? launch_lds(moe_gate_up_kernel<E, 8, 2, false>, g13, 512, lds, stream, a)
                                   : launch_lds(moe_gate_up_kernel<E, 8, 1, false>, g13, 512, lds, stream, a);
        if (st != GR_OK) return st;
        // few tokens and experts: the sum over the experts within the product, in two passes
        // at most (a third costs what the kernel that it saves does)
        const int64_t parts = tiles * ((a.I + 128 * kFewSteps - 1) / (128 * kFewSteps));
        if (a.T <= kFewTokens && parts <= 32) {
            const int64_t units = a.H / 16, room = kSumTiles;
            int64_t grid = units < kCus ? units : kCus;
            if (parts > 16 && grid * room < units) grid = (units + room - 1) / room;
            return parts > 16 ? launch_lds(moe_down_few_kernel<E, true>, dim3((uint32_t)grid), 1024, lds, stream, a)
                              : launch_lds(moe_down_few_kernel<E, false>, dim3((uint32_t)grid), 1024, lds, stream, a);
        }
        st = d2.passes        ? launch_lds(moe_down_kernel<16, 2, true>, g2, 1024, lds, stream, a)
             : d2.waves == 16 ? launch_lds(moe_down_kernel<16, 2, false>, g2, 1024, lds, stream, a)
             : d2.steps == 2  ? launch_lds(moe_down_kernel<8, 2, false>, g2, 512, lds, stream, a)
                              : launch_lds(moe_down_kernel<8, 1, false>, g2, 512, lds, stream, a);
        if (st != GR_OK) return st;
    }
    const int64_t per = kCombineThreads * 4;
    const dim3 g((uint32_t)((a.H + per - 1) / per), (uint32_t)(a.T < 65535 ? a.T : 65535));
    return launch_grid(moe_combine_kernel<E>, g, kCombineThreads, stream, a);
}

// Two kernels where one CU would read Wr (E * H values) for longer than the second
// kernel takes, and the tokens do not fill the chip by themselves: for one token,
// one kernel takes 20 us at 64 x 4096 and 6.4 at 32 x 2048, two take 5.4.
int64_t route_workspace(int64_t T, int64_t H, int64_t E) {
    if (T > 512 || E * H <= 32768 || H > (int64_t(1) << 24)) return 0;
    const int64_t slice = 32 * gr::w4::kSliceSteps, bytes = (H + slice - 1) / slice * T * E * 4;
    return aligned(bytes);
}

template <typename E>
int run_route(const gr::w4::RouteArgs& a, hipStream_t stream) {
    using namespace gr::w4;
    const int64_t tiles = (a.T + 15) / 16;
    if (a.partial != nullptr) {
        const int64_t slice = 32 * kSliceSteps;
        const dim3 grid((uint32_t)((a.E + 15) / 16), (uint32_t)((a.H + slice - 1) / slice), (uint32_t)tiles);
        const int st = launch_grid(moe_logits_kernel<E>, grid, 64 * kSliceWaves, stream, a);
        if (st != GR_OK) return st;
        const int64_t picks = (a.T + kPickWaves - 1) / kPickWaves;
        if (a.E <= 64) return launch(moe_pick_kernel<1>, picks, 64 * kPickWaves, stream, a);
        if (a.E <= 256) return launch(moe_pick_kernel<4>, picks, 64 * kPickWaves, stream, a);
        return launch(moe_pick_kernel<16>, picks, 64 * kPickWaves, stream, a);
    }
    // tokens beyond what one grid counts (2^32 threads) go in further launches
    const int64_t most = (int64_t(1) << 31) / kRouteThreads;
    for (int64_t at = 0; at < tiles; at += most) {
        RouteArgs b = a;
        b.x += at * 16 * a.ldx;
        b.ids += at * 16 * a.topk;
        b.weights += at * 16 * a.topk;
        b.T -= at * 16;
        const int64_t grid = tiles - at < most ? tiles - at : most;
        const int st = a.E <= 16    ? launch(moe_route_kernel<E, 1, 1>, grid, kRouteThreads, stream, b)
                       : a.E <= 32  ? launch(moe_route_kernel<E, 2, 1>, grid, kRouteThreads, stream, b)
                       : a.E <= 64  ? launch(moe_route_kernel<E, 4, 1>, grid, kRouteThreads, stream, b)
                       : a.E <= 256 ? launch(moe_route_kernel<E, 4, 4>, grid, kRouteThreads, stream, b)
                                    : launch(moe_route_kernel<E, 4, 16>, grid, kRouteThreads, stream, b);
        if (st != GR_OK) return st;
    }
    return GR_OK;
}

}  // namespace

extern "C" {

int rms_norm_mx(int64_t M, int64_t N, const uint16_t* X, int64_t ldx, const uint16_t* R, int64_t ldr,
                const uint16_t* weight, float eps, uint16_t* S, int64_t lds, void* Y, int64_t ldy, uint8_t* SY,
                int64_t ld_sy, int fmt, int out_fmt, void* stream) {
    if (M < 0 || N < 0) return GR_ERR_INVALID_DIM;
    if (M > kMaxDim || N > kMaxDim) return GR_ERR_TOO_LARGE;
    const int64_t nmin = N > 1 ? N : 1;
    if (ldx < nmin || (R && ldr < nmin) || (S && lds < nmin)) return GR_ERR_INVALID_LD;
    if (!known_fmt(fmt) || !(eps >= 0.0f) || !std::isfinite(eps) || (S && !R)) return GR_ERR_INVALID_ARG;
    Region y, e;
    int st = validate_out(M, N, Y, ldy, SY, ld_sy, out_fmt, &y, &e);
    if (st != GR_OK) return st;
    if (M == 0 || N == 0) return GR_OK;
    if (!X) return GR_ERR_NULL_PTR;
    const Region x = matrix16(X, M, N, ldx), r = matrix16(R, M, N, ldr), s = matrix16(S, M, N, lds),
                 w = matrix16(weight, 1, N, N);
    if (x.bytes < 0 || r.bytes < 0 || s.bytes < 0) return GR_ERR_TOO_LARGE;
    // S may be X or R itself and a 16-bit Y may be X itself: each thread has
    // read what it overwrites
    const bool s_is_x = S == X && lds == ldx, s_is_r = S == R && lds == ldr;
    const bool y_is_x = Y == static_cast<const void*>(X) && ldy == ldx && out_fmt == GR_OUT_16;
    if ((overlaps(s, x) && !s_is_x) || (overlaps(s, r) && !s_is_r) || overlaps(s, w) || overlaps(s, y) ||
        overlaps(s, e) || (overlaps(y, x) && !y_is_x) || overlaps(y, r) || overlaps(y, w) || overlaps(e, x) ||
        overlaps(e, r) || overlaps(e, w))
        return GR_ERR_ALIAS;
    // X and R may be the same matrix or overlap, as they are only read; but a
    // write into one of them must not reach the other
    if ((s_is_x && overlaps(s, r) && !s_is_r) || (s_is_r && overlaps(s, x) && !s_is_x)) return GR_ERR_ALIAS;
    st = check_device();
    if (st != GR_OK) return st;
    const gr::mx::NormArgs a{X,   R,   weight, S,  static_cast<uint8_t*>(Y),           SY,    M,  N,
                             ldx, ldr, lds,    out_fmt == GR_OUT_16 ? ldy * 2 : ldy, ld_sy, eps};
    hipStream_t h = static_cast<hipStream_t>(stream);
    return fmt == GR_FMT_BF16 ? run_norm<gr::ElemBF16>(a, out_fmt, h) : run_norm<gr::ElemF16>(a, out_fmt, h);
}

int gated_act_mx(int64_t M, int64_t N, const uint16_t* G, int64_t ldg, const uint16_t* U, int64_t ldu, int act,
                 void* Y, int64_t ldy, uint8_t* SY, int64_t ld_sy, int fmt, int out_fmt, void* stream) {
    if (M < 0 || N < 0) return GR_ERR_INVALID_DIM;
    if (M > kMaxDim || N > kMaxDim) return GR_ERR_TOO_LARGE;
    const int64_t nmin = N > 1 ? N : 1;
    if (ldg < nmin || (U && ldu < nmin)) return GR_ERR_INVALID_LD;
    if (!known_fmt(fmt) || !known_act(act)) return GR_ERR_INVALID_ARG;
    Region y, e;
    int st = validate_out(M, N, Y, ldy, SY, ld_sy, out_fmt, &y, &e);
    if (st != GR_OK) return st;
    if (M == 0 || N == 0) return GR_OK;
    if (!G) return GR_ERR_NULL_PTR;
    const Region g = matrix16(G, M, N, ldg), u = matrix16(U, M, N, ldu);
    if (g.bytes < 0 || u.bytes < 0) return GR_ERR_TOO_LARGE;
    // a 16-bit Y may be G or U itself
    const bool y_is_g = Y == static_cast<const void*>(G) && ldy == ldg && out_fmt == GR_OUT_16;
    const bool y_is_u = Y == static_cast<const void*>(U) && ldy == ldu && out_fmt == GR_OUT_16;
    if ((overlaps(y, g) && !y_is_g) || (overlaps(y, u) && !y_is_u) || overlaps(e, g) || overlaps(e, u))
        return GR_ERR_ALIAS;
    st = check_device();
    if (st != GR_OK) return st;
    gr::mx::GatedArgs a{G, U, static_cast<uint8_t*>(Y), SY, M, N, ldg, ldu, ldy, ld_sy, act};
    // rows without padding are one long row (blocks of 32 stay within rows)
    const int64_t cols = out_cols(N, out_fmt);
    // (unless that row were too long for one grid)
    if (N % 32 == 0 && M * N < (int64_t(1) << 35) && ldg == N && (!U || ldu == N) && ldy == cols && (out_fmt == GR_OUT_16 || ld_sy == N / 32)) {
        a.N = M * N;
        a.M = 1;
    }
    if (out_fmt == GR_OUT_16) a.ldy_bytes = ldy * 2;
    hipStream_t h = static_cast<hipStream_t>(stream);
    return fmt == GR_FMT_BF16 ? run_gated<gr::ElemBF16>(a, out_fmt, h) : run_gated<gr::ElemF16>(a, out_fmt, h);
}

int gemm_w4_bt_workspace_size(int64_t M, int64_t N, int64_t K, int64_t* bytes) {
    if (!bytes) return GR_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 0 || K % 32 != 0) return GR_ERR_INVALID_DIM;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return GR_ERR_TOO_LARGE;
    *bytes = w4_workspace(M, N, K);
    return GR_OK;
}

int gemm_w4_bt(int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda, const uint8_t* Bt, int64_t ldbt,
               const uint8_t* scale_b, int64_t ld_sb, const uint16_t* bias, int act, uint16_t* C, int64_t ldc,
               int fmt, void* workspace, int64_t workspace_bytes, void* stream) {
    int st = validate_w4(M, N, K, A, lda, Bt, ldbt, scale_b, ld_sb, bias, act, C, ldc, fmt);
    if (st != GR_OK) return st;
    if (workspace_bytes < 0 || reinterpret_cast<uintptr_t>(workspace) % kWorkspaceAlign != 0) return GR_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return GR_OK;
    // (too small a workspace is none)
    const int64_t need = w4_workspace(M, N, K);
    const W4Plan p = w4_plan(M, N, K, workspace && workspace_bytes >= need);
    if (p.splits > 1) {
        const Region ws{reinterpret_cast<uintptr_t>(workspace), need};
        if (overlaps(ws, matrix16(C, M, N, ldc)) || overlaps(ws, matrix16(A, M, K, lda)) ||
            overlaps(ws, matrix8(Bt, N, K / 2, ldbt)) || overlaps(ws, matrix8(scale_b, N, K / 32, ld_sb)) ||
            overlaps(ws, matrix16(bias, 1, N, N)))
            return GR_ERR_ALIAS;
    }
    st = check_device();
    if (st != GR_OK) return st;
    const gr::w4::LinearArgs a{A,   Bt,    scale_b, bias, C,   M, N, K, lda, ldbt, ld_sb, ldc, act, 1,
                               p.splits > 1 ? static_cast<float*>(workspace) : nullptr, 0, 0};
    hipStream_t h = static_cast<hipStream_t>(stream);
    return fmt == GR_FMT_BF16 ? run_w4<gr::ElemBF16>(a, p, h) : run_w4<gr::ElemF16>(a, p, h);
}

int gemm_mxfp4_linear_bt(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const uint8_t* scale_a,
                         int64_t ld_sa, const uint8_t* Bt, int64_t ldbt, const uint8_t* scale_b, int64_t ld_sb,
                         const uint16_t* bias, int act, uint16_t* C, int64_t ldc, int fmt, void* stream) {
    gr_plan_t plan;
    int st = gemm_mxfp4_bt_plan(M, N, K, A, lda, scale_a, ld_sa, Bt, ldbt, scale_b, ld_sb, bias, act, C, ldc, fmt, &plan);
    if (st != GR_OK) return st;
    if (M == 0 || N == 0) return GR_OK;
    if (!fp4_streams(M, N, K, ldbt, ld_sb, plan.path))
        return gemm_mxfp4_bt(M, N, K, A, lda, scale_a, ld_sa, Bt, ldbt, scale_b, ld_sb, bias, act, C, ldc, fmt, stream);
    st = validate_w4(M, N, K, nullptr, K > 1 ? K : 1, Bt, ldbt, scale_b, ld_sb, bias, act, C, ldc, fmt, false);
    if (st != GR_OK) return st;
    if (lda < (K > 1 ? K / 2 : 1) || ld_sa < (K > 1 ? K / 32 : 1)) return GR_ERR_INVALID_LD;
    if (M == 0 || N == 0) return GR_OK;
    if (K > 0 && (!A || !scale_a)) return GR_ERR_NULL_PTR;
    const Region c = matrix16(C, M, N, ldc), a = matrix8(A, M, K / 2, lda), s = matrix8(scale_a, M, K / 32, ld_sa);
    if (a.bytes < 0 || s.bytes < 0) return GR_ERR_TOO_LARGE;
    if (overlaps(c, a) || overlaps(c, s)) return GR_ERR_ALIAS;
    st = check_device();
    if (st != GR_OK) return st;
    const gr::w4::Fp4Args args{A, scale_a, Bt, scale_b, bias, C, M, N, K, lda, ld_sa, ldbt, ld_sb, ldc, act, 1};
    hipStream_t h = static_cast<hipStream_t>(stream);
    return fmt == GR_FMT_BF16 ? run_fp4<gr::ElemBF16>(args, h) : run_fp4<gr::ElemF16>(args, h);
}

int moe_route_workspace_size(int64_t T, int64_t H, int64_t E, int64_t* bytes) {
    if (!bytes) return GR_ERR_INVALID_ARG;
    if (T < 0 || H < 0 || E < 1) return GR_ERR_INVALID_DIM;
    if (T > kMaxDim || H > kMaxDim || E > gr::w4::kMaxExperts) return GR_ERR_TOO_LARGE;
    *bytes = route_workspace(T, H, E);
    return GR_OK;
}

int moe_route(int64_t T, int64_t H, int64_t E, int64_t topk, const uint16_t* X, int64_t ldx, const uint16_t* Wr,
              int64_t ldwr, const float* bias, int renorm, int32_t* ids, float* weights, int fmt, void* workspace,
              int64_t workspace_bytes, void* stream) {
    if (T < 0 || H < 0 || E < 1) return GR_ERR_INVALID_DIM;
    if (topk < 1 || topk > E || !known_fmt(fmt) || (renorm != 0 && renorm != 1) || workspace_bytes < 0)
        return GR_ERR_INVALID_ARG;
    if (T > kMaxDim || H > kMaxDim || E > gr::w4::kMaxExperts || topk > gr::w4::kMaxTopK) return GR_ERR_TOO_LARGE;
    const int64_t hmin = H > 1 ? H : 1;
    if (ldx < hmin || ldwr < hmin) return GR_ERR_INVALID_LD;
    if (T == 0) return GR_OK;
    if (!ids || !weights || (H > 0 && (!X || !Wr))) return GR_ERR_NULL_PTR;
    if (reinterpret_cast<uintptr_t>(workspace) % kWorkspaceAlign != 0) return GR_ERR_INVALID_ARG;
    // (too small a workspace is none, as for the products)
    int64_t need = route_workspace(T, H, E);
    if (!workspace || workspace_bytes < need) need = 0;
    const Region x = matrix16(X, T, H, ldx), w = matrix16(Wr, E, H, ldwr),
                 b{reinterpret_cast<uintptr_t>(bias), bias ? E * 4 : 0}, i{reinterpret_cast<uintptr_t>(ids), T * topk * 4},
                 v{reinterpret_cast<uintptr_t>(weights), T * topk * 4},
                 s{reinterpret_cast<uintptr_t>(workspace), need};
    if (x.bytes < 0 || w.bytes < 0) return GR_ERR_TOO_LARGE;
    if (overlaps(i, v) || overlaps(i, x) || overlaps(i, w) || overlaps(i, b) || overlaps(v, x) || overlaps(v, w) ||
        overlaps(v, b) || overlaps(s, x) || overlaps(s, w) || overlaps(s, b) || overlaps(s, i) || overlaps(s, v))
        return GR_ERR_ALIAS;
    int st = check_device();
    if (st != GR_OK) return st;
    const gr::w4::RouteArgs a{X,   Wr,  bias,   ids,       weights, T,
                              H,   ldx, ldwr,   (int)E,    (int)topk, renorm,
                              need > 0 ? static_cast<float*>(workspace) : nullptr};
    hipStream_t h = static_cast<hipStream_t>(stream);
    return fmt == GR_FMT_BF16 ? run_route<gr::ElemBF16>(a, h) : run_route<gr::ElemF16>(a, h);
}

int moe_w4_workspace_size(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk, int64_t* bytes) {
    if (!bytes) return GR_ERR_INVALID_ARG;
    const int st = validate_moe_dims(T, H, I, E, topk);
    if (st != GR_OK) return st;
    *bytes = moe_workspace(T, H, I, topk);
    return GR_OK;
}

int moe_w4(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk, const uint16_t* X, int64_t ldx,
           const int32_t* ids, const float* weights, const uint8_t* W13, const uint8_t* S13, const uint16_t* b13,
           const uint8_t* W2, const uint8_t* S2, const uint16_t* b2, int act, uint16_t* C, int64_t ldc, int fmt,
           void* workspace, int64_t workspace_bytes, void* stream) {
    int st = validate_moe_dims(T, H, I, E, topk);
    if (st != GR_OK) return st;
    const int64_t hmin = H > 1 ? H : 1;
    if (ldx < hmin || ldc < hmin) return GR_ERR_INVALID_LD;
    if (!known_act(act) || !known_fmt(fmt) || workspace_bytes < 0) return GR_ERR_INVALID_ARG;
    if (T == 0 || H == 0) return GR_OK;
    if (!C || !ids || !weights || (I > 0 && (!X || !W13 || !S13 || !W2 || !S2))) return GR_ERR_NULL_PTR;
    const int64_t need = moe_workspace(T, H, I, topk);
    if (need > 0 && !workspace) return GR_ERR_NULL_PTR;
    if (reinterpret_cast<uintptr_t>(workspace) % kWorkspaceAlign != 0) return GR_ERR_INVALID_ARG;
    if (workspace_bytes < need) return GR_ERR_SCRATCH;
    const Region x = matrix16(X, T, H, ldx), c = matrix16(C, T, H, ldc),
                 ws{reinterpret_cast<uintptr_t>(workspace), need};
    if (x.bytes < 0 || c.bytes < 0) return GR_ERR_TOO_LARGE;
    const Region in[] = {x,
                         {reinterpret_cast<uintptr_t>(ids), T * topk * 4},
                         {reinterpret_cast<uintptr_t>(weights), T * topk * 4},
                         {reinterpret_cast<uintptr_t>(W13), E * I * H},
                         {reinterpret_cast<uintptr_t>(S13), E * I * H / 16},
                         {reinterpret_cast<uintptr_t>(W2), E * I * H / 2},
                         {reinterpret_cast<uintptr_t>(S2), E * I * H / 32},
                         {reinterpret_cast<uintptr_t>(b13), b13 ? E * I * 4 : 0},
                         {reinterpret_cast<uintptr_t>(b2), b2 ? E * H * 2 : 0}};
    if (overlaps(c, ws)) return GR_ERR_ALIAS;
    for (const Region& r : in)
        if (overlaps(c, r) || overlaps(ws, r)) return GR_ERR_ALIAS;
    st = check_device();
    if (st != GR_OK) return st;
    uint8_t* const at = static_cast<uint8_t*>(workspace);
    const gr::w4::MoeArgs a{X,
                            ids,
                            weights,
                            W13,
                            S13,
                            W2,
                            S2,
                            b13,
                            b2,
                            reinterpret_cast<uint16_t*>(at),
                            reinterpret_cast<float*>(at + moe_h_bytes(T, I, topk)),
                            reinterpret_cast<int32_t*>(at + moe_h_bytes(T, I, topk) + moe_y_bytes(T, H, topk)),
                            C,
                            T,
                            H,
                            I,
                            ldx,
                            ldc,
                            (int)E,
                            (int)topk,
                            act,
                            1,
                            1};
    hipStream_t h = static_cast<hipStream_t>(stream);
    return fmt == GR_FMT_BF16 ? run_moe<gr::ElemBF16>(a, h) : run_moe<gr::ElemF16>(a, h);
}

}  // extern "C"
