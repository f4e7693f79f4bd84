// Host side of the sandwich norm with its gradients and of the orthogonalised update.
// See include/gemm_relu.h.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/gemm_relu.h"
#include "own_products.hpp"
#include "ortho_fold_kernel.hpp"
#include "ortho_small_kernel.hpp"
#include "sandwich_kernel.hpp"

namespace {

constexpr int64_t kCus = 256;
constexpr int64_t kOrthoMax = 65536;  // either side of an update

// ---- sandwich norm ----------------------------------------------------------------------

// f<TPR, C>() for rows of N columns: threads per row and chunks of 8 columns per thread.
// `WIDE` (the backward pass, which needs the registers): one chunk as far as it goes.  Else two
// from 2048 columns on and half as many threads, so that a CU holds more rows (forward, 8192 x 8192:
// 93 us, 98 with one chunk; 64 x 8192 4.1 and 4.2, 1 x 4096 3.1 and 2.9).
template <bool WIDE, typename F>
int by_width(int64_t N, F&& f) {
    using std::integral_constant;
#define GR_CASE(TPR, C) return f(integral_constant<int, TPR>{}, integral_constant<int, C>{})
    if (N <= 512) GR_CASE(64, 1);
    if (N <= 1024) GR_CASE(128, 1);
    if (N <= 2048) GR_CASE(256, 1);
    if constexpr (WIDE) {
        if (N <= 4096) GR_CASE(512, 1);
        if (N <= 8192) GR_CASE(1024, 1);
    } else {
        if (N <= 4096) GR_CASE(256, 2);
        if (N <= 8192) GR_CASE(512, 2);
    }
    if (N <= 16384) GR_CASE(1024, 2);
    GR_CASE(1024, 4);
#undef GR_CASE
}

int check_sandwich(int64_t M, int64_t N, int64_t G, bool gate, float scale, float eps, int fmt) {
    const int dims = check_dims({M, N, G});
    if (dims != GR_OK) return dims;
    if (gate ? G < 1 || M % G != 0 : G != 0) return GR_ERR_INVALID_DIM;
    if (!known_fmt(fmt) || !std::isfinite(scale) || !std::isfinite(eps) || eps < 0.0f) return GR_ERR_INVALID_ARG;
    return N > gr::sandwich::MAX_N ? GR_ERR_TOO_LARGE : GR_OK;
}

template <typename E>
int run_sandwich(const gr::sandwich::Args& a, hipStream_t stream) {
    return by_width<false>(a.N, [&](auto tpr, auto c) {
        constexpr int TPR = decltype(tpr)::value, C = decltype(c)::value;
        using namespace gr::sandwich;
        // (a launch takes less than 2^32 threads)
        constexpr int64_t most = (int64_t(1) << 20) * rows_at_once(TPR);
        const int threads = threads_for(TPR);
        int st = GR_OK;
        for (int64_t first = 0; st == GR_OK && first < a.M; first += most) {
            Args part = a;
            part.first = first;
            const int64_t rows = a.M - first < most ? a.M - first : most, grid = ceil_div(rows, rows_at_once(TPR));
            st = a.N % 8 == 0 ? launch(forward_kernel<E, TPR, C, true>, grid, threads, stream, part)
                              : launch(forward_kernel<E, TPR, C, false>, grid, threads, stream, part);
        }
        return st;
    });
}

// How the rows are dealt out: slots (each with a partial sum of every column), and
// how many of them share a gate's rows (0: a slot has whole gates).  As many workgroups as
// the chip holds of 512 threads (of 1024: half as many), four rows or more to a slot where there are that
// many.
struct Deal {
    int64_t slots, split;
};
Deal deal(int64_t M, int64_t N, int64_t groups) {
    if (M == 0) return {0, 1};
    const int64_t rows = M / groups, most = N <= 512 ? 8 * kCus : N <= 4096 ? 2 * kCus : kCus;
    if (groups > most) return {most, 0};
    int64_t split = most / groups;
    if (split > ceil_div(rows, 4)) split = ceil_div(rows, 4);
    return {groups * split, split};
}

int64_t sandwich_need(int64_t M, int64_t N, int64_t G) { return aligned(deal(M, N, G > 0 ? G : 1).slots * 2 * N * 4); }

template <typename E>
int run_sandwich_backward(const gr::sandwich::BwdArgs& a, hipStream_t stream) {
    using namespace gr::sandwich;
    int st = GR_OK;
    if (a.slots > 0)
        st = by_width<true>(a.N, [&](auto tpr, auto c) {
            constexpr int TPR = decltype(tpr)::value, C = decltype(c)::value;
            const int64_t grid = ceil_div(a.slots, rows_at_once(TPR));
            const int threads = threads_for(TPR);
            if (a.N % 8 == 0)
                return a.split > 0 ? launch(backward_kernel<E, TPR, C, true, true>, grid, threads, stream, a)
                                   : launch(backward_kernel<E, TPR, C, false, true>, grid, threads, stream, a);
            return a.split > 0 ? launch(backward_kernel<E, TPR, C, true, false>, grid, threads, stream, a)
                               : launch(backward_kernel<E, TPR, C, false, false>, grid, threads, stream, a);
        });
    // (not by the partial sums' address: without rows there are none, and the sums are zeros)
    if (st != GR_OK || !(a.dw || a.dnext_w || a.dgate)) return st;
    return launch_grid(reduce_kernel<E>, dim3((uint32_t)ceil_div(a.N, REDUCE_COLS), 2), 256, stream, a);
}

// ---- orthogonalised update ----------------------------------------------------------------

struct OrthoLayout {
    bool tall;
    int64_t r, c;    // narrow and wide side
    int64_t rp, cp;  // padded
    int64_t parts, x, a;  // bytes: partial sums, one of the four X buffers, one of A and B
    bool small;           // in one workgroup's LDS, without a workspace
    bool fold;            // two launches a step: no X^T, no B
    int64_t total() const { return small ? 0 : fold ? parts + 2 * x + a : parts + 4 * x + 2 * a; }
};

OrthoLayout ortho_layout(int64_t B, int64_t rows, int64_t cols) {
    OrthoLayout l;
    l.tall = rows > cols;
    l.r = l.tall ? cols : rows;
    l.c = l.tall ? rows : cols;
    l.rp = round_up(l.r, 64);
    l.cp = round_up(l.c, 64);
    l.parts = aligned(B * gr::ortho::PARTS * 8);
    l.x = aligned(B * l.rp * l.cp * 2);
    l.a = aligned(B * l.rp * l.rp * 2);
    l.small = l.rp <= gr::ortho::SMALL_R && 2 * l.rp * (l.rp + l.cp) <= gr::ortho::SMALL_LDS;
    l.fold = !l.small && l.rp <= gr::ortho::FOLD_R;
    return l;
}

template <typename In>
int ortho_prepare(const gr::ortho::PrepArgs& a, int64_t B, hipStream_t stream) {
    using namespace gr::ortho;
    int st = launch_grid(square_sum_kernel<In>, dim3(PARTS, (uint32_t)B), 256, stream, a);
    if (st != GR_OK) return st;
    const uint32_t tc = (uint32_t)(a.cols_pad / gr::train::TILE);
    return launch_grid(normalise_kernel<In>, dim3((uint32_t)(a.rows_pad / gr::train::TILE) * tc, (uint32_t)B), 256, stream, a,
                       tc);
}

template <typename In>
int run_small(const OrthoLayout& l, int64_t B, const gr::ortho::SmallArgs& a, hipStream_t stream) {
    using namespace gr::ortho;
    return l.rp <= 64 ? launch(small_kernel<In, 64>, B, SMALL_THREADS, stream, a)
                      : launch(small_kernel<In, 128>, B, SMALL_THREADS, stream, a);
}

// Workgroups that walk over a matrix's blocks of columns: as many as the chip holds for all of the matrices.
template <int RP>
int run_fold_step(gr::ortho::FoldTo to, const OrthoLayout& l, int64_t B, const gr::ortho::FoldArgs& a, hipStream_t stream) {
    using namespace gr::ortho;
    const int64_t held = kCus * (FOLD_R / RP), blocks = l.cp / FOLD_COLS;
    const dim3 grid((uint32_t)std::min(blocks, std::max<int64_t>(1, held / B)), (uint32_t)B);
    if (to == kNextX) return launch_grid(fold_kernel<RP, kNextX>, grid, 2 * RP, stream, a);
    if (to == kResult) return launch_grid(fold_kernel<RP, kResult>, grid, 2 * RP, stream, a);
    return launch_grid(fold_kernel<RP, kResultTall>, grid, 2 * RP, stream, a);
}

int run_fold(const OrthoLayout& l, int64_t B, int64_t rows, int64_t cols, const float (&k)[3], int steps, float scale, uint16_t* out,
             int64_t ldo, int64_t batch_o, uint16_t* const (&x)[2], uint16_t* d, hipStream_t stream) {
    using namespace gr::ortho;
    const int64_t rp = l.rp, cp = l.cp, bx = rp * cp, ba = rp * rp;
    for (int s = 0; s < steps; ++s) {
        const gr::own::PolyArgs p{nullptr, d, 0, rp, SCALE_A / (SCALE_X * SCALE_X), 0.0f, -SCALE_A, bx, bx, ba, 0, ba};
        int st = symmetric<ElemF16>(B, rp, cp, x[s % 2], cp, d, rp, p, stream);
        if (st != GR_OK) return st;
        const FoldTo to = s + 1 < steps ? kNextX : l.tall ? kResultTall : kResult;
        const FoldArgs a{x[s % 2], d, to == kNextX ? x[(s + 1) % 2] : out, rows, cols, ldo, batch_o, (uint32_t)cp, k[2],
                         k[1] + 2.0f * k[2], k[0] + k[1] + k[2], scale};
        st = rp <= 64    ? run_fold_step<64>(to, l, B, a, stream)
             : rp <= 128 ? run_fold_step<128>(to, l, B, a, stream)
             : rp <= 192 ? run_fold_step<192>(to, l, B, a, stream)
                         : run_fold_step<256>(to, l, B, a, stream);
        if (st != GR_OK) return st;
    }
    return GR_OK;
}

template <typename Out>
int run_ortho(const OrthoLayout& l, int64_t B, const float (&k)[3], int steps, float scale, uint16_t* out, int64_t ldo,
              int64_t batch_o, uint16_t* const (&x)[2], uint16_t* const (&xt)[2], uint16_t* a, uint16_t* b,
              hipStream_t stream) {
    using namespace gr::own;
    using gr::ortho::SCALE_A;
    using gr::ortho::SCALE_X;
    using Half = ElemF16;
    const float all = k[0] + k[1] + k[2];
    const int64_t rp = l.rp, cp = l.cp, bx = rp * cp, ba = rp * rp;
    for (int s = 0; s < steps; ++s) {
        const uint16_t *X = x[s % 2], *Xt = xt[s % 2];
        PolyArgs p{nullptr, a, 0, rp, SCALE_A / (SCALE_X * SCALE_X), 0.0f, 0.0f, bx, bx, ba, 0, ba};
        int st = symmetric<Half>(B, rp, cp, X, cp, a, rp, p, stream);
        if (st != GR_OK) return st;
        p = PolyArgs{a, b, rp, rp, k[2] / SCALE_A, k[1], -SCALE_A * (k[1] + k[2]), ba, ba, ba, ba, ba};
        st = symmetric<Half>(B, rp, rp, a, rp, b, rp, p, stream);
        if (st != GR_OK) return st;
        if (s + 1 < steps) {
            p = PolyArgs{X, xt[(s + 1) % 2], cp, rp, 1.0f / SCALE_A, all, 0.0f, ba, bx, bx, bx, bx};
            st = batched<Poly<Half, Half, false>>(B, rp, cp, rp, b, rp, Xt, rp, x[(s + 1) % 2], cp, p, stream);
        } else if (!l.tall) {
            p = PolyArgs{X, nullptr, cp, 0, scale / (SCALE_A * SCALE_X), scale * all / SCALE_X, 0.0f, ba, bx, batch_o, bx, 0};
            st = batched<Poly<Half, Out, false>>(B, l.r, l.c, rp, b, rp, Xt, rp, out, ldo, p, stream);
        } else {
            p = PolyArgs{Xt, nullptr, rp, 0, scale / (SCALE_A * SCALE_X), scale * all / SCALE_X, 0.0f, bx, ba, batch_o, bx, 0};
            st = batched<Poly<Half, Out, false>>(B, l.c, l.r, rp, Xt, rp, b, rp, out, ldo, p, stream);
        }
        if (st != GR_OK) return st;
    }
    return GR_OK;
}

}  // namespace

extern "C" {

int sandwich_norm_fwd(int64_t M, int64_t N, const uint16_t* Y, int64_t ldy, const uint16_t* R, int64_t ldr, const uint16_t* w,
                      const uint16_t* next_w, const uint16_t* gate, int64_t G, int64_t ld_gate, float scale, float eps,
                      uint16_t* total, int64_t ldt, uint16_t* normed, int64_t ldn, int fmt, void* stream) {
    int st = check_sandwich(M, N, G, gate != nullptr, scale, eps, fmt);
    if (st != GR_OK) return st;
    if (ldy < least(N) || ldr < least(N) || ldt < least(N) || (normed && ldn < least(N)) || (gate && ld_gate < least(N)))
        return GR_ERR_INVALID_LD;
    if (M == 0 || N == 0) return GR_OK;
    if (!Y || !R || !total) return GR_ERR_NULL_PTR;
    const Region y = matrix(Y, M, N, ldy), r = matrix(R, M, N, ldr), t = matrix(total, M, N, ldt),
                 n = matrix(normed, M, N, ldn);
    // a row is read whole before it is written: an output may lie on an input
    const bool t_on_y = total == Y && ldt == ldy, t_on_r = total == R && ldt == ldr;
    const bool n_on_y = normed == Y && ldn == ldy, n_on_r = normed == R && ldn == ldr;
    const Region none{0, 0};
    const Region t_only[] = {t}, n_only[] = {n};
    const Region t_read[] = {t_on_y ? none : y, t_on_r ? none : r, n, vector(w, N), vector(next_w, N), matrix(gate, G, N, ld_gate)};
    const Region n_read[] = {n_on_y ? none : y, n_on_r ? none : r, vector(w, N), vector(next_w, N), matrix(gate, G, N, ld_gate)};
    st = check_regions(t_only, t_read);
    if (st == GR_OK) st = check_regions(n_only, n_read);
    if (st == GR_OK) st = check_device();
    if (st != GR_OK) return st;
    const gr::sandwich::Args a{Y, R, w, next_w, gate, total, normed, M, N, ldy, ldr, ldt, ldn, ld_gate, gate ? M / G : 1, scale, eps, 0};
    hipStream_t h = static_cast<hipStream_t>(stream);
    return fmt == GR_FMT_BF16 ? run_sandwich<ElemBF16>(a, h) : run_sandwich<ElemF16>(a, h);
}

int sandwich_norm_bwd_workspace_size(int64_t M, int64_t N, int64_t G, int64_t* bytes) {
    if (!bytes) return GR_ERR_INVALID_ARG;
    const int st = check_sandwich(M, N, G, G > 0, 1.0f, 0.0f, GR_FMT_BF16);
    if (st != GR_OK) return st;
    *bytes = sandwich_need(M, N, G);
    return GR_OK;
}

int sandwich_norm_bwd(int64_t M, int64_t N, const uint16_t* dT, int64_t ld_dt, const uint16_t* dN, int64_t ld_dn,
                      const uint16_t* Y, int64_t ldy, const uint16_t* T, int64_t ldt, const uint16_t* w,
                      const uint16_t* next_w, const uint16_t* gate, int64_t G, int64_t ld_gate, float scale, float eps,
                      uint16_t* dY, int64_t ld_dy, uint16_t* dR, int64_t ld_dr, uint16_t* dw, uint16_t* dnext_w,
                      uint16_t* dgate, int64_t ld_dgate, int fmt, void* workspace, int64_t workspace_bytes, void* stream) {
    int st = check_sandwich(M, N, G, gate != nullptr, scale, eps, fmt);
    if (st != GR_OK) return st;
    const int64_t low = least(N);
    if (ldy < low || ldt < low || ld_dy < low || ld_dr < low || (dT && ld_dt < low) || (dN && ld_dn < low) ||
        (gate && ld_gate < low) || (dgate && ld_dgate < low))
        return GR_ERR_INVALID_LD;
    if ((dgate && !gate) || (dnext_w && !dN && M > 0)) return GR_ERR_INVALID_ARG;
    if (N == 0) return GR_OK;
    if (M > 0 && (!Y || !T || !dY || !dR || (!dT && !dN))) return GR_ERR_NULL_PTR;
    const bool sums = dw || dnext_w || dgate;
    if (M == 0 && !sums) return GR_OK;
    const int64_t need = sums ? sandwich_need(M, N, G) : 0;
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != GR_OK) return st;
    const Region written[] = {matrix(dY, M, N, ld_dy), matrix(dR, M, N, ld_dr), vector(dw, N), vector(dnext_w, N),
                              matrix(dgate, G, N, ld_dgate), {reinterpret_cast<uintptr_t>(workspace), need}};
    const Region read[] = {matrix(dT, M, N, ld_dt), matrix(dN, M, N, ld_dn), matrix(Y, M, N, ldy), matrix(T, M, N, ldt),
                           vector(w, N), vector(next_w, N), matrix(gate, G, N, ld_gate)};
    st = check_regions(written, read);
    if (st == GR_OK) st = check_device();
    if (st != GR_OK) return st;
    const int64_t groups = gate ? G : 1;
    const Deal d = deal(M, N, groups);
    // (without sums a workspace is not needed: the partial sums are not written)
    const gr::sandwich::BwdArgs a{dT, dN, Y, T, w, next_w, gate, dY, dR, dw, dnext_w, dgate,
                                  sums ? static_cast<float*>(workspace) : nullptr, M, N, ld_dt, ld_dn, ldy, ldt, ld_dy, ld_dr,
                                  ld_gate, ld_dgate, M / groups, groups, d.split, d.slots, scale, eps};
    hipStream_t h = static_cast<hipStream_t>(stream);
    return fmt == GR_FMT_BF16 ? run_sandwich_backward<ElemBF16>(a, h) : run_sandwich_backward<ElemF16>(a, h);
}

int orthogonalize_workspace_size(int64_t B, int64_t rows, int64_t cols, int64_t* bytes) {
    if (!bytes) return GR_ERR_INVALID_ARG;
    const int dims = check_dims({B, rows, cols});
    if (dims != GR_OK) return dims;
    if (B > 65535 || rows > kOrthoMax || cols > kOrthoMax) return GR_ERR_TOO_LARGE;
    *bytes = B > 0 && rows > 0 && cols > 0 ? ortho_layout(B, rows, cols).total() : 0;
    return GR_OK;
}

int orthogonalize_update(int64_t B, int64_t rows, int64_t cols, const void* G, int64_t ldg, int64_t batch_g, int g_fmt,
                         const float* coefficients, int steps, float scale, float eps, uint16_t* out, int64_t ldo,
                         int64_t batch_o, void* workspace, int64_t workspace_bytes, void* stream) {
    const int dims = check_dims({B, rows, cols});
    if (dims != GR_OK) return dims;
    if (B > 65535 || rows > kOrthoMax || cols > kOrthoMax) return GR_ERR_TOO_LARGE;
    if (ldg < least(cols) || ldo < least(cols)) return GR_ERR_INVALID_LD;
    if ((!known_fmt(g_fmt) && g_fmt != GR_FMT_F32) || !coefficients || steps < 1 || steps > 64 || !std::isfinite(scale) ||
        !std::isfinite(eps) || eps < 0.0f)
        return GR_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
        if (!std::isfinite(coefficients[i])) return GR_ERR_INVALID_ARG;
    if (B == 0 || rows == 0 || cols == 0) return GR_OK;
    if (!G || !out) return GR_ERR_NULL_PTR;
    const int64_t size = g_fmt == GR_FMT_F32 ? 2 : 1;
    const int64_t span_o = span_bytes(rows, cols, ldo);
    int64_t span_g = span_bytes(rows, cols, ldg);
    if (span_g < 0 || span_o < 0) return GR_ERR_TOO_LARGE;
    span_g *= size;
    if (B > 1 && (batch_g < span_g / (2 * size) || batch_o < span_o / 2)) return GR_ERR_INVALID_LD;
    if (B > 1 && (batch_g > kMaxSpanBytes / (8 * B) || batch_o > kMaxSpanBytes / (8 * B))) return GR_ERR_TOO_LARGE;
    const OrthoLayout l = ortho_layout(B, rows, cols);
    int st = check_workspace(workspace, workspace_bytes, l.total());
    if (st != GR_OK) return st;
    const Region written[] = {{reinterpret_cast<uintptr_t>(out), (B - 1) * batch_o * 2 + span_o},
                              {reinterpret_cast<uintptr_t>(workspace), l.total()}};
    const Region read[] = {{reinterpret_cast<uintptr_t>(G), (B - 1) * batch_g * 2 * size + span_g}};
    st = check_regions(written, read);
    if (st == GR_OK) st = check_device();
    if (st != GR_OK) return st;
    hipStream_t h = static_cast<hipStream_t>(stream);
    const float k[3] = {coefficients[0], coefficients[1], coefficients[2]};
    if (l.small) {
        const gr::ortho::SmallArgs a{G, out, rows, cols, ldg, batch_g, ldo, batch_o, (uint32_t)l.cp, l.tall ? 1 : 0, steps,
                                     k[1], k[2], k[0] + k[1] + k[2], scale, eps};
        return g_fmt == GR_FMT_F32    ? run_small<gr::ortho::ElemF32>(l, B, a, h)
               : g_fmt == GR_FMT_BF16 ? run_small<ElemBF16>(l, B, a, h)
                                      : run_small<ElemF16>(l, B, a, h);
    }
    uint8_t* at = static_cast<uint8_t*>(workspace);
    auto take = [&](int64_t bytes) {
        uint16_t* const p = reinterpret_cast<uint16_t*>(at);
        at += bytes;
        return p;
    };
    double* const part = reinterpret_cast<double*>(take(l.parts));
    uint16_t* const x[2] = {take(l.x), take(l.x)};
    uint16_t* const a = take(l.a);
    // (not there where the steps are folded)
    uint16_t* const xt[2] = {l.fold ? nullptr : take(l.x), l.fold ? nullptr : take(l.x)};
    uint16_t* const b = l.fold ? nullptr : take(l.a);
    const int64_t rows_pad = l.tall ? l.cp : l.rp, cols_pad = l.tall ? l.rp : l.cp;
    const gr::ortho::PrepArgs prep{G,        rows,     cols,         ldg, batch_g, part, l.tall ? xt[0] : x[0], l.tall ? x[0] : xt[0],
                                   rows_pad, cols_pad, l.rp * l.cp, eps};
    st = g_fmt == GR_FMT_F32    ? ortho_prepare<gr::ortho::ElemF32>(prep, B, h)
         : g_fmt == GR_FMT_BF16 ? ortho_prepare<ElemBF16>(prep, B, h)
                                : ortho_prepare<ElemF16>(prep, B, h);
    if (st != GR_OK) return st;
    if (l.fold) return run_fold(l, B, rows, cols, k, steps, scale, out, ldo, batch_o, x, a, h);
    return run_ortho<ElemBF16>(l, B, k, steps, scale, out, ldo, batch_o, x, xt, a, b, h);
}

}  // extern "C"
