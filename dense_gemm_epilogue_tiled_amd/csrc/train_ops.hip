// Host side of the products of training: the gated linear layer and the gradients of
// linear layers.  See include/gemm_relu.h.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gemm_relu.h"
#include "own_products.hpp"
#include "tile3_kernel.hpp"
#include "train_kernel.hpp"

namespace {

gr::train::Job job(const uint16_t* src, int64_t rows, int64_t cols, int64_t lds, uint16_t* dst, int64_t ldd, int64_t pad,
                   bool transposed) {
    using gr::train::TILE;
    const int64_t tr = ceil_div(transposed ? pad : rows, TILE), tc = ceil_div(transposed ? cols : pad, TILE);
    return {src, dst, rows, cols, lds, ldd, pad, (uint32_t)(tc > 0 ? tc : 1), (uint32_t)(tr * tc)};
}
const gr::train::Job kNoJob{nullptr, nullptr, 0, 0, 0, 0, 0, 1, 0};

template <bool TRANSPOSED>
int relayout(const gr::train::Job& a, const gr::train::Job& b, hipStream_t stream) {
    if (a.tiles + b.tiles == 0) return GR_OK;
    return launch(gr::train::relayout_kernel<TRANSPOSED>, (int64_t)a.tiles + b.tiles, gr::train::THREADS, stream, a, b);
}

// ---- the gated linear layer -----------------------------------------------------------

constexpr int kSmallMRows = 16;

// K that is not a whole number of 32-deep steps (0 included): x and the weight are
// copied into the workspace with K padded by zeros.
bool gated_packs(int64_t H) { return H % 32 != 0 || H == 0; }
int64_t gated_pitch(int64_t H) { return H > 0 ? round_up(H, 64) : 64; }

int64_t gated_need(int64_t M, int64_t I, int64_t H) {
    if (M == 0 || I == 0 || !gated_packs(H)) return 0;
    return aligned(M * gated_pitch(H) * 2) + aligned(2 * I * gated_pitch(H) * 2);
}

template <typename Base>
int run_gated(int64_t M, int64_t I, int64_t H, const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
              const gr::own::GatedArgs& ep, uint16_t* C, int64_t ldc, uint8_t* ws, hipStream_t stream) {
    using E = gr::own::Gated<Base>;
    int64_t K = H;
    if (gated_packs(H)) {
        K = gated_pitch(H);
        uint16_t* const xp = reinterpret_cast<uint16_t*>(ws);
        uint16_t* const wp = reinterpret_cast<uint16_t*>(ws + aligned(M * K * 2));
        const int st = relayout<false>(job(X, M, H, ldx, xp, K, K, false), job(W, 2 * I, H, ldw, wp, K, K, false), stream);
        if (st != GR_OK) return st;
        X = xp;
        W = wp;
        ldx = ldw = K;
    }
    if (M <= kSmallMRows && K % gr::smallm::BTS_KC == 0) {
        using namespace gr::smallm;
        constexpr int W4 = 4, cols = 8 * W4;
        const gr::own::GatedArgs args = ep;
        if (I % cols == 0)
            return launch(gemm_relu_smallm_bt_stream_kernel<false, E, W4, 16>, ceil_div(I, cols), 64 * W4, stream, X, W, C,
                          M, I, K, ldx, ldw, ldc, args);
        return launch(gemm_relu_smallm_bt_stream_kernel<true, E, W4, 16>, ceil_div(I, cols), 64 * W4, stream, X, W, C, M, I,
                      K, ldx, ldw, ldc, args);
    }
    return product<E>(choose(1, M, I, K, 2), 1, M, I, K, X, ldx, W, ldw, C, ldc, ep, stream);
}

// ---- gradients ------------------------------------------------------------------------

// dX = dY W with 256 x 256 tiles and no epilogue but the rounding; other shapes take
// gemm_bias_act's paths.
template <typename Base>
struct Bare : Base {
    static __device__ __forceinline__ uint16_t relu_round(float x) { return (uint16_t)gr::own::round2<Base>(x, x); }
};

bool input_grad_tiles(int64_t M, int64_t K, int64_t N, const uint16_t* dY, int64_t lddy, const uint16_t* W, int64_t ldw) {
    using namespace gr::tile3;
    return M >= BM && N > 0 && N % BKA == 0 && rows16(dY, lddy) && rows16(W, ldw) && lddy <= gr::tile2::MAX_LDA &&
           ldw <= gr::tile2::MAX_LDB && ceil_div(M, BM) * ceil_div(K, BN) > 128;
}

int input_grad_need(int64_t M, int64_t K, int64_t N, const uint16_t* dY, int64_t lddy, const uint16_t* W, int64_t ldw,
                    const uint16_t* dX, int64_t lddx, int64_t* bytes) {
    *bytes = 0;
    if (M == 0 || K == 0 || input_grad_tiles(M, K, N, dY, lddy, W, ldw)) return GR_OK;
    return gemm_relu_f16_workspace_size(M, K, N, dY, lddy, W, ldw, dX, lddx, bytes);
}

template <typename Base>
int input_grad(int64_t M, int64_t K, int64_t N, const uint16_t* dY, int64_t lddy, const uint16_t* W, int64_t ldw,
               uint16_t* dX, int64_t lddx, uint8_t* ws, int64_t ws_bytes, hipStream_t stream) {
    if (input_grad_tiles(M, K, N, dY, lddy, W, ldw)) {
        using namespace gr::tile3;
        using E = Bare<Base>;
        const uint32_t tm = (uint32_t)ceil_div(M, BM), tn = (uint32_t)ceil_div(K, BN);
        const int vec = 8;
        const gr::EpiArgs ep{nullptr, gr::kActNone, 1.0f};
        if (M % BM == 0 && K % BN == 0)
            return launch(gemm_relu_tile3_kernel<false, E>, (int64_t)tm * tn, THREADS, stream, dY, W, dX, M, K, N, lddy, ldw,
                          lddx, tm, tn, kGroupM, vec, ep);
        return launch(gemm_relu_tile3_kernel<true, E>, (int64_t)tm * tn, THREADS, stream, dY, W, dX, M, K, N, lddy, ldw,
                      lddx, tm, tn, kGroupM, vec, ep);
    }
    return gemm_bias_act_ws(M, K, N, dY, lddy, W, ldw, nullptr, GR_ACT_NONE, dX, lddx,
                            Base::kIsF16 ? GR_FMT_F16 : GR_FMT_BF16, ws_bytes > 0 ? ws : nullptr, ws_bytes, stream, -1);
}

// dW = dY^T X from the transposed operands (pitch Mp each).
template <typename Base>
int weight_grad(int64_t N, int64_t K, int64_t Mp, const uint16_t* dYt, const uint16_t* Xt, uint16_t* dW, int64_t lddw,
                hipStream_t stream) {
    return product<gr::own::Plain<Base>>(choose(1, N, K, Mp, 1), 1, N, K, Mp, dYt, Mp, Xt, Mp, dW, lddw, gr::own::PlainArgs{},
                                         stream);
}

template <typename Base>
int bias_grad(int64_t N, int64_t Mp, const uint16_t* dYt, uint16_t* dB, hipStream_t stream) {
    return launch(gr::train::row_sums_kernel<Base>, ceil_div(N, 4), gr::train::THREADS, stream, dYt, N, Mp, Mp, dB);
}

int64_t padded_tokens(int64_t M) { return M > 0 ? round_up(M, gr::train::PAD) : gr::train::PAD; }

// The parts of the workspace, in order; only those of the gradients that are asked for.
struct GradLayout {
    int64_t dyt, xt, dy, product;  // bytes: dY^T, X^T, dY (of the gated layer), what dX's product takes
    int64_t total() const { return dyt + xt + dy + product; }
};

int linear_layout(int64_t M, int64_t N, int64_t K, const uint16_t* dY, int64_t lddy, const uint16_t* W, int64_t ldw,
                  const uint16_t* dX, int64_t lddx, const uint16_t* dW, const uint16_t* dB, GradLayout* l) {
    const int64_t Mp = padded_tokens(M);
    l->dyt = (dW || dB) ? aligned(2 * N * Mp) : 0;
    l->xt = dW ? aligned(2 * K * Mp) : 0;
    l->dy = 0;
    l->product = 0;
    if (!dX) return GR_OK;
    const int st = input_grad_need(M, K, N, dY, lddy, W, ldw, dX, lddx, &l->product);
    l->product = aligned(l->product);
    return st;
}


int validate_linear_backward(int64_t M, int64_t N, int64_t K, const uint16_t* dY, int64_t lddy, const uint16_t* X, int64_t ldx,
                             const uint16_t* W, int64_t ldw, const uint16_t* dX, int64_t lddx, const uint16_t* dW,
                             int64_t lddw, const uint16_t* dB) {
    if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K)) return GR_ERR_INVALID_DIM;
    if (lddy < least(N)) return GR_ERR_INVALID_LD;
    if (dX && (ldw < least(K) || lddx < least(K))) return GR_ERR_INVALID_LD;
    if (dW && (ldx < least(K) || lddw < least(K))) return GR_ERR_INVALID_LD;
    if (M > 0 && N > 0 && !dY && (dX || dW || dB)) return GR_ERR_NULL_PTR;
    if (N > 0 && K > 0 && M > 0 && ((dX && !W) || (dW && !X))) return GR_ERR_NULL_PTR;
    if (padded_tokens(M) > kMaxPitch) return GR_ERR_TOO_LARGE;
    return GR_OK;
}

template <typename Base>
int run_linear_backward(int64_t M, int64_t N, int64_t K, const uint16_t* dY, int64_t lddy, const uint16_t* X, int64_t ldx,
                        const uint16_t* W, int64_t ldw, uint16_t* dX, int64_t lddx, uint16_t* dW, int64_t lddw, uint16_t* dB,
                        uint8_t* ws, const GradLayout& l, hipStream_t stream) {
    const int64_t Mp = padded_tokens(M);
    uint16_t* const dyt = reinterpret_cast<uint16_t*>(ws);
    uint16_t* const xt = reinterpret_cast<uint16_t*>(ws + l.dyt);
    int st = GR_OK;
    if (N > 0 && (dB || (dW && K > 0)))
        st = relayout<true>(job(dY, M, N, lddy, dyt, Mp, Mp, true), dW ? job(X, M, K, ldx, xt, Mp, Mp, true) : kNoJob,
                            stream);
    if (st == GR_OK && dW && N > 0 && K > 0) st = weight_grad<Base>(N, K, Mp, dyt, xt, dW, lddw, stream);
    if (st == GR_OK && dB && N > 0) st = bias_grad<Base>(N, Mp, dyt, dB, stream);
    if (st == GR_OK && dX && M > 0 && K > 0)
        st = input_grad<Base>(M, K, N, dY, lddy, W, ldw, dX, lddx, ws + l.dyt + l.xt, l.product, stream);
    return st;
}

int gated_layout(int64_t M, int64_t I, int64_t H, const uint16_t* W, int64_t ldw, const uint16_t* dX, int64_t lddx,
                 const uint16_t* dW, const uint16_t* dB, GradLayout* l) {
    const int64_t Mp = padded_tokens(M), ld = round_up(2 * I, 8);
    l->dyt = (dW || dB) ? aligned(4 * I * Mp) : 0;
    l->xt = dW ? aligned(2 * H * Mp) : 0;
    l->dy = aligned(2 * M * ld);
    l->product = 0;
    if (!dX) return GR_OK;
    // the gradient of the products lies in the workspace: an aligned address that is
    // nobody's stands for it
    const uint16_t* const place = reinterpret_cast<const uint16_t*>(uintptr_t(1) << 62);
    const int st = input_grad_need(M, H, 2 * I, place, ld, W, ldw, dX, lddx, &l->product);
    l->product = aligned(l->product);
    return st;
}

int validate_gated_backward(int64_t M, int64_t I, int64_t H, const uint16_t* dH, int64_t lddh, const uint16_t* X,
                            int64_t ldx, const uint16_t* W, int64_t ldw, const uint16_t* GU, int64_t ldgu,
                            const uint16_t* dX, int64_t lddx, const uint16_t* dW, int64_t lddw, const uint16_t* dB) {
    if (!dim_ok(M) || !dim_ok(I) || !dim_ok(2 * I) || !dim_ok(H)) return GR_ERR_INVALID_DIM;
    if (lddh < least(I) || ldgu < least(2 * I)) return GR_ERR_INVALID_LD;
    if (dX && (ldw < least(H) || lddx < least(H))) return GR_ERR_INVALID_LD;
    if (dW && (ldx < least(H) || lddw < least(H))) return GR_ERR_INVALID_LD;
    const bool any = dX || dW || dB;
    if (any && M > 0 && I > 0 && (!dH || !GU)) return GR_ERR_NULL_PTR;
    if (M > 0 && I > 0 && H > 0 && ((dX && !W) || (dW && !X))) return GR_ERR_NULL_PTR;
    if (padded_tokens(M) > kMaxPitch || 2 * I + 8 > kMaxPitch) return GR_ERR_TOO_LARGE;
    return GR_OK;
}

template <typename Base>
int run_gated_backward(int64_t M, int64_t I, int64_t H, const uint16_t* dH, int64_t lddh, const uint16_t* X, int64_t ldx,
                       const uint16_t* W, int64_t ldw, const uint16_t* GU, int64_t ldgu, int act, uint16_t* dX, int64_t lddx,
                       uint16_t* dW, int64_t lddw, uint16_t* dB, uint8_t* ws, const GradLayout& l, hipStream_t stream) {
    using namespace gr::train;
    const int64_t Mp = padded_tokens(M), ld = round_up(2 * I, 8);
    uint16_t* const dyt = reinterpret_cast<uint16_t*>(ws);
    uint16_t* const xt = reinterpret_cast<uint16_t*>(ws + l.dyt);
    uint16_t* const dgu = reinterpret_cast<uint16_t*>(ws + l.dyt + l.xt);
    int st = GR_OK;
    if (I > 0) {
        const GatedBwdArgs a{dH, GU, dgu, l.dyt > 0 ? dyt : nullptr, M, I, lddh, ldgu, ld, Mp, act};
        const uint32_t tc = (uint32_t)ceil_div(I, TILE);
        st = launch(gated_backward_kernel<Base>, Mp / TILE * tc, THREADS, stream, a, tc);
    }
    if (st == GR_OK && dW && I > 0 && H > 0) {
        st = relayout<true>(job(X, M, H, ldx, xt, Mp, Mp, true), kNoJob, stream);
        if (st == GR_OK) st = weight_grad<Base>(2 * I, H, Mp, dyt, xt, dW, lddw, stream);
    }
    if (st == GR_OK && dB && I > 0) st = bias_grad<Base>(2 * I, Mp, dyt, dB, stream);
    if (st == GR_OK && dX && M > 0 && H > 0)
        st = input_grad<Base>(M, H, 2 * I, dgu, ld, W, ldw, dX, lddx, ws + l.dyt + l.xt + l.dy, l.product, stream);
    return st;
}

}  // namespace

extern "C" {

int gated_linear_workspace_size(int64_t M, int64_t I, int64_t H, int64_t* bytes) {
    if (!bytes) return GR_ERR_INVALID_ARG;
    if (!dim_ok(M) || !dim_ok(I) || !dim_ok(2 * I) || !dim_ok(H)) return GR_ERR_INVALID_DIM;
    *bytes = gated_need(M, I, H);
    return GR_OK;
}

int gated_linear_bt(int64_t M, int64_t I, int64_t H, const uint16_t* X, int64_t ldx, const uint16_t* W13, int64_t ldw,
                    const uint16_t* b13, int act, uint16_t* C, int64_t ldc, uint16_t* GU, int64_t ldgu, int fmt,
                    void* workspace, int64_t workspace_bytes, void* stream) {
    if (!dim_ok(M) || !dim_ok(I) || !dim_ok(2 * I) || !dim_ok(H)) return GR_ERR_INVALID_DIM;
    if (ldx < least(H) || ldw < least(H) || ldc < least(I) || (GU && ldgu < least(2 * I))) return GR_ERR_INVALID_LD;
    if (!known_act(act) || !known_fmt(fmt)) return GR_ERR_INVALID_ARG;
    if (M == 0 || I == 0) return GR_OK;
    if (!C || (H > 0 && (!X || !W13))) return GR_ERR_NULL_PTR;
    if (ldx > kMaxPitch || ldw > kMaxPitch) return GR_ERR_TOO_LARGE;
    const int64_t need = gated_need(M, I, H);
    int st = check_workspace(workspace, workspace_bytes, need);
    if (st != GR_OK) return st;
    const Region written[] = {matrix(C, M, I, ldc), matrix(GU, M, 2 * I, ldgu), {reinterpret_cast<uintptr_t>(workspace), need}};
    const Region read[] = {matrix(X, M, H, ldx), matrix(W13, 2 * I, H, ldw), vector(b13, 2 * I)};
    st = check_regions(written, read);
    if (st != GR_OK) return st;
    st = check_device();
    if (st != GR_OK) return st;
    const gr::own::GatedArgs ep{b13, GU, ldgu, I, act};
    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    hipStream_t h = static_cast<hipStream_t>(stream);
    return fmt == GR_FMT_BF16 ? run_gated<ElemBF16>(M, I, H, X, ldx, W13, ldw, ep, C, ldc, ws, h)
                              : run_gated<ElemF16>(M, I, H, X, ldx, W13, ldw, ep, C, ldc, ws, h);
}

int linear_backward_workspace_size(int64_t M, int64_t N, int64_t K, const uint16_t* dY, int64_t lddy, const uint16_t* X,
                                   int64_t ldx, const uint16_t* W, int64_t ldw, const uint16_t* dX, int64_t lddx,
                                   const uint16_t* dW, int64_t lddw, const uint16_t* dB, int64_t* bytes) {
    if (!bytes) return GR_ERR_INVALID_ARG;
    int st = validate_linear_backward(M, N, K, dY, lddy, X, ldx, W, ldw, dX, lddx, dW, lddw, dB);
    if (st != GR_OK) return st;
    GradLayout l;
    st = linear_layout(M, N, K, dY, lddy, W, ldw, dX, lddx, dW, dB, &l);
    *bytes = l.total();
    return st;
}

int linear_backward(int64_t M, int64_t N, int64_t K, const uint16_t* dY, int64_t lddy, const uint16_t* X, int64_t ldx,
                    const uint16_t* W, int64_t ldw, uint16_t* dX, int64_t lddx, uint16_t* dW, int64_t lddw, uint16_t* dB,
                    int fmt, void* workspace, int64_t workspace_bytes, void* stream) {
    int st = validate_linear_backward(M, N, K, dY, lddy, X, ldx, W, ldw, dX, lddx, dW, lddw, dB);
    if (st != GR_OK) return st;
    if (!known_fmt(fmt)) return GR_ERR_INVALID_ARG;
    GradLayout l;
    st = linear_layout(M, N, K, dY, lddy, W, ldw, dX, lddx, dW, dB, &l);
    if (st != GR_OK) return st;
    st = check_workspace(workspace, workspace_bytes, l.total());
    if (st != GR_OK) return st;
    const Region written[] = {matrix(dX, M, K, lddx), matrix(dW, N, K, lddw), vector(dB, N),
                              {reinterpret_cast<uintptr_t>(workspace), l.total()}};
    const Region read[] = {matrix(dY, M, N, lddy), matrix(dW ? X : nullptr, M, K, ldx), matrix(dX ? W : nullptr, N, K, ldw)};
    st = check_regions(written, read);
    if (st != GR_OK) return st;
    st = check_device();
    if (st != GR_OK) return st;
    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    hipStream_t h = static_cast<hipStream_t>(stream);
    return fmt == GR_FMT_BF16
               ? run_linear_backward<ElemBF16>(M, N, K, dY, lddy, X, ldx, W, ldw, dX, lddx, dW, lddw, dB, ws, l, h)
               : run_linear_backward<ElemF16>(M, N, K, dY, lddy, X, ldx, W, ldw, dX, lddx, dW, lddw, dB, ws, l, h);
}

int gated_linear_backward_workspace_size(int64_t M, int64_t I, int64_t H, const uint16_t* W13, int64_t ldw,
                                         const uint16_t* dX, int64_t lddx, const uint16_t* dW13, const uint16_t* dB13,
                                         int64_t* bytes) {
    if (!bytes) return GR_ERR_INVALID_ARG;
    if (!dim_ok(M) || !dim_ok(I) || !dim_ok(2 * I) || !dim_ok(H)) return GR_ERR_INVALID_DIM;
    if (dX && (ldw < least(H) || lddx < least(H))) return GR_ERR_INVALID_LD;
    if (M > 0 && I > 0 && H > 0 && dX && !W13) return GR_ERR_NULL_PTR;
    GradLayout l;
    const int st = gated_layout(M, I, H, W13, ldw, dX, lddx, dW13, dB13, &l);
    *bytes = l.total();
    return st;
}

int gated_linear_backward(int64_t M, int64_t I, int64_t H, const uint16_t* dH, int64_t lddh, const uint16_t* X, int64_t ldx,
                          const uint16_t* W13, int64_t ldw, const uint16_t* GU, int64_t ldgu, int act, uint16_t* dX,
                          int64_t lddx, uint16_t* dW13, int64_t lddw, uint16_t* dB13, int fmt, void* workspace,
                          int64_t workspace_bytes, void* stream) {
    int st = validate_gated_backward(M, I, H, dH, lddh, X, ldx, W13, ldw, GU, ldgu, dX, lddx, dW13, lddw, dB13);
    if (st != GR_OK) return st;
    if (!known_act(act) || !known_fmt(fmt)) return GR_ERR_INVALID_ARG;
    if (!dX && !dW13 && !dB13) return GR_OK;
    GradLayout l;
    st = gated_layout(M, I, H, W13, ldw, dX, lddx, dW13, dB13, &l);
    if (st != GR_OK) return st;
    st = check_workspace(workspace, workspace_bytes, l.total());
    if (st != GR_OK) return st;
    const Region written[] = {matrix(dX, M, H, lddx), matrix(dW13, 2 * I, H, lddw), vector(dB13, 2 * I),
                              {reinterpret_cast<uintptr_t>(workspace), l.total()}};
    const Region read[] = {matrix(dH, M, I, lddh), matrix(GU, M, 2 * I, ldgu), matrix(dW13 ? X : nullptr, M, H, ldx),
                           matrix(dX ? W13 : nullptr, 2 * I, H, ldw)};
    st = check_regions(written, read);
    if (st != GR_OK) return st;
    st = check_device();
    if (st != GR_OK) return st;
    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    hipStream_t h = static_cast<hipStream_t>(stream);
    return fmt == GR_FMT_BF16 ? run_gated_backward<ElemBF16>(M, I, H, dH, lddh, X, ldx, W13, ldw, GU, ldgu, act, dX, lddx,
                                                             dW13, lddw, dB13, ws, l, h)
                              : run_gated_backward<ElemF16>(M, I, H, dH, lddh, X, ldx, W13, ldw, GU, ldgu, act, dX, lddx,
                                                            dW13, lddw, dB13, ws, l, h);
}

}  // extern "C"
