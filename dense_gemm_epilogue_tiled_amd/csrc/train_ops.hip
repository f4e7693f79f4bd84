// Host side of the products of training: the gated linear layer and the gradients of
// linear layers.  See include/gemm_relu.h.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gemm_relu.h"
#include "gemv_kernel.hpp"
#include "own_products.hpp"
#include "tile3_kernel.hpp"
#include "train_kernel.hpp"

namespace {

// Copies with padded or transposed rows, all of a call's in one launch.
struct Relayouts {
    gr::train::Jobs jobs{};
    int count = 0;
    int64_t tiles = 0;

    Relayouts() {
        for (gr::train::Job& j : jobs.job) j.tiles_c = 1;
    }
    // dst: src (rows x cols, pitch lds) with rows of ldd = pad elements, or src's transpose.
    void add(bool transposed, const uint16_t* src, int64_t rows, int64_t cols, int64_t lds, uint16_t* dst, int64_t pad) {
        using gr::train::TILE;
        const int64_t tr = ceil_div(transposed ? pad : rows, TILE), tc = ceil_div(transposed ? cols : pad, TILE);
        if (tr * tc == 0) return;
        jobs.job[count++] = {src, dst, rows, cols, lds, pad, pad, (uint32_t)tc, (uint32_t)(tr * tc), transposed ? 1 : 0};
        tiles += tr * tc;
    }
    int run(hipStream_t stream) const {
        return tiles == 0 ? GR_OK : launch(gr::train::relayout_kernel, tiles, gr::train::THREADS, stream, jobs);
    }
};

// ---- the gated linear layer -----------------------------------------------------------

constexpr int kSmallMRows = 16;
constexpr int kGemvRows = 4;

// K that is not a whole number of 32-deep steps (0 included), with more tokens than the
// kernel for few takes: x and the weight are copied into the workspace with K padded by zeros.
bool gated_packs(int64_t H) { return H % 32 != 0 || H == 0; }
int64_t gated_pitch(int64_t H) { return H > 0 ? round_up(H, 64) : 64; }

int64_t gated_need(int64_t M, int64_t I, int64_t H) {
    if (M <= kGemvRows || I == 0 || !gated_packs(H)) return 0;
    return aligned(M * gated_pitch(H) * 2) + aligned(2 * I * gated_pitch(H) * 2);
}

template <typename Base>
int run_gated(int64_t M, int64_t I, int64_t H, const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
              const gr::own::GatedArgs& ep, uint16_t* C, int64_t ldc, uint8_t* ws, hipStream_t stream) {
    using E = gr::own::Gated<Base>;
    if (M <= kGemvRows) {
        using namespace gr::gemv;
        const Args a{X, W, C, M, I, H, ldx, ldw, ldc, ep};
        const int64_t grid = held_grid(ceil_div(I, WAVES * COLS));
        if (M == 1) return launch(gated_gemv_kernel<Base, 1>, grid, THREADS, stream, a);
        if (M == 2) return launch(gated_gemv_kernel<Base, 2>, grid, THREADS, stream, a);
        return launch(gated_gemv_kernel<Base, 4>, grid, THREADS, stream, a);
    }
    int64_t K = H;
    if (gated_packs(H)) {
        K = gated_pitch(H);
        uint16_t* const xp = reinterpret_cast<uint16_t*>(ws);
        uint16_t* const wp = reinterpret_cast<uint16_t*>(ws + aligned(M * K * 2));
        Relayouts copies;
        copies.add(false, X, M, H, ldx, xp, K);
        copies.add(false, W, 2 * I, H, ldw, wp, K);
        const int st = copies.run(stream);
        if (st != GR_OK) return st;
        X = xp;
        W = wp;
        ldx = ldw = K;
    }
    if (M <= kSmallMRows && K % gr::smallm::BTS_KC == 0) {
        // two waves to a workgroup, so that the last round of workgroups is a small part of all
        // (5 x 4096 x 4096: 12.6 us, 16.9 with four; 16 x 11008 x 4096: 42.7 and 43.6)
        constexpr int W2 = 2;
        const gr::own::GatedArgs args = ep;
        return launch(gr::smallm::gemm_relu_smallm_bt_stream_kernel<true, E, W2, 16>, ceil_div(I, 8 * W2), 64 * W2, stream, X, W,
                      C, M, I, K, ldx, ldw, ldc, args);
    }
    return product<E>(choose(1, M, I, K, 2), 1, M, I, K, X, ldx, W, ldw, C, ldc, ep, stream);
}

// ---- gradients ------------------------------------------------------------------------

// How dX = dY W (M x K, sums over N) is computed: 256 x 256 tiles with no epilogue but the
// rounding where they are many; on W transposed, with N padded to whole strips by
// zeros, where the product of row-major operands would have misaligned rows or a ragged
// depth (333 x 2080 x 1001: 41 us in place, 13 with the copies) and the copies are not most
// of the work, and where W is so small that its copy beside the other ones costs less than a
// launch of the product's own; else gemm_bias_act's paths.
constexpr int64_t kSmallWeight = int64_t(1) << 21;  // elements
enum InputGrad { kTiles, kTransposed, kPaths };

template <typename Base>
struct Bare : Base {
    static __device__ __forceinline__ uint16_t relu_round(float x) { return (uint16_t)gr::own::round2<Base>(x, x); }
};

int64_t padded_depth(int64_t N) { return round_up(N, 64); }

InputGrad input_grad_kind(int64_t M, int64_t K, int64_t N, const uint16_t* dY, int64_t lddy, const uint16_t* W, int64_t ldw) {
    using namespace gr::tile3;
    const bool whole = rows16(dY, lddy) && rows16(W, ldw) && N > 0;
    if (whole && M >= BM && N % BKA == 0 && lddy <= gr::tile2::MAX_LDA && ldw <= gr::tile2::MAX_LDB &&
        ceil_div(M, BM) * ceil_div(K, BN) > 128)
        return kTiles;
    const bool ragged = M > kStreamRows && !(whole && N % 32 == 0);
    if (N > 0 && padded_depth(N) <= kMaxPitch && (ragged || N <= kSmallWeight / K)) return kTransposed;
    return kPaths;
}

// Bytes for W^T, for dY with N padded (not for one that comes padded, `padded`), and for the
// paths of gemm_bias_act.
struct InputGradLayout {
    InputGrad kind = kPaths;
    int64_t wt = 0, dy = 0, paths = 0;
    int64_t total() const { return wt + dy + paths; }
};

int input_grad_layout(int64_t M, int64_t K, int64_t N, const uint16_t* dY, int64_t lddy, bool padded, const uint16_t* W,
                      int64_t ldw, const uint16_t* dX, int64_t lddx, InputGradLayout* l) {
    *l = InputGradLayout{};
    if (M == 0 || K == 0) return GR_OK;
    l->kind = input_grad_kind(M, K, N, dY, lddy, W, ldw);
    if (l->kind == kTransposed) {
        l->wt = aligned(2 * K * padded_depth(N));
        l->dy = padded ? 0 : aligned(2 * M * padded_depth(N));
    } else if (l->kind == kPaths) {
        const int st = gemm_relu_f16_workspace_size(M, K, N, dY, lddy, W, ldw, dX, lddx, &l->paths);
        l->paths = aligned(l->paths);
        return st;
    }
    return GR_OK;
}

// The copies that it works on.
void input_grad_copies(const InputGradLayout& l, int64_t M, int64_t K, int64_t N, const uint16_t* dY, int64_t lddy,
                       const uint16_t* W, int64_t ldw, uint8_t* ws, Relayouts* copies) {
    if (l.kind != kTransposed) return;
    const int64_t Np = padded_depth(N);
    copies->add(true, W, N, K, ldw, reinterpret_cast<uint16_t*>(ws), Np);
    if (l.dy > 0) copies->add(false, dY, M, N, lddy, reinterpret_cast<uint16_t*>(ws + l.wt), Np);
}

template <typename Base>
int input_grad(const InputGradLayout& l, int64_t M, int64_t K, int64_t N, const uint16_t* dY, int64_t lddy, const uint16_t* W,
               int64_t ldw, uint16_t* dX, int64_t lddx, uint8_t* ws, hipStream_t stream) {
    if (l.kind == kTiles) {
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
    if (l.kind == kTransposed) {
        const int64_t Np = padded_depth(N);
        const uint16_t* const dyp = l.dy > 0 ? reinterpret_cast<const uint16_t*>(ws + l.wt) : dY;
        return product<gr::own::Plain<Base>>(choose(1, M, K, Np, 1), 1, M, K, Np, dyp, Np, reinterpret_cast<const uint16_t*>(ws),
                                             Np, dX, lddx, gr::own::PlainArgs{}, stream);
    }
    return gemm_bias_act_ws(M, K, N, dY, lddy, W, ldw, nullptr, GR_ACT_NONE, dX, lddx,
                            Base::kIsF16 ? GR_FMT_F16 : GR_FMT_BF16, l.paths > 0 ? ws : nullptr, l.paths, stream, -1);
}

template <typename Base>
int bias_grad(int64_t N, int64_t Mp, const uint16_t* dYt, uint16_t* dB, hipStream_t stream) {
    return launch(gr::train::row_sums_kernel<Base>, held_grid(ceil_div(N, 4)), gr::train::THREADS, stream, dYt, N, Mp, Mp, dB);
}

int64_t padded_tokens(int64_t M) { return M > 0 ? round_up(M, gr::train::PAD) : gr::train::PAD; }

WeightPlan weight_plan(int64_t M, int64_t N, int64_t K) {
    return plan_weight({N, K, padded_tokens(M)}, {M, K, padded_depth(N)});
}
// fp32 sums of the ranges of tokens.
int64_t parts_need(int64_t M, int64_t N, int64_t K) {
    const WeightPlan plan = weight_plan(M, N, K);
    return plan.splits > 1 ? aligned(plan.splits * N * K * 4) : 0;
}

// dX, dW (N x K) and dB from what the copies made ready; rest: input_grad's workspace.
template <typename Base>
int grad_products(const InputGradLayout& l, int64_t M, int64_t N, int64_t K, int64_t Mp, const uint16_t* dYt, const uint16_t* Xt,
                  const uint16_t* dY, int64_t lddy, const uint16_t* W, int64_t ldw, uint16_t* dX, int64_t lddx, uint16_t* dW,
                  int64_t lddw, uint16_t* dB, float* part, uint8_t* rest, hipStream_t stream) {
    const bool weight = dW && N > 0 && K > 0, input = dX && M > 0 && K > 0, bias = dB && N > 0;
    // by the shapes alone, so that a gradient has the same bits with and without the others
    const int64_t Np = padded_depth(N);
    const WeightPlan plan = weight_plan(M, N, K);
    const Kernel kernel = plan.kernel;  // dW's
    const bool together = plan.together && input && l.kind == kTransposed;
    int st = GR_OK;
    if (kernel != kTile256 && (weight || together)) {
        Small<Base> small;
        if (weight) {
            small.add(N, K, Mp, dYt, Mp, Xt, Mp, dW, lddw);
            if (plan.splits > 1) {
                gr::own::Product& p = small.args.product[0];
                p.splits = (uint32_t)plan.splits;
                p.k_per = plan.k_per;
                p.part = part;
            }
        }
        if (together)
            small.add(M, K, Np, l.dy > 0 ? reinterpret_cast<const uint16_t*>(rest + l.wt) : dY, Np,
                      reinterpret_cast<const uint16_t*>(rest), Np, dX, lddx);
        if (weight && bias) {
            small.args.sums = dB;
            small.args.sum_of = dYt;
            small.args.sum_rows = N;
            small.args.sum_k = Mp;
        }
        st = small.run(kernel, stream);
        if (st == GR_OK && weight && plan.splits > 1) {
            using namespace gr::train;
            const float* const from = part;
            const int vec = K % 4 == 0 ? 4 : 1;
            const int64_t grid = ceil_div(N * K, THREADS * vec) < 2048 ? ceil_div(N * K, THREADS * vec) : 2048;
            st = vec == 4 ? launch(sum_splits_kernel<Base, 4>, grid, THREADS, stream, from, plan.splits, N, K, dW, lddw)
                          : launch(sum_splits_kernel<Base, 1>, grid, THREADS, stream, from, plan.splits, N, K, dW, lddw);
        }
    } else if (weight) {
        st = product<gr::own::Plain<Base>>(kernel, 1, N, K, Mp, dYt, Mp, Xt, Mp, dW, lddw, gr::own::PlainArgs{}, stream);
    }
    if (st == GR_OK && bias && (kernel == kTile256 || !weight)) st = bias_grad<Base>(N, Mp, dYt, dB, stream);
    if (st == GR_OK && input && !together) st = input_grad<Base>(l, M, K, N, dY, lddy, W, ldw, dX, lddx, rest, stream);
    return st;
}

// The parts of the workspace, in order; only those of the gradients that are asked for.
struct GradLayout {
    int64_t dyt, xt, dy, parts;  // bytes: dY^T, X^T, dY (of the gated layer), fp32 sums
    InputGradLayout input;       // what dX's product takes
    int64_t total() const { return dyt + xt + dy + parts + input.total(); }
};

int linear_layout(int64_t M, int64_t N, int64_t K, const uint16_t* dY, int64_t lddy, const uint16_t* W, int64_t ldw,
                  const uint16_t* dX, int64_t lddx, const uint16_t* dW, const uint16_t* dB, GradLayout* l) {
    const int64_t Mp = padded_tokens(M);
    l->dyt = (dW || dB) ? aligned(2 * N * Mp) : 0;
    l->xt = dW ? aligned(2 * K * Mp) : 0;
    l->dy = 0;
    l->parts = dW ? parts_need(M, N, K) : 0;
    l->input = InputGradLayout{};
    return dX ? input_grad_layout(M, K, N, dY, lddy, false, W, ldw, dX, lddx, &l->input) : GR_OK;
}


int validate_linear_backward(int64_t M, int64_t N, int64_t K, const uint16_t* dY, int64_t lddy, const uint16_t* X, int64_t ldx,
                             const uint16_t* W, int64_t ldw, const uint16_t* dX, int64_t lddx, const uint16_t* dW,
                             int64_t lddw, const uint16_t* dB) {
    const int dims = check_dims({M, N, K});
    if (dims != GR_OK) return dims;
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
    float* const part = reinterpret_cast<float*>(ws + l.dyt + l.xt);
    uint8_t* const rest = ws + l.dyt + l.xt + l.parts;
    Relayouts copies;
    if (dB || (dW && K > 0)) copies.add(true, dY, M, N, lddy, dyt, Mp);
    if (dW && N > 0) copies.add(true, X, M, K, ldx, xt, Mp);
    if (dX && M > 0 && K > 0) input_grad_copies(l.input, M, K, N, dY, lddy, W, ldw, rest, &copies);
    const int st = copies.run(stream);
    if (st != GR_OK) return st;
    return grad_products<Base>(l.input, M, N, K, Mp, dyt, xt, dY, lddy, W, ldw, dX, lddx, dW, lddw, dB, part, rest, stream);
}

int gated_layout(int64_t M, int64_t I, int64_t H, const uint16_t* W, int64_t ldw, const uint16_t* dX, int64_t lddx,
                 const uint16_t* dW, const uint16_t* dB, GradLayout* l) {
    const int64_t Mp = padded_tokens(M), ld = padded_depth(2 * I);
    l->dyt = (dW || dB) ? aligned(4 * I * Mp) : 0;
    l->xt = dW ? aligned(2 * H * Mp) : 0;
    l->dy = aligned(2 * M * ld);
    l->parts = dW ? parts_need(M, 2 * I, H) : 0;
    l->input = InputGradLayout{};
    if (!dX) return GR_OK;
    // the gradient of the products lies in the workspace: an aligned address that is
    // nobody's stands for it
    const uint16_t* const place = reinterpret_cast<const uint16_t*>(uintptr_t(1) << 62);
    return input_grad_layout(M, H, 2 * I, place, least(ld), true, W, ldw, dX, lddx, &l->input);
}

// Sides that the size and the call take alike.
int check_gated_backward(int64_t M, int64_t I, int64_t H) {
    const int dims = check_dims({M, I, 2 * I, H});
    if (dims != GR_OK) return dims;
    return padded_tokens(M) > kMaxPitch || 2 * I + 64 > kMaxPitch ? GR_ERR_TOO_LARGE : GR_OK;
}

int validate_gated_backward(int64_t M, int64_t I, int64_t H, const uint16_t* dH, int64_t lddh, const uint16_t* X,
                            int64_t ldx, const uint16_t* W, int64_t ldw, const uint16_t* GU, int64_t ldgu,
                            const uint16_t* dX, int64_t lddx, const uint16_t* dW, int64_t lddw, const uint16_t* dB) {
    const int dims = check_dims({M, I, 2 * I, H});
    if (dims != GR_OK) return dims;
    if (lddh < least(I) || ldgu < least(2 * I)) return GR_ERR_INVALID_LD;
    if (dX && (ldw < least(H) || lddx < least(H))) return GR_ERR_INVALID_LD;
    if (dW && (ldx < least(H) || lddw < least(H))) return GR_ERR_INVALID_LD;
    const bool any = dX || dW || dB;
    if (any && M > 0 && I > 0 && (!dH || !GU)) return GR_ERR_NULL_PTR;
    if (M > 0 && I > 0 && H > 0 && ((dX && !W) || (dW && !X))) return GR_ERR_NULL_PTR;
    return check_gated_backward(M, I, H);
}

template <typename Base>
int run_gated_backward(int64_t M, int64_t I, int64_t H, const uint16_t* dH, int64_t lddh, const uint16_t* X, int64_t ldx,
                       const uint16_t* W, int64_t ldw, const uint16_t* GU, int64_t ldgu, int act, uint16_t* dX, int64_t lddx,
                       uint16_t* dW, int64_t lddw, uint16_t* dB, uint8_t* ws, const GradLayout& l, hipStream_t stream) {
    using namespace gr::train;
    const int64_t Mp = padded_tokens(M), ld = padded_depth(2 * I);
    uint16_t* const dyt = reinterpret_cast<uint16_t*>(ws);
    uint16_t* const xt = reinterpret_cast<uint16_t*>(ws + l.dyt);
    uint16_t* const dgu = reinterpret_cast<uint16_t*>(ws + l.dyt + l.xt);
    float* const part = reinterpret_cast<float*>(ws + l.dyt + l.xt + l.dy);
    uint8_t* const rest = ws + l.dyt + l.xt + l.dy + l.parts;
    Relayouts copies;
    if (dW && I > 0) copies.add(true, X, M, H, ldx, xt, Mp);
    if (dX && M > 0 && H > 0) input_grad_copies(l.input, M, H, 2 * I, dgu, least(ld), W, ldw, rest, &copies);
    int st = GR_OK;
    if (I > 0) {
        const GatedBwdArgs a{dH, GU, dgu, l.dyt > 0 ? dyt : nullptr, M, I, lddh, ldgu, ld, Mp, act};
        const uint32_t tc = (uint32_t)ceil_div(I, TILE), tiles = (uint32_t)(Mp / TILE) * tc;
        st = launch(gated_backward_kernel<Base>, tiles + copies.tiles, THREADS, stream, a, tc, tiles, copies.jobs);
    } else {
        st = copies.run(stream);
    }
    if (st != GR_OK) return st;
    return grad_products<Base>(l.input, M, 2 * I, H, Mp, dyt, xt, dgu, least(ld), W, ldw, dX, lddx, dW, lddw, dB, part, rest, stream);
}

}  // namespace

extern "C" {

int gated_linear_workspace_size(int64_t M, int64_t I, int64_t H, int64_t* bytes) {
    if (!bytes) return GR_ERR_INVALID_ARG;
    const int dims = check_dims({M, I, 2 * I, H});
    if (dims != GR_OK) return dims;
    if (M > 0 && I > 0 && H > kMaxPitch) return GR_ERR_TOO_LARGE;  // (no pitch fits: the call refuses it)
    *bytes = gated_need(M, I, H);
    return GR_OK;
}

int gated_linear_bt(int64_t M, int64_t I, int64_t H, const uint16_t* X, int64_t ldx, const uint16_t* W13, int64_t ldw,
                    const uint16_t* b13, int act, uint16_t* C, int64_t ldc, uint16_t* GU, int64_t ldgu, int fmt,
                    void* workspace, int64_t workspace_bytes, void* stream) {
    const int dims = check_dims({M, I, 2 * I, H});
    if (dims != GR_OK) return dims;
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
    const int dims = check_dims({M, I, 2 * I, H});
    if (dims != GR_OK) return dims;
    if (dX && (ldw < least(H) || lddx < least(H))) return GR_ERR_INVALID_LD;
    if (M > 0 && I > 0 && H > 0 && dX && !W13) return GR_ERR_NULL_PTR;
    int st = check_gated_backward(M, I, H);
    if (st != GR_OK) return st;
    GradLayout l;
    st = gated_layout(M, I, H, W13, ldw, dX, lddx, dW13, dB13, &l);
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
