// Host side of the products with an epilogue of their own: argument checks, the choice of a
// kernel and its launch.
#pragma once

#include <algorithm>
#include <initializer_list>
#include <utility>

#include "host.hpp"
#include "own_epilogue.hpp"
#include "smallm_kernel.hpp"
#include "tile128_kernel.hpp"
#include "tile3t_kernel.hpp"

namespace {

using gr::ElemBF16;
using gr::ElemF16;

constexpr int kStreamW = 4, kStreamR = 2, kStreamWOne = 8, kStreamNB = 64, kStreamRows = 64;
constexpr int64_t kMaxPitch = gr::tile2::MAX_LDA;  // 32-bit copy offsets over 256 rows

bool known_fmt(int fmt) { return fmt == GR_FMT_F16 || fmt == GR_FMT_BF16; }
bool known_act(int act) { return act >= 0 && act < gr::kActCount; }
int check_dims(std::initializer_list<int64_t> dims) {
    for (int64_t v : dims)
        if (v < 0) return GR_ERR_INVALID_DIM;
    for (int64_t v : dims)
        if (v > kMaxDim) return GR_ERR_TOO_LARGE;
    return GR_OK;
}
int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
int64_t aligned(int64_t bytes) { return round_up(bytes, kWorkspaceAlign); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t least(int64_t cols) { return cols > 1 ? cols : 1; }
// Workgroups for kernels that go over their rows with the grid's stride: a launch takes less than
// 2^32 threads.
int64_t held_grid(int64_t workgroups) { return workgroups < (1 << 20) ? workgroups : 1 << 20; }
bool rows16(const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; }

struct Region {
    uintptr_t at;
    int64_t bytes;
};
Region matrix(const void* p, int64_t rows, int64_t cols, int64_t ld) {
    return {reinterpret_cast<uintptr_t>(p), p ? span_bytes(rows, cols, ld) : 0};
}
Region vector(const void* p, int64_t n) { return {reinterpret_cast<uintptr_t>(p), p ? 2 * n : 0}; }

// GR_OK if none of the written regions meets another or one that is read.
template <int W, int R>
int check_regions(const Region (&written)[W], const Region (&read)[R]) {
    for (const Region& r : read)
        if (r.bytes < 0) return GR_ERR_TOO_LARGE;
    for (const Region& w : written)
        if (w.bytes < 0) return GR_ERR_TOO_LARGE;
    for (int i = 0; i < W; ++i) {
        for (int j = i + 1; j < W; ++j)
            if (overlaps(written[i].at, written[i].bytes, written[j].at, written[j].bytes)) return GR_ERR_ALIAS;
        for (const Region& r : read)
            if (overlaps(written[i].at, written[i].bytes, r.at, r.bytes)) return GR_ERR_ALIAS;
    }
    return GR_OK;
}

int check_workspace(const void* ws, int64_t bytes, int64_t need) {
    if (bytes < 0 || reinterpret_cast<uintptr_t>(ws) % kWorkspaceAlign != 0) return GR_ERR_INVALID_ARG;
    if (need == 0) return GR_OK;
    if (!ws) return GR_ERR_NULL_PTR;
    return bytes < need ? GR_ERR_SCRATCH : GR_OK;
}

// The kernels of C (M x N) = own epilogue of A Bt^T, both operands k-contiguous, for a
// type with an epilogue of its own.  `rows` of Bt make a column of C (2: paired).
enum Kernel { kTile256, kTile128, kStream4, kStream8 };
static_assert(gr::tile3t::BM == 256 && gr::tile3t::BN == 256 && gr::tile128::BM == 128 && gr::tile128::BN == 128, "sides");

// 256 x 256 tiles, a CU each, rather than 128 x 128, two to a CU: where the former are more
// than half as many as CUs and, with a short K, their rounds do not take longer.  A round of
// the latter takes about three quarters of the time, and the last one half of that on average
// (sums over 64 and 512 of 9536 x 1546, 266 and 975 tiles: 27.5 and 50.8 us with the large ones,
// 17.0 and 39.8 with the small; 8192 x 4096, 512 and 2048 tiles: 22.5 and 48.3, 28.8 and 58.5;
// over 2048 of 9536 x 1546: 113 and 117).
bool large_tiles(int64_t large, int64_t small, int64_t K) {
    return large > 128 && (K >= 2048 || 6 * small + 1536 > 4096 * ceil_div(large, 256));
}

// Which of them, for B products at once: up to 64 rows, and products of at most 512 blocks of 64 x 64 (sums of
// N x rows) with a K long enough to fill them, are streamed; else tiles.  The borders between
// streams and tiles are those of the transposed-B ReLU kernels, whose main loops these are.
// `triangle`: of N x N only the tiles on and below the diagonal (3000 x 3000 orthogonalised, 78
// large and 300 small tiles: 1101 us with the large, 957).
Kernel choose(int64_t B, int64_t M, int64_t N, int64_t K, int rows, bool triangle = false) {
    const int64_t on = kStreamNB / rows;
    const int64_t blocks = B * ceil_div(M, kStreamRows) * ceil_div(N, on);
    if (N >= on && (M <= kStreamRows || (blocks <= 256 && K >= 256) || (blocks <= 512 && K >= 1024)))
        return blocks <= 256 ? kStream8 : kStream4;
    auto tiles = [&](int64_t side) {
        const int64_t m = ceil_div(M, side), n = ceil_div(N, side / rows);
        return B * (triangle ? m * (m + 1) / 2 : m * n);
    };
    return K % gr::tile3t::BKS == 0 && M >= gr::tile3t::BM && large_tiles(tiles(256), tiles(128), K) ? kTile256 : kTile128;
}

constexpr uint32_t kGroupM = 4;  // tile rows that walk the columns together (see tile_of_workgroup)

template <typename E>
int product(Kernel kernel, int64_t B, int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda, const uint16_t* Bt,
            int64_t ldb, uint16_t* C, int64_t ldc, const typename E::Args& ep, hipStream_t stream) {
    constexpr int rows = E::kPairs ? 2 : 1;
    const typename E::Args args = ep;
    const int vec = 8;
    switch (kernel) {
        case kTile256: {
            using namespace gr::tile3t;
            constexpr int on = BN / rows;
            const uint32_t tm = (uint32_t)ceil_div(M, BM), tn = (uint32_t)ceil_div(N, on);
            if (M % BM == 0 && N % on == 0)
                return launch_grid(gemm_relu_tile3t_kernel<false, E>, dim3(tm * tn, (uint32_t)B), THREADS, stream, A, Bt, C, M, N, K, lda,
                              ldb, ldc, tm, tn, kGroupM, vec, args);
            return launch_grid(gemm_relu_tile3t_kernel<true, E>, dim3(tm * tn, (uint32_t)B), THREADS, stream, A, Bt, C, M, N, K, lda, ldb,
                          ldc, tm, tn, kGroupM, vec, args);
        }
        case kTile128: {
            using namespace gr::tile128;
            constexpr int on = BN / rows;
            const uint32_t tm = (uint32_t)ceil_div(M, BM), tn = (uint32_t)ceil_div(N, on);
            float* const part = nullptr;
            const int64_t whole = 0;
            if (M % BM == 0 && N % on == 0)
                return launch_grid(gemm_relu_tile128_kernel<false, false, true, E>, dim3(tm * tn, (uint32_t)B), THREADS, stream, A, Bt, C,
                              M, N, K, lda, ldb, ldc, tm, tn, kGroupM, vec, part, whole, args);
            return launch_grid(gemm_relu_tile128_kernel<true, false, true, E>, dim3(tm * tn, (uint32_t)B), THREADS, stream, A, Bt, C, M, N,
                          K, lda, ldb, ldc, tm, tn, kGroupM, vec, part, whole, args);
        }
        default: {
            using namespace gr::smallm;
            const uint32_t nb = (uint32_t)ceil_div(N, kStreamNB / rows);
            const int64_t blocks = ceil_div(M, kStreamRows) * nb, halves = ceil_div(M, kStreamRows / 2) * nb;
            // plain order where the column blocks fall on the XCDs evenly
            const uint32_t order = nb % 4 == 0 ? (gr::kNoXcdRemap | 1u) : kGroupM;
            float* const part = nullptr;
            // blocks of 32 rows where the chip holds those, too: a CU reads a quarter less and
            // half as many idle (gated layer, 77 x 1501 x 2080: 12.0 us with 64 rows, 9.7; 128 x
            // 704 x 2048 8.6 and 7.1; 32 x 8192 x 4096, rows of 64 half empty, 38.0 and 37.2)
            if (kernel == kStream8 && B * halves <= 256)
                return launch_grid(gemm_relu_smallm_stream_kernel<kStreamNB, kStreamWOne, kStreamR, stream::WHOLE, E, false, 2,
                                                                  true, true>,
                                   dim3((uint32_t)halves, (uint32_t)B), 64 * kStreamWOne, stream, A, Bt, C, part, M, N, K,
                                   lda, ldb, ldc, K, nb, order, args);
            if (kernel == kStream8)
                return launch_grid(gemm_relu_smallm_stream_kernel<kStreamNB, kStreamWOne, kStreamR, stream::WHOLE, E, false, 4,
                                                             true, true>,
                              dim3((uint32_t)blocks, (uint32_t)B), 64 * kStreamWOne, stream, A, Bt, C, part, M, N, K, lda, ldb, ldc, K, nb, order, args);
            return launch_grid(
                gemm_relu_smallm_stream_kernel<kStreamNB, kStreamW, kStreamR, stream::WHOLE, E, false, 4, true, true>,
                dim3((uint32_t)blocks, (uint32_t)B), 64 * kStreamW, stream, A, Bt, C, part, M, N, K, lda, ldb, ldc, K, nb, order, args);
        }
    }
}

// How a weight's gradient, a plain product whose K are the tokens, is computed beside an
// input's.  Streamed, where the blocks (of both, if `together`: one launch) fit the chip, or
// are half as many again and those of the longer product begin first (333 x 2080 x 1001, 528
// and 96 blocks: 22 us, 28 as tiles and blocks of their own launches; 864 blocks would lose: 35 against 33).
// Its K is then cut into `splits` ranges for blocks that would stay empty otherwise, if that
// saves a wave kPassSteps steps of 32, which take about as long as the second pass over the
// ranges' sums (whole and cut, all of linear_backward in bf16: 8192 tokens x 256 x 256 47 and
// 23 us, 6061 x 320 x 222 40 and 22, 4096 x 64 x 64 23 and 11; 1024 x 1024 x 1024 saves too
// little: 19 whole).  Of the
// three ways to stream the one with the fewest steps per wave, where those of blocks that do
// not all fit count one and a half.  Else 128 x 128 tiles together where each alone would
// take them, or by itself by the rule above.
struct Shape {
    int64_t M, N, K;
};
struct WeightPlan {
    Kernel kernel;
    bool together;
    int64_t splits, k_per;
};

// `other` blocks of a product with `other_steps` of 32 run beside; false: more than fit.
constexpr int64_t kPassSteps = 10;
bool plan_stream(const Shape& p, int64_t other, int64_t other_steps, WeightPlan* plan) {
    const int64_t blocks = ceil_div(p.M, kStreamRows) * ceil_div(p.N, kStreamNB);
    if (blocks == 0) return false;
    struct Way {
        Kernel kernel;
        int64_t waves, most, cost;
    };
    int64_t least_cost = -1;
    for (const Way& way : {Way{kStream8, kStreamWOne, 256, 2}, Way{kStream4, kStreamW, 512, 2}, Way{kStream4, kStreamW, 768, 3}}) {
        if (blocks + other > way.most || (other == 0 && way.most > 512)) continue;
        const int64_t step = 32 * way.waves, splits = std::min<int64_t>((way.most - other) / blocks, 32);
        const int64_t cut = round_up(ceil_div(p.K, splits), step), k_per = p.K / step - cut / step >= kPassSteps ? cut : p.K;
        const int64_t steps = k_per / step + (k_per < p.K ? kPassSteps : 0);
        const int64_t cost = way.cost * std::max(steps, other_steps / way.waves);
        if (least_cost < 0 || cost < least_cost) {
            *plan = {way.kernel, other > 0, ceil_div(p.K, k_per), k_per};
            least_cost = cost;
        }
    }
    return least_cost >= 0;
}

WeightPlan plan_weight(const Shape& weight, const Shape& input) {
    WeightPlan plan{choose(1, weight.M, weight.N, weight.K, 1), false, 1, weight.K};
    const int64_t beside = ceil_div(input.M, kStreamRows) * ceil_div(input.N, kStreamNB);
    if (weight.N >= kStreamNB && input.N >= kStreamNB && beside > 0 && plan_stream(weight, beside, input.K / 32, &plan)) return plan;
    plan.together = plan.kernel == kTile128 && choose(1, input.M, input.N, input.K, 1) == kTile128;
    WeightPlan cut = plan;
    if (!plan.together && weight.N >= kStreamNB && plan_stream(weight, 0, 0, &cut) && cut.splits > 1) return cut;
    return plan;
}

// Up to two plain products and the sums over the rows of the first one's A, in one launch
// where they are small: then a launch takes longer than a product.
template <typename Base>
struct Small {
    gr::own::TwoArgs args{};
    int count = 0;

    void add(int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda, const uint16_t* Bt, int64_t ldb, uint16_t* C,
             int64_t ldc) {
        args.product[count++] = {A, Bt, C, M, N, K, lda, ldb, ldc, 1, 0, 0, 1, K, nullptr};
    }
    int run(Kernel kernel, hipStream_t stream) {
        using E = gr::own::Two<Base>;
        // the longer blocks begin first
        if (args.product[1].k_per > args.product[0].k_per) std::swap(args.product[0], args.product[1]);
        const int64_t side = kernel == kTile128 ? gr::tile128::BM : kStreamRows;
        int64_t grid = 0;
        for (int i = 0; i < count; ++i) {
            gr::own::Product& p = args.product[i];
            p.n_blocks = (uint32_t)ceil_div(p.N, side);
            p.blocks = (uint32_t)ceil_div(p.M, side) * p.n_blocks;
            p.order = kernel != kTile128 && p.n_blocks % 4 == 0 ? (gr::kNoXcdRemap | 1u) : kGroupM;
            grid += (int64_t)p.blocks * p.splits;
        }
        const gr::own::TwoArgs a = args;
        const int64_t none = 0;
        const uint16_t* const in = nullptr;
        uint16_t* const out = nullptr;
        float* const part = nullptr;
        const uint32_t zero = 0;
        if (kernel == kTile128) {
            using namespace gr::tile128;
            grid += ceil_div(a.sum_rows, THREADS / 64);
            return launch(gemm_relu_tile128_kernel<true, false, true, E>, grid, THREADS, stream, in, in, out, none, none, none,
                          none, none, none, zero, zero, zero, 8, part, none, a);
        }
        using namespace gr::smallm;
        const int waves = kernel == kStream8 ? kStreamWOne : kStreamW;
        grid += ceil_div(a.sum_rows, waves);
        if (kernel == kStream8)
            return launch(gemm_relu_smallm_stream_kernel<kStreamNB, kStreamWOne, kStreamR, stream::WHOLE, E, false, 4, true, true>,
                          grid, 64 * waves, stream, in, in, out, part, none, none, none, none, none, none, none, zero, zero, a);
        return launch(gemm_relu_smallm_stream_kernel<kStreamNB, kStreamW, kStreamR, stream::WHOLE, E, false, 4, true, true>, grid,
                      64 * waves, stream, in, in, out, part, none, none, none, none, none, none, none, zero, zero, a);
    }
};

// The same for B products of one shape (grid y), and for symmetric ones C = own
// epilogue of A A^T, A N x K.
template <typename E>
int batched(int64_t B, int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda, const uint16_t* Bt, int64_t ldb,
            uint16_t* C, int64_t ldc, const typename E::Args& ep, hipStream_t stream) {
    return product<E>(choose(B, M, N, K, 1), B, M, N, K, A, lda, Bt, ldb, C, ldc, ep, stream);
}

// Below the diagonal half of the tiles are left out; ep.ct is C, which gets the others from
// their mirror images.  The streamed blocks are computed all: they fit the chip at once
// either way.
template <typename In>
int symmetric(int64_t B, int64_t N, int64_t K, const uint16_t* A, int64_t lda, uint16_t* C, int64_t ldc,
              gr::own::PolyArgs ep, hipStream_t stream) {
    using namespace gr::own;
    const Kernel kernel = choose(B, N, N, K, 1, true);
    if (kernel == kStream4 || kernel == kStream8) {
        ep.ct = nullptr;
        return product<Poly<In, In, false>>(kernel, B, N, N, K, A, lda, A, lda, C, ldc, ep, stream);
    }
    using E = Poly<In, In, true>;
    const int vec = 8;
    if (kernel == kTile256) {
        using namespace gr::tile3t;
        const uint32_t t = (uint32_t)ceil_div(N, BM);
        const dim3 grid(t * (t + 1) / 2, (uint32_t)B);
        if (N % BM == 0)
            return launch_grid(gemm_relu_tile3t_kernel<false, E>, grid, THREADS, stream, A, A, C, N, N, K, lda, lda, ldc, t, t,
                               kGroupM, vec, ep);
        return launch_grid(gemm_relu_tile3t_kernel<true, E>, grid, THREADS, stream, A, A, C, N, N, K, lda, lda, ldc, t, t,
                           kGroupM, vec, ep);
    }
    using namespace gr::tile128;
    const uint32_t t = (uint32_t)ceil_div(N, BM);
    const dim3 grid(t * (t + 1) / 2, (uint32_t)B);
    float* const part = nullptr;
    const int64_t whole = 0;
    if (N % BM == 0)
        return launch_grid(gemm_relu_tile128_kernel<false, false, true, E>, grid, THREADS, stream, A, A, C, N, N, K, lda, lda,
                           ldc, t, t, kGroupM, vec, part, whole, ep);
    return launch_grid(gemm_relu_tile128_kernel<true, false, true, E>, grid, THREADS, stream, A, A, C, N, N, K, lda, lda, ldc,
                       t, t, kGroupM, vec, part, whole, ep);
}

}  // namespace
