// A Linear layer on DFP-8 operands (int8 mantissas, one shared exponent per
// tensor) with bias, activation and residual in the product's epilogue, and
// its backward pass ("Mixed Precision Training of Convolutional Neural
// Networks using Integer Operations", sections 3 and 4: integer products,
// the exponents added, the operations around them in floating point).
//
//   z = fl(X W^T) 2^(eX + eW) + bias,  Y = act(z) + residual
//   dZ = dY act'(Z) -> dZ8, edZ;  dX = fl(dZ8 W) 2^(edZ + eW),
//   G = fl(dZ8^T X) 2^(edZ + eX),  gb = column sums of dZ
//
// The sums are exact in int32, so how a product is cut never shows in its
// result.  Five ways, by the sizes (make_plan): a forward product of few rows
// or few outputs, the reduction cut among a workgroup's wavefronts
// (dfp8_rows.h); large and middle products in 256 x 256 and 128 x 128 tiles
// (dfp8_tile256.h, dfp8_tile128.h); the others in 64 x 64 tiles (dfp8_tile.h), a
// long reduction of few tiles in ranges whose int32 sums a second pass adds, and
// contiguous sides shorter than 16 bytes in the same tiles with careful loads.
#include "dfp8_convert.h"
#include "dfp8_rows.h"
#include "dfp8_tile128.h"

namespace ionn {
namespace {

using namespace dfp8;

constexpr int64_t kMaxSide = int64_t(1) << 30;

bool sizes_ok(int64_t B, int64_t IN, int64_t OUT) {
    return B >= 0 && IN >= 0 && OUT >= 0 && B <= kMaxSide && IN <= kMaxSide && OUT <= kMaxSide;
}

// ---- how a product is cut ------------------------------------------------------

enum Path {
    ROWS = IONN_DFP8_ROWS,
    TILE256 = IONN_DFP8_TILES_256,
    TILE128 = IONN_DFP8_TILES_128,
    TILE = IONN_DFP8_TILES,
    TINY = IONN_DFP8_NARROW
};

struct Plan {
    Path path;
    int64_t tiles;
    int split;
    int rows, cols;  // ROWS: groups of 16 rows and of 16 outputs in a workgroup
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// By the sizes alone (the workspace query knows no addresses); operands whose
// address does not suit TILE256 and TILE128 take TILE.
template <bool A_KM, bool B_KM>
Plan make_plan(int64_t M, int64_t N, int64_t K, bool forward) {
    Plan p{TILE, ceil_div(M, 64) * ceil_div(N, 64), 1, 0, 0};
    const int64_t a_side = A_KM ? K : M, b_side = B_KM ? K : N;  // contiguous
    // Straight into matrix operands: the smallest tile that a grid of one
    // workgroup per compute unit covers, for these products are bound by one
    // trip after another of the longest workgroup (in tiles of 64, 256 x 784 x
    // 256 takes 5.4 us against 2.7, 512 x 1024 x 1024 5.7 against 4.4).  A long
    // reduction is better cut between workgroups (K = 32768, 32 rows, 64
    // outputs: 14.3 us here, 9.5 in tiles; 256 x 12000 x 1000 18.5 and 16.6; but
    // 32 x 16384 x 256 8.6 and 9.5), a short one leaves the largest tile no
    // lead (512 x 256 x 1024: 3.7 us both).  Few rows against many outputs are
    // bound by reading W, here too: 32 x 4096 x 16384 20 against 24.5 us, but
    // 37.6 and 37.7 at 32768 outputs; for up to 8 rows a second group of
    // outputs is no gain (8 x 1024 x 65536 14.1 against 16.4 us; 16 x 4096 x
    // 16384 18.7 against 16.9).
    if (forward && K >= kRowsMinK) {
        const auto fits = [&](int rows, int cols) { return ceil_div(M, 16 * rows) * ceil_div(N, 16 * cols) <= 256; };
        // (a grid of more threads than the runtime takes: B = 1, IN = 16, 2^27 outputs)
        const auto starts = [&](int cols) { return ceil_div(N, 16 * cols) <= max_groups(kRowWaves * 64); };
        if (K <= 16384 && fits(1, 1)) p.rows = 1, p.cols = 1;
        else if (K <= 16384 && fits(1, 2)) p.rows = 1, p.cols = 2;
        else if (K <= 8192 && fits(2, 2)) p.rows = 2, p.cols = 2;
        else if (K <= 8192 && K >= 512 && fits(4, 2)) p.rows = 4, p.cols = 2;
        else if (M <= 8 && N > 4096 && starts(1)) p.rows = 1, p.cols = 1;
        else if (M <= 16 && K <= 16384 && starts(2)) p.rows = 1, p.cols = 2;
        else if (M <= 32 && K <= 16384 && N <= 16384) p.rows = 2, p.cols = 2;
        if (p.rows) {
            p.path = ROWS;
            return p;
        }
    }
    if (a_side < 16 || b_side < 16) {
        p.path = TINY;
        return p;
    }
    const int64_t lda = a_side, ldb = b_side;
    // The tile size that is expected to end first; in us, fitted to
    // measurements: a round of 256 x 256 tiles, one per compute unit, takes 23 (15
    // without an activation) and K / 110; 128 x 128 tiles, two at a time on a
    // compute unit, by the tiles that one gets; 64 x 64 tiles by the share of M N K.
    // Forward in tiles of 64, 128 and 256: 1000 x 1024 x 2048 8.3, 11.2 and 26 us;
    // 2048^3 22.5, 17.6 and 35; 2048 x 4096 x 4096 67, 42 and 54; 4096^3 128, 78
    // and 70.  With both gradients: 512^3 12, 19 and 35; 4096 x 1024 x 4096 110, 81
    // (74 in one grid) and 121.
    if (tile256_fits<A_KM, B_KM>(nullptr, lda, nullptr, ldb, M, N, K)) {
        const int64_t tiles256 = ceil_div(M, 256) * ceil_div(N, 256), tiles128 = ceil_div(M, 128) * ceil_div(N, 128);
        const double rounds = double(ceil_div(tiles256, 256)), each = double(ceil_div(tiles128, 256)), k = double(K);
        const double t64 = (forward ? 5.0 : 2.5) + double(M) * double(N) * k / 65536.0 / (forward ? 6800.0 : 6500.0);
        const double t128 = forward ? 3.5 + 2.6 * each + k * (0.0022 + 0.0031 * each)
                                    : 2.5 + 1.8 * each + k * (0.0018 + 0.0031 * each);
        const double t256 = rounds * ((forward ? 23.0 : 15.0) + k / 110.0);
        if (t256 < t64 && t256 < t128) p.path = TILE256;
        else if (t128 < t64) p.path = TILE128;
        if (p.path != TILE) return p;
    }
    // few tiles over a long reduction: ranges of at least four steps, about
    // two workgroups per compute unit
    const int64_t steps = ceil_div(K, BK);
    if (p.tiles < 256 && steps >= 16) {
        int64_t split = ceil_div(512, p.tiles);
        if (split > steps / 4) split = steps / 4;
        if (split > 32) split = 32;
        p.split = int(split);
    }
    return p;
}

size_t part_bytes(const Plan &p, int64_t M, int64_t N) {
    return p.split > 1 ? (size_t(p.split) * M * N * sizeof(int32_t) + 15) & ~size_t(15) : 0;
}

Product make_product(const Plan &pl, const int8_t *A, int64_t lda, const int8_t *B, int64_t ldb, const Epi &ep,
                     int64_t M, int64_t N, int64_t K, void *part) {
    return Product{A,      B,      lda,      ldb, ep, int(M), int(N), int(K), pl.split, static_cast<int32_t *>(part),
                   int(pl.tiles * pl.split)};
}

template <class T, bool A_KM, bool B_KM, bool LINEAR>
void launch_tile256(const Product &p, hipStream_t st) {
    const int64_t tiles = ceil_div(p.M, 256) * ceil_div(p.N, 256);
    tile256_kernel<T, A_KM, B_KM, LINEAR><<<dim3(unsigned(tiles)), dim3(g256::NT), 0, st>>>(
        p.A, p.lda, p.B, p.ldb, uint32_t((A_KM ? p.M : p.K) * p.lda), uint32_t((B_KM ? p.N : p.K) * p.ldb), p.ep, p.M, p.N,
        p.K);
}

void as_tiles128(Product &p) { p.blocks = int(ceil_div(p.M, 128) * ceil_div(p.N, 128)); }

// The path a planned product takes with these operands.
Path path_of(const Plan &pl, const int8_t *A, const int8_t *B) {
    return (pl.path == TILE256 || pl.path == TILE128) && !(aligned(A, 16) && aligned(B, 16)) ? TILE : pl.path;
}

// (a plan of larger tiles that falls back to 64 x 64 tiles has that many of them)
void as_tiles(Product &p) { p.blocks = int(ceil_div(p.M, 64) * ceil_div(p.N, 64) * p.split); }

unsigned sum_groups(const Product &p) { return unsigned(ceil_div(int64_t(p.M) * ceil_div(p.N, 4), NT)); }

template <class T>
void launch_forward(const Plan &pl, Product p, hipStream_t st) {
    const Path path = path_of(pl, p.A, p.B);
    if (path == ROWS) {
        if (pl.rows == 1 && pl.cols == 1) launch_rows<T, 1, 1>(p, st);
        else if (pl.rows == 1) launch_rows<T, 1, 2>(p, st);
        else if (pl.rows == 2) launch_rows<T, 2, 2>(p, st);
        else launch_rows<T, 4, 2>(p, st);
    } else if (path == TILE256) {
        launch_tile256<T, true, true, false>(p, st);
    } else if (path == TILE128) {
        as_tiles128(p);
        tile128_kernel<T><<<dim3(unsigned(p.blocks)), dim3(NT), 0, st>>>(p);
    } else {
        as_tiles(p);
        const dim3 grid(unsigned(p.blocks)), block(NT);
        if (path == TINY) tile_kernel<T, 64, 64, 2, true, true, false, true><<<grid, block, 0, st>>>(p);
        else tile_kernel<T, 64, 64, 4, true, true, false, false><<<grid, block, 0, st>>>(p);
        if (p.split > 1) sum_kernel<T, false><<<dim3(sum_groups(p)), block, 0, st>>>(p);
    }
}

// dX's product d and G's g; one of blocks = 0 is not asked for.
template <class T>
void launch_backward(const Plan &pd, Product d, const Plan &pg, Product g, hipStream_t st) {
    if (d.blocks && path_of(pd, d.A, d.B) == TILE256) {
        launch_tile256<T, true, false, true>(d, st);
        d.blocks = 0;
    }
    if (g.blocks && path_of(pg, g.A, g.B) == TILE256) {
        launch_tile256<T, false, false, true>(g, st);
        g.blocks = 0;
    }
    const dim3 block(NT);
    const bool d128 = d.blocks && path_of(pd, d.A, d.B) == TILE128, g128 = g.blocks && path_of(pg, g.A, g.B) == TILE128;
    if (d128 || g128) {
        Product d2 = d, g2 = g;
        as_tiles128(d2);
        as_tiles128(g2);
        if (!d128) d2.blocks = 0;
        if (!g128) g2.blocks = 0;
        tile128_pair_kernel<T><<<dim3(unsigned(d2.blocks) + unsigned(g2.blocks)), block, 0, st>>>(d2, g2);
        if (d128) d.blocks = 0;
        if (g128) g.blocks = 0;
    }
    if (d.blocks && pd.path == TINY) {
        tile_kernel<T, 64, 64, 2, true, false, true, true><<<dim3(unsigned(d.blocks)), block, 0, st>>>(d);
        d.blocks = 0;
    }
    if (g.blocks && pg.path == TINY) {
        tile_kernel<T, 64, 64, 2, false, false, true, true><<<dim3(unsigned(g.blocks)), block, 0, st>>>(g);
        g.blocks = 0;
    }
    if (d.blocks) as_tiles(d);
    if (g.blocks) as_tiles(g);
    if (d.blocks + g.blocks == 0) return;
    tile_pair_kernel<T, 64, 64, 4><<<dim3(unsigned(d.blocks) + unsigned(g.blocks)), block, 0, st>>>(d, g);
    const unsigned sd = d.blocks && d.split > 1 ? sum_groups(d) : 0u, sg = g.blocks && g.split > 1 ? sum_groups(g) : 0u;
    if (sd + sg) sum_pair_kernel<T><<<dim3(sd + sg), block, 0, st>>>(d, g, int(sd));
}

// The workgroups of a product, on the path that it takes.
int64_t groups_of(const Plan &pl, const Product &p) {
    const Path path = path_of(pl, p.A, p.B);
    if (path == ROWS) return ceil_div(p.N, 16 * pl.cols);
    const int side = path == TILE256 ? 256 : path == TILE128 ? 128 : 64;
    return ceil_div(p.M, side) * ceil_div(p.N, side) * (side == 64 ? pl.split : 1);
}

// Whether their launches are within what the runtime takes.
bool launches(const Plan &pl, const Product &p) {
    return groups_of(pl, p) <= max_groups(path_of(pl, p.A, p.B) == ROWS ? kRowWaves * 64 : NT);
}
bool launches(const Plan &pd, const Product &d, const Plan &pg, const Product &g) {
    if (!d.blocks || !g.blocks) return (!d.blocks || launches(pd, d)) && (!g.blocks || launches(pg, g));
    const Path path = path_of(pd, d.A, d.B);
    if ((path == TILE || path == TILE128) && path == path_of(pg, g.A, g.B))  // in one grid
        return groups_of(pd, d) + groups_of(pg, g) <= max_groups(NT);
    return launches(pd, d) && launches(pg, g);
}

// (products whose tiles can be counted; twice: the two products of a backward
// pass share a grid)
bool tiles_ok(int64_t M, int64_t N) { return 2 * ceil_div(M, 64) * ceil_div(N, 64) <= 0x7fffffff; }

// edZ = 0 (and status 0) for an empty error; G and gb of an empty batch, dX
// of an empty layer.
__global__ void zero_bytes_kernel(uint8_t *p, int64_t n) {
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x)
        p[i] = 0;
}

void zero_bytes(void *p, int64_t n, hipStream_t st) {
    if (p == nullptr || n <= 0) return;
    const int64_t b = (n + 255) / 256;
    zero_bytes_kernel<<<dim3(unsigned(b < 2048 ? b : 2048)), dim3(256), 0, st>>>(static_cast<uint8_t *>(p), n);
}

}  // namespace
}  // namespace ionn

using namespace ionn;

extern "C" {

size_t dfp8_linear_fwd_workspace_bytes(int64_t B, int64_t IN, int64_t OUT) {
    if (!sizes_ok(B, IN, OUT) || B == 0 || OUT == 0) return 0;
    return part_bytes(make_plan<true, true>(B, OUT, IN, true), B, OUT);
}

int dfp8_linear_fwd(const int8_t *X, const int32_t *eX, const int8_t *W, const int32_t *eW, const float *bias, int act,
                    const void *residual, void *Z, void *Y, int dtype, int64_t B, int64_t IN, int64_t OUT,
                    uint32_t *absmax_Y, void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    IONN_REQUIRE(dtype_ok(dtype), IONN_ERR_ARG, "dfp8_linear_fwd: dtype = %d", dtype);
    IONN_REQUIRE(act >= IONN_ACT_NONE && act <= IONN_ACT_SILU, IONN_ERR_ARG, "dfp8_linear_fwd: act = %d", act);
    IONN_REQUIRE(sizes_ok(B, IN, OUT) && IN <= IONN_DFP8_MAX_REDUCTION && tiles_ok(B, OUT), IONN_ERR_SHAPE,
                 "dfp8_linear_fwd: B=%lld IN=%lld OUT=%lld (IN at most %d)", (long long)B, (long long)IN,
                 (long long)OUT, IONN_DFP8_MAX_REDUCTION);
    if (B == 0 || OUT == 0) return IONN_OK;
    IONN_REQUIRE(Y && eX && eW && (IN == 0 || (X && W)), IONN_ERR_ARG, "dfp8_linear_fwd: NULL tensor");
    IONN_REQUIRE(Z == nullptr || (Z != Y && Z != residual), IONN_ERR_ARG,
                 "dfp8_linear_fwd: Z must not be Y or the residual");
    const size_t es = dtype_size(dtype);
    IONN_REQUIRE(aligned(Y, es) && aligned(Z, es) && aligned(residual, es) && aligned(bias, 4) && aligned(eX, 4) &&
                     aligned(eW, 4) && aligned(absmax_Y, 4),
                 IONN_ERR_ALIGN, "dfp8_linear_fwd: tensors must be aligned to their element size");
    const size_t need = dfp8_linear_fwd_workspace_bytes(B, IN, OUT);
    IONN_REQUIRE(need == 0 || (workspace && aligned(workspace, 16) && workspace_bytes >= need), IONN_ERR_WORKSPACE,
                 "dfp8_linear_fwd: needs a 16-byte aligned workspace of %zu bytes", need);
    const Epi ep{eX, eW, bias, residual, Z, Y, absmax_Y, act};
    const Plan plan = make_plan<true, true>(B, OUT, IN, true);
    const Product p = make_product(plan, X, IN, W, IN, ep, B, OUT, IN, workspace);
    IONN_REQUIRE(launches(plan, p), IONN_ERR_SHAPE, "dfp8_linear_fwd: B=%lld OUT=%lld have too many tiles",
                 (long long)B, (long long)OUT);
    with_dtype(dtype, [&](auto tag) { launch_forward<decltype(tag)>(plan, p, as_stream(stream)); });
    return check_launch("dfp8_linear_fwd");
}

int dfp8_linear_path(int product, int64_t B, int64_t IN, int64_t OUT) {
    if (product < 0 || product > 2 || !sizes_ok(B, IN, OUT)) return -1;
    if (product == 0) return make_plan<true, true>(B, OUT, IN, true).path;
    return product == 1 ? make_plan<true, false>(B, IN, OUT, false).path : make_plan<false, false>(OUT, IN, B, false).path;
}

size_t dfp8_linear_bwd_workspace_bytes(int64_t B, int64_t IN, int64_t OUT) {
    if (!sizes_ok(B, IN, OUT) || B == 0 || OUT == 0) return 0;
    size_t n = act_workspace_bytes(B, OUT);
    if (IN > 0)
        n += part_bytes(make_plan<true, false>(B, IN, OUT, false), B, IN) +
             part_bytes(make_plan<false, false>(OUT, IN, B, false), OUT, IN);
    return n;
}

int dfp8_linear_bwd(const void *dY, const void *Z, int act, int dtype, const int8_t *X, const int32_t *eX,
                    const int8_t *W, const int32_t *eW, int8_t *dZ8, int32_t *edZ, void *dX, void *G, float *gb,
                    int64_t B, int64_t IN, int64_t OUT, int32_t *status_out, void *workspace, size_t workspace_bytes,
                    void *stream) {
    clear_error();
    IONN_REQUIRE(dtype_ok(dtype), IONN_ERR_ARG, "dfp8_linear_bwd: dtype = %d", dtype);
    IONN_REQUIRE(act >= IONN_ACT_NONE && act <= IONN_ACT_SILU, IONN_ERR_ARG, "dfp8_linear_bwd: act = %d", act);
    IONN_REQUIRE(sizes_ok(B, IN, OUT) && (dX == nullptr || OUT <= IONN_DFP8_MAX_REDUCTION) &&
                     (G == nullptr || B <= IONN_DFP8_MAX_REDUCTION) && tiles_ok(B, IN) && tiles_ok(OUT, IN) &&
                     tiles_ok(B, OUT),
                 IONN_ERR_SHAPE, "dfp8_linear_bwd: B=%lld IN=%lld OUT=%lld (OUT with dX, B with G: at most %d)",
                 (long long)B, (long long)IN, (long long)OUT, IONN_DFP8_MAX_REDUCTION);
    const bool error = B > 0 && OUT > 0;  // there is an error to go by
    IONN_REQUIRE(edZ && (!error || (dY && dZ8 && (Z || act == IONN_ACT_NONE))), IONN_ERR_ARG,
                 "dfp8_linear_bwd: NULL dY, Z, dZ8 or edZ");
    IONN_REQUIRE(!error || IN == 0 || ((dX == nullptr || (W && eW)) && (G == nullptr || (X && eX))), IONN_ERR_ARG,
                 "dfp8_linear_bwd: dX needs W and eW, G needs X and eX");
    const size_t es = dtype_size(dtype);
    IONN_REQUIRE(aligned(dY, es) && aligned(Z, es) && aligned(dX, es) && aligned(G, es) && aligned(gb, 4) &&
                     aligned(eX, 4) && aligned(eW, 4) && aligned(edZ, 4) && aligned(status_out, 4),
                 IONN_ERR_ALIGN, "dfp8_linear_bwd: tensors must be aligned to their element size");
    const size_t need = dfp8_linear_bwd_workspace_bytes(B, IN, OUT);
    IONN_REQUIRE(need == 0 || (workspace && aligned(workspace, 16) && workspace_bytes >= need), IONN_ERR_WORKSPACE,
                 "dfp8_linear_bwd: needs a 16-byte aligned workspace of %zu bytes", need);
    hipStream_t st = as_stream(stream);
    if (!error) {
        zero_bytes(edZ, 4, st);
        zero_bytes(status_out, 4, st);
        zero_bytes(dX, B * IN * int64_t(es), st);
        zero_bytes(G, OUT * IN * int64_t(es), st);
        zero_bytes(gb, OUT * 4, st);
        return check_launch("dfp8_linear_bwd");
    }
    char *parts = static_cast<char *>(workspace) + act_workspace_bytes(B, OUT);
    const Plan pd = make_plan<true, false>(B, IN, OUT, false), pg = make_plan<false, false>(OUT, IN, B, false);
    const Epi ed{edZ, eW, nullptr, nullptr, nullptr, dX, nullptr, IONN_ACT_NONE};
    const Epi eg{edZ, eX, nullptr, nullptr, nullptr, G, nullptr, IONN_ACT_NONE};
    Product d = make_product(pd, dZ8, OUT, W, IN, ed, B, IN, OUT, parts);
    Product g = make_product(pg, dZ8, OUT, X, IN, eg, OUT, IN, B, parts + part_bytes(pd, B, IN));
    if (!dX || IN == 0) d.blocks = 0;
    if (!G || IN == 0) g.blocks = 0;
    IONN_REQUIRE(launches(pd, d, pg, g), IONN_ERR_SHAPE, "dfp8_linear_bwd: B=%lld IN=%lld OUT=%lld have too many tiles",
                 (long long)B, (long long)IN, (long long)OUT);
    if (int rc = launch_act_bwd(dY, Z, act, dtype, B, OUT, dZ8, edZ, gb, status_out, workspace, st)) return rc;
    if (IN == 0) return IONN_OK;
    with_dtype(dtype, [&](auto tag) { launch_backward<decltype(tag)>(pd, d, pg, g, st); });
    return check_launch("dfp8_linear_bwd");
}

}  // extern "C"
