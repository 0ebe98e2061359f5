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
#include "dfp8_plan.h"

namespace ionn {
namespace {

using namespace dfp8;

template <class T, bool A_KM, bool B_KM, bool LINEAR>
void launch_tile256(const Product &p, hipStream_t st) {
    const int64_t tiles = ceil_div(p.M, 256) * ceil_div(p.N, 256);
    tile256_kernel<T, A_KM, B_KM, LINEAR><<<dim3(unsigned(tiles)), dim3(g256::NT), 0, st>>>(
        p.A, p.lda, p.B, p.ldb, uint32_t((A_KM ? p.M : p.K) * p.lda), uint32_t((B_KM ? p.N : p.K) * p.ldb), p.ep, p.M, p.N,
        p.K);
}

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

bool both_launch(const Plan &pd, const Product &d, const Plan &pg, const Product &g) {
    if (!d.blocks || !g.blocks) return (!d.blocks || launches(pd, d)) && (!g.blocks || launches(pg, g));
    const Path path = path_of(pd, d.A, d.B);
    if ((path == TILE || path == TILE128) && path == path_of(pg, g.A, g.B))  // in one grid
        return groups_of(pd, d) + groups_of(pg, g) <= max_groups(NT);
    return launches(pd, d) && launches(pg, g);
}

// The two products of a backward pass; one that is not asked for has no blocks.
struct Pair {
    Plan pd, pg;
    Product d, g;
};
Plan plan_of_dX(const BackwardSizes &s) { return make_plan<true, false>(s.B, s.IN, s.OUT, false, s.ldz, s.ldw); }
Plan plan_of_G(const BackwardSizes &s) { return make_plan<false, false>(s.OUT, s.IN, s.B, false, s.ldz, s.ldx); }
Pair make_pair(const BackwardProducts &p) {
    const int64_t B = p.s.B, IN = p.s.IN, OUT = p.s.OUT;
    Pair r;
    r.pd = plan_of_dX(p.s);
    r.pg = plan_of_G(p.s);
    const Epi ed{p.edZ, p.eW, nullptr, nullptr, nullptr, p.dX, nullptr, IONN_ACT_NONE};
    const Epi eg{p.edZ, p.eX, nullptr, nullptr, nullptr, p.G, nullptr, IONN_ACT_NONE};
    char *parts = static_cast<char *>(p.parts);
    r.d = make_product(r.pd, p.dZ8, p.s.ldz, p.W, p.s.ldw, ed, B, IN, OUT, parts);
    r.g = make_product(r.pg, p.dZ8, p.s.ldz, p.X, p.s.ldx, eg, OUT, IN, B, parts + part_bytes(r.pd, B, IN));
    if (!p.dX) r.d.blocks = 0;
    if (!p.G) r.g.blocks = 0;
    return r;
}

// edZ = 0 (and status 0) for an empty error; G and gb of an empty batch, dX
// of an empty layer.
__global__ void zero_bytes_kernel(uint8_t *p, int64_t n) {
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x)
        p[i] = 0;
}

}  // namespace

void zero_bytes(void *p, int64_t n, hipStream_t st) {
    if (p == nullptr || n <= 0) return;
    const int64_t b = (n + 255) / 256;
    zero_bytes_kernel<<<dim3(unsigned(b < 2048 ? b : 2048)), dim3(256), 0, st>>>(static_cast<uint8_t *>(p), n);
}

namespace dfp8 {

size_t backward_part_bytes(const BackwardSizes &s) {
    return part_bytes(plan_of_dX(s), s.B, s.IN) + part_bytes(plan_of_G(s), s.OUT, s.IN);
}

void backward_plans(const BackwardSizes &s, Plan &dX, Plan &G) {
    dX = plan_of_dX(s);
    G = plan_of_G(s);
}

bool backward_launches(const BackwardProducts &p) {
    const Pair r = make_pair(p);
    return both_launch(r.pd, r.d, r.pg, r.g);
}

void launch_backward_products(const BackwardProducts &p, int dtype, hipStream_t st) {
    const Pair r = make_pair(p);
    with_dtype(dtype, [&](auto tag) { launch_backward<decltype(tag)>(r.pd, r.d, r.pg, r.g, st); });
}

}  // namespace dfp8
}  // namespace ionn

using namespace ionn;
using namespace ionn::dfp8;

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
    if (IN > 0) n += backward_part_bytes({B, IN, OUT, OUT, IN, IN});
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
    const BackwardProducts p{dZ8, X, W, edZ, eX, eW, dX, G, {B, IN, OUT, OUT, IN, IN},
                             static_cast<char *>(workspace) + act_workspace_bytes(B, OUT)};
    IONN_REQUIRE(IN == 0 || backward_launches(p), IONN_ERR_SHAPE,
                 "dfp8_linear_bwd: B=%lld IN=%lld OUT=%lld have too many tiles", (long long)B, (long long)IN,
                 (long long)OUT);
    if (int rc = launch_act_bwd(dY, Z, act, dtype, B, OUT, dZ8, edZ, gb, status_out, workspace, st)) return rc;
    if (IN == 0) return IONN_OK;
    launch_backward_products(p, dtype, st);
    return check_launch("dfp8_linear_bwd");
}

}  // extern "C"
