// A Linear layer on DFP-8 operands (int8 mantissas, one shared exponent per
// tensor) with bias, activation and residual in the product's epilogue, and
// its backward pass ("Mixed Precision Training of Convolutional Neural
// Networks using Integer Operations", sections 3 and 4: integer products,
// the exponents added, the operations around them in floating point).
//
//   z = fl(X W^T) 2^(eX + eW) + bias,  Y = act(z) + residual
//   dZ = dY act'(Z) -> dZ8, edZ;  dX = fl(dZ8 W) 2^(edZ + eW),
//   G = fl(dZ8^T X) 2^(edZ + eX),  gb = column sums of dZ
#include "dfp8_convert.h"
#include "dfp8_rows.h"
#include "dfp8_tile256.h"

namespace ionn {
namespace {

using namespace dfp8;

constexpr int64_t kMaxSide = int64_t(1) << 30;

bool sizes_ok(int64_t B, int64_t IN, int64_t OUT) {
    return B >= 0 && IN >= 0 && OUT >= 0 && B <= kMaxSide && IN <= kMaxSide && OUT <= kMaxSide;
}

// C [M][N] of type `dtype` from the product over K; M, N >= 1.
template <bool A_KM, bool B_KM, bool LINEAR>
void launch_product(const int8_t *A, int64_t lda, const int8_t *B, int64_t ldb, const Epi &ep, int dtype, int M,
                    int N, int K, hipStream_t st) {
    const int64_t tiles = int64_t((M + 63) / 64) * ((N + 63) / 64);
    const int64_t tiles256 = int64_t((M + 255) / 256) * ((N + 255) / 256);
    with_dtype(dtype, [&](auto tag) {
        using T = decltype(tag);
        if constexpr (!LINEAR) {
            if (M <= kRowsMax && K >= kRowsMinK) {
                const dim3 grid(unsigned((N + 15) / 16)), block(kRowWaves * 64);
                if (M <= 16) rows_kernel<T, 1><<<grid, block, 0, st>>>(A, B, ep, M, N, K);
                else if (M <= 32) rows_kernel<T, 2><<<grid, block, 0, st>>>(A, B, ep, M, N, K);
                else rows_kernel<T, 4><<<grid, block, 0, st>>>(A, B, ep, M, N, K);
                return;
            }
        }
        if (tiles256 >= 64 && tile256_fits<A_KM, B_KM>(A, lda, B, ldb, M, N, K)) {
            tile256_kernel<T, A_KM, B_KM, LINEAR><<<dim3(unsigned(tiles256)), dim3(g256::NT), 0, st>>>(
                A, lda, B, ldb, uint32_t((A_KM ? M : K) * lda), uint32_t((B_KM ? N : K) * ldb), ep, M, N, K);
            return;
        }
        const int a_side = A_KM ? K : M, b_side = B_KM ? K : N;  // contiguous
        if (a_side < 16 || b_side < 16)
            tile_kernel<T, 64, 64, 2, A_KM, B_KM, LINEAR, true>
                <<<dim3(unsigned(tiles)), dim3(NT), 0, st>>>(A, lda, B, ldb, ep, M, N, K);
        else
            tile_kernel<T, 64, 64, 4, A_KM, B_KM, LINEAR, false>
                <<<dim3(unsigned(tiles)), dim3(NT), 0, st>>>(A, lda, B, ldb, ep, M, N, K);
    });
}

bool tiles_ok(int64_t M, int64_t N) { return ((M + 63) / 64) * ((N + 63) / 64) <= 0x7fffffff; }

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
    if (!sizes_ok(B, IN, OUT)) return 0;
    return 0;
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
    launch_product<true, true, false>(X, IN, W, IN, ep, dtype, int(B), int(OUT), int(IN), as_stream(stream));
    return check_launch("dfp8_linear_fwd");
}

size_t dfp8_linear_bwd_workspace_bytes(int64_t B, int64_t IN, int64_t OUT) {
    if (!sizes_ok(B, IN, OUT) || B == 0 || OUT == 0) return 0;
    return act_workspace_bytes(B, OUT);
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
    if (int rc = launch_act_bwd(dY, Z, act, dtype, B, OUT, dZ8, edZ, gb, status_out, workspace, st)) return rc;
    if (IN == 0) return IONN_OK;
    if (dX) {
        const Epi ep{edZ, eW, nullptr, nullptr, nullptr, dX, nullptr, IONN_ACT_NONE};
        launch_product<true, false, true>(dZ8, OUT, W, IN, ep, dtype, int(B), int(IN), int(OUT), st);
    }
    if (G) {
        const Epi ep{edZ, eX, nullptr, nullptr, nullptr, G, nullptr, IONN_ACT_NONE};
        launch_product<false, false, true>(dZ8, OUT, X, IN, ep, dtype, int(OUT), int(IN), int(B), st);
    }
    return check_launch("dfp8_linear_bwd");
}

}  // extern "C"
