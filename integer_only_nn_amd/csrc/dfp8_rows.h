// Forward product of few rows or few outputs (gfx950, v_mfma_i32_16x16x64_i8):
// tokens being generated, bound by reading W once, and small layers, bound by
// the trips to memory of one workgroup.
//
// A workgroup takes RG groups of 16 rows and NG groups of 16 outputs; its eight
// wavefronts split the reduction, each with 128 bytes of every row in flight
// while it multiplies the 128 before them, and their sums meet in LDS.  At 1 x
// 4096 x 4096 that is 256 workgroups and four trips a wavefront: 5.1 us, of
// which an empty launch in a graph is about 2 and W's 16.8 MB at the rate of a
// copy 3.2; 1 x 4096 x 32768 25 us, W at 5.3 TB/s.  256 x 784 x 256 2.7 us, 32 x
// 4096 x 4096 5.9.  512 bytes in flight instead of 128 are loads past the end
// where the reduction is short (16 x 1024 x 4096 4.4 against 3.3 us).  The
// weights are the first operand, so a lane ends with four consecutive outputs
// of one row.
#pragma once

#include "dfp8_tile.h"

namespace ionn {
namespace dfp8 {

constexpr int kRowWaves = 8;
constexpr int kRowsMinK = 16;

// K >= 16; RG groups of 16 rows, NG groups of 16 outputs.  GATED: N outputs of
// W's 2 N rows; the first NG / 2 groups are gate rows, the others the up rows of
// the same outputs.
template <class T, int RG, int NG, bool GATED = false>
__global__ __launch_bounds__(kRowWaves * 64) void rows_kernel(const int8_t *__restrict__ X, const int8_t *__restrict__ W,
                                                              Epi ep, int M, int N, int K) {
    constexpr int kDeep = 2;
    static_assert(RG * NG <= kRowWaves, "a wavefront for each group of sums");
    __shared__ v4i sums[RG * NG][kRowWaves][64];
    __shared__ v4i stage[kRowWaves][NG + RG][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    constexpr int NO = GATED ? NG / 2 : NG;  // groups of outputs
    static_assert(!GATED || NG % 2 == 0, "both halves of a group");
    const int n0 = int(blockIdx.x) * (16 * NO), m0 = int(blockIdx.y) * (16 * RG);
    // this wavefront's range of k: whole pieces of 64
    const int pieces = (K + 63) / 64, per = (pieces + kRowWaves - 1) / kRowWaves;
    const int k_begin = 64 * per * wave, k_end = min(K, k_begin + 64 * per);
    // Four lanes load 64 bytes of a row (loaded in the order of the operands,
    // neighbours in different rows, each lane is an access of its own: 16 x
    // 16384 x 256 16.1 us against 8.6), and LDS, private to the wavefront,
    // hands them to the lanes that multiply them: bytes 16 c .. of row r's piece
    // at position c ^ (r >> 2) of the row, which spreads 16 rows over the banks
    // (the counters still show 4 clocks of conflicts for each piece; another
    // order of the rows changed neither them nor the time).
    const int lr = lane >> 2, kl = 16 * (lane & 3);  // loads: row, bytes of the piece
    const int r = lane & 15;                         // multiplies: row
    const int put = 4 * lr + ((lane & 3) ^ (lr >> 2)), get = 4 * r + ((lane >> 4) ^ (r >> 2));
    // Every load is unconditional, so that all of them are in flight at once: a
    // row past the end repeats the last one (its sums are not stored), and a
    // piece past K - 16 is the row's last 16 bytes, of which W's copy keeps
    // only those no piece before it has counted.
    typedef v4i loose __attribute__((aligned(1)));
    const int8_t *w[NG], *x[RG];
#pragma unroll
    for (int h = 0; h < NG; ++h) w[h] = W + (int64_t(min(n0 + 16 * (h % NO) + lr, N - 1)) + int64_t(h / NO) * N) * K;
#pragma unroll
    for (int g = 0; g < RG; ++g) x[g] = X + int64_t(min(m0 + 16 * g + lr, M - 1)) * K;
    // what the epilogue needs besides the sums is loaded ahead of them: the
    // wavefront finishes rows m0 + 16 (wave % RG) .., outputs n0 + 16 (wave / RG) ..
    const int ea = *ep.ea, eb = *ep.eb, n = n0 + 16 * (wave / RG) + 4 * (lane >> 4);
    float bias[4] = {}, bias_up[4] = {};
    if (wave < RG * NO) {
        if (GATED) load_bias2(ep, n, N, bias, bias_up);
        else load_bias(ep, n, N, bias);
    }
    v4i acc[NG][RG];
#pragma unroll
    for (int h = 0; h < NG; ++h)
#pragma unroll
        for (int g = 0; g < RG; ++g) acc[h][g] = v4i{0, 0, 0, 0};
    struct Trip {
        v4i a[NG][kDeep], b[RG][kDeep];
    };
    const auto load = [&](Trip &t, int k0) __attribute__((always_inline)) {
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int k = min(k0 + 64 * d + kl, K - 16);
#pragma unroll
            for (int h = 0; h < NG; ++h) t.a[h][d] = *reinterpret_cast<const loose *>(w[h] + k);
#pragma unroll
            for (int g = 0; g < RG; ++g) t.b[g][d] = *reinterpret_cast<const loose *>(x[g] + k);
        }
    };
    const auto multiply = [&](Trip &t, int k0) __attribute__((always_inline)) {
        if (k0 + 64 * kDeep > k_end || k0 + 64 * kDeep > K) {
#pragma unroll
            for (int d = 0; d < kDeep; ++d) {
                const int k = k0 + 64 * d + kl;
                const int past = k0 + 64 * d < k_end ? max(0, k - (K - 16)) : 16;  // bytes to drop
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = past - 4 * i;
                    const int keep = int(p <= 0 ? ~0u : (p >= 4 ? 0u : ~0u << (8 * p)));
#pragma unroll
                    for (int h = 0; h < NG; ++h) t.a[h][d][i] &= keep;
                }
            }
        }
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
#pragma unroll
            for (int h = 0; h < NG; ++h) stage[wave][h][put] = t.a[h][d];
#pragma unroll
            for (int g = 0; g < RG; ++g) stage[wave][NG + g][put] = t.b[g][d];
            in_order();
            v4i a[NG], b[RG];
#pragma unroll
            for (int h = 0; h < NG; ++h) a[h] = stage[wave][h][get];
#pragma unroll
            for (int g = 0; g < RG; ++g) b[g] = stage[wave][NG + g][get];
            in_order();
#pragma unroll
            for (int h = 0; h < NG; ++h)
#pragma unroll
                for (int g = 0; g < RG; ++g)
                    acc[h][g] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[h], b[g], acc[h][g], 0, 0, 0);
        }
    };
    if (k_begin < k_end) {
        constexpr int kStep = 64 * kDeep;
        Trip t0, t1;
        load(t0, k_begin);
        for (int k0 = k_begin; k0 < k_end; k0 += 2 * kStep) {
            if (k0 + kStep < k_end) load(t1, k0 + kStep);
            multiply(t0, k0);
            if (k0 + kStep >= k_end) break;
            if (k0 + 2 * kStep < k_end) load(t0, k0 + 2 * kStep);
            multiply(t1, k0 + kStep);
        }
    }
#pragma unroll
    for (int h = 0; h < NG; ++h)
#pragma unroll
        for (int g = 0; g < RG; ++g) sums[h * RG + g][wave][lane] = acc[h][g];
    __syncthreads();
    if (wave >= RG * NO) return;
    v4i s = sums[wave][0][lane];
#pragma unroll
    for (int o = 1; o < kRowWaves; ++o) s += sums[wave][o][lane];
    const int e2 = ea + eb;
    uint32_t top = 0;
    if constexpr (GATED) {
        v4i u = sums[RG * NO + wave][0][lane];
#pragma unroll
        for (int o = 1; o < kRowWaves; ++o) u += sums[RG * NO + wave][o][lane];
        with_act(ep.act, [&](auto ac) __attribute__((always_inline)) {
            top = finish_gated4<T, decltype(ac)::value>(s, u, ep, e2, bias, bias_up, m0 + 16 * (wave % RG) + r, n, M, N);
        });
    } else with_act(ep.act, [&](auto ac) __attribute__((always_inline)) {
        top = finish4<T, decltype(ac)::value, false>(s, ep, e2, bias, m0 + 16 * (wave % RG) + r, n, M, N);
    });
    if (ep.absmax) {
        top = wave_max_u32(top);
        if (lane == 0) publish_max_u32(ep.absmax, top);
    }
}

template <class T, int RG, int NG, bool GATED = false>
void launch_rows(const Product &p, hipStream_t st) {
    constexpr int kCols = 16 * (GATED ? NG / 2 : NG);
    const dim3 grid(unsigned((p.N + kCols - 1) / kCols), unsigned((p.M + 16 * RG - 1) / (16 * RG)));
    rows_kernel<T, RG, NG, GATED><<<grid, dim3(kRowWaves * 64), 0, st>>>(p.A, p.B, p.ep, p.M, p.N, p.K);
}

}  // namespace dfp8
}  // namespace ionn
