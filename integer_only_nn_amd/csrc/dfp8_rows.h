// Forward product of up to 16 rows (tokens being generated): bound by reading
// W once, so W goes straight from memory into matrix-core operands and nothing
// of it through LDS (gfx950, v_mfma_i32_16x16x64_i8).
//
// A workgroup takes 16 outputs; its eight wavefronts split the reduction, each
// with kDeep pieces of 16 rows x 64 bytes of W in flight, and their sums meet
// in LDS.  At 1 x 4096 x 4096 that is 256 workgroups whose wavefronts load
// all they need of W in one go, one trip to memory: 5.7 us, of which a launch
// in a graph is 3.3 and W's 16.8 MB at the rate of a copy 3.2; 1 x 4096 x 32768
// reads W at 4.6 TB/s.  The weights are the first operand, so a lane ends with
// four consecutive outputs of one row.
#pragma once

#include "dfp8_tile.h"

namespace ionn {
namespace dfp8 {

constexpr int kRowWaves = 8;
constexpr int kRowsMax = 16;  // rows of X
constexpr int kRowsMinK = 16;

// K >= 16.
template <class T>
__global__ __launch_bounds__(kRowWaves * 64) void rows_kernel(const int8_t *__restrict__ X, const int8_t *__restrict__ W,
                                                              Epi ep, int M, int N, int K) {
    constexpr int kDeep = 8;
    __shared__ v4i sums[kRowWaves][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int n0 = int(blockIdx.x) * 16;
    // this wavefront's range of k: whole pieces of 64
    const int pieces = (K + 63) / 64, per = (pieces + kRowWaves - 1) / kRowWaves;
    const int k_begin = 64 * per * wave, k_end = min(K, k_begin + 64 * per);
    const int r = lane & 15, kl = 16 * (lane >> 4);
    // Every load is unconditional, so that all of them are in flight at once: a
    // row past the end repeats the last one (its sums are not stored), and a
    // piece past K - 16 is the row's last 16 bytes, of which X's copy keeps
    // only those no piece before it has counted.
    typedef v4i loose __attribute__((aligned(1)));
    const int8_t *w = W + int64_t(min(n0 + r, N - 1)) * K;
    const int8_t *x = X + int64_t(min(r, M - 1)) * K;
    // what the epilogue needs besides the sums is loaded ahead of them
    const int ea = *ep.ea, eb = *ep.eb, n = n0 + 4 * (lane >> 4);
    float bias[4];
    load_bias(ep, n, N, bias);
    v4i acc = {0, 0, 0, 0};
    for (int k0 = k_begin; k0 < k_end; k0 += 64 * kDeep) {
        v4i a[kDeep], b[kDeep];
#pragma unroll
        for (int d = 0; d < kDeep; ++d) a[d] = *reinterpret_cast<const loose *>(w + min(k0 + 64 * d + kl, K - 16));
#pragma unroll
        for (int d = 0; d < kDeep; ++d) b[d] = *reinterpret_cast<const loose *>(x + min(k0 + 64 * d + kl, K - 16));
        if (k0 + 64 * kDeep > k_end || k0 + 64 * kDeep > K) {
#pragma unroll
            for (int d = 0; d < kDeep; ++d) {
                const int k = k0 + 64 * d + kl;
                const int past = k0 + 64 * d < k_end ? max(0, k - (K - 16)) : 16;  // bytes to drop
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = past - 4 * i;
                    b[d][i] &= int(p <= 0 ? ~0u : (p >= 4 ? 0u : ~0u << (8 * p)));
                }
            }
        }
#pragma unroll
        for (int d = 0; d < kDeep; ++d) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[d], b[d], acc, 0, 0, 0);
    }
    sums[wave][lane] = acc;
    __syncthreads();
    if (wave > 0) return;
    v4i s = sums[0][lane];
#pragma unroll
    for (int o = 1; o < kRowWaves; ++o) s += sums[o][lane];
    const int e2 = ea + eb;
    uint32_t top = 0;
    with_act(ep.act, [&](auto ac) __attribute__((always_inline)) {
        top = finish4<T, decltype(ac)::value, false>(s, ep, e2, bias, r, n, M, N);
    });
    if (ep.absmax) {
        top = wave_max_u32(top);
        if (lane == 0) publish_max_u32(ep.absmax, top);
    }
}

}  // namespace dfp8
}  // namespace ionn
