// The middle sizes of the DFP-8 Linear layer: 128 x 128 output tiles on the
// conditions of dfp8_tile256.h (row pitches and addresses in multiples of 16),
// for products that 256 x 256 tiles would leave most compute units without.
//
// Four wavefronts (2 x 2) of 64 x 64 outputs; a 128-deep K step is 32 KiB,
// loaded straight into one of kStages LDS stages (buffer_load ... lds, eight
// instructions a wavefront), so that kStages - 1 steps are in flight and no
// register holds them.  A wavefront waits for its own loads of the step it
// needs (they return in order) and all meet at one barrier a step, behind which
// the stage read last is loaded again.  Two stages, so that two workgroups share
// a compute unit and one's epilogue overlaps the other's products: 2048 x 4096 x
// 4096 42 us forward (1640 TOP/s) against 49 with four stages and one
// workgroup, though 256 tiles alone would rather have four (4096 x 4096 x 1024,
// 27.4 against 25.3).  Bound by what LDS takes in and gives out: a step moves
// 32 KiB into it and 64 KiB out for 512 clocks of the matrix cores.
//
// Layouts: K-major [128 rows][128 B], 16-byte piece c of row r at position
// c ^ fK(r & 15); M-major [128 k][128 B], piece c of row k at c ^ fT(k).  An
// instruction writes eight whole rows, its lanes load the pieces that belong
// there.  Edges as in dfp8_tile256.h: what lies past an operand's end is past
// its buffer resource and comes back as zeros, and where both operands are
// K-major A's pieces past K are sent out of range.
#pragma once

#include "dfp8_tile256.h"

namespace ionn {
namespace dfp8 {

template <bool KMAJOR>
struct Src128 {
    v4i rsrc;
    uint32_t off[4];  // of the lane's piece in each of the wavefront's four instructions, at k = 0
    int col[2];       // K-major: its first k, by the instruction's parity
    uint32_t step;    // bytes from one K step to the next
    __device__ __forceinline__ void init(const int8_t *b, int ld, uint32_t bytes, int r0, int wave, int lane) {
        const uint64_t a = uint64_t(uintptr_t(b));
        rsrc = v4i{__builtin_amdgcn_readfirstlane(int(uint32_t(a))),
                   __builtin_amdgcn_readfirstlane(int(uint32_t(a >> 32) & 0xffffu)),  // stride 0
                   __builtin_amdgcn_readfirstlane(int(bytes)),                        // size
                   0x00020000};
        const int sub = lane >> 3, at = lane & 7;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int row = 8 * (4 * wave + q) + sub;
            if (KMAJOR) {
                col[q & 1] = 16 * (at ^ g256::fK(row & 15));
                off[q] = uint32_t(r0 + row) * uint32_t(ld) + uint32_t(col[q & 1]);
            } else {
                off[q] = uint32_t(row) * uint32_t(ld) + uint32_t(r0 + 16 * (at ^ fT<128>(row)));
            }
        }
        step = KMAJOR ? uint32_t(BK) : uint32_t(BK) * uint32_t(ld);
    }
    // step kt to LDS (a step past the last, and with MASK the pieces past K, out of range)
    template <bool MASK>
    __device__ __forceinline__ void load(int kt, int K, uint32_t lds, int wave) const {
        const uint32_t ko = uint32_t(kt) * step;
        const int left = K - kt * BK;
        uint32_t v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = left > (MASK && KMAJOR ? col[q & 1] : 0) ? off[q] + ko : kOut;
        const uint32_t to = lds + uint32_t(wave) * 4096u;
#pragma unroll
        for (int q = 0; q < 4; ++q) g256::dma16(rsrc, v[q], 0u, to + 1024u * uint32_t(q));
    }
};

// vmcnt(n) lgkmcnt(0) and the barrier, with no memory operation moved across
template <int VM>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((VM & 15) | (7 << 4) | ((VM >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

constexpr int kStages = 2;
constexpr int kStage128 = 2 * 128 * BK;

// Tile id of a product.
template <class T, bool A_KM, bool B_KM, bool LINEAR>
__device__ __forceinline__ void run_tile128(const Product &p, int id, int8_t *lds) {
    constexpr bool MASK = A_KM && B_KM;
    const int M = p.M, N = p.N, K = p.K;
    const Epi &ep = p.ep;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int wm = 64 * (wave >> 1), wn = 64 * (wave & 1);
    int tm, tn;
    gemm::tile_coords(id, (M + 127) / 128, (N + 127) / 128, tm, tn);
    const int m0 = tm * 128, n0 = tn * 128;
    Src128<A_KM> sa;
    Src128<B_KM> sb;
    sa.init(p.A, int(p.lda), uint32_t((A_KM ? M : K) * p.lda), m0, wave, lane);
    sb.init(p.B, int(p.ldb), uint32_t((B_KM ? N : K) * p.ldb), n0, wave, lane);
    const uint32_t base = g256::lds_addr(lds);
    const int e2 = *ep.ea + *ep.eb;
    v16i acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = v16i{};
    const int nk = (K + BK - 1) / BK;
    const auto load = [&](int kt) __attribute__((always_inline)) {
        const uint32_t to = base + uint32_t(kt % kStages) * uint32_t(kStage128);
        sa.template load<MASK>(kt, K, to, wave);
        sb.template load<MASK>(kt, K, to + 128 * BK, wave);
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) load(s);
    for (int kt = 0; kt < nk; ++kt) {
        wait_and_meet<8 * (kStages - 2)>();
        load(kt + kStages - 1);
        const int8_t *As = lds + (kt % kStages) * kStage128, *Bs = As + 128 * BK;
#pragma unroll
        for (int sl = 0; sl < BK / 32; ++sl) {
            v4i a[2], b[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) a[i] = read_frag<128, A_KM>(As, wm + 32 * i, sl, lane);
#pragma unroll
            for (int j = 0; j < 2; ++j) b[j] = read_frag<128, B_KM>(Bs, wn + 32 * j, sl, lane);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[j], a[i], acc[i][j], 0, 0, 0);
        }
    }
    // no load of this kernel is in flight any more and every wavefront is done with the stages: 16 KiB for each
    wait_and_meet<0>();
    v4i *buf = reinterpret_cast<v4i *>(lds) + 1024 * wave;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const v16i &s = acc[i][j];
                const int r = 32 * i + (lane & 31), c = 8 * j + 2 * q + (lane >> 5);
                buf[16 * r + (c ^ (r & 15))] = v4i{s[4 * q], s[4 * q + 1], s[4 * q + 2], s[4 * q + 3]};
            }
    const int c = 2 * (lane & 7), n = n0 + wn + 8 * (lane & 7);
    float bias[8] = {};
    if (!LINEAR) load_bias(ep, n, N, bias);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the wavefront's own writes
    __builtin_amdgcn_wave_barrier();
    uint32_t top = 0;
    with_act(LINEAR ? int(IONN_ACT_NONE) : ep.act, [&](auto ac) __attribute__((always_inline)) {
#pragma unroll 2
        for (int k = 0; k < 8; ++k) {
            const int r = 8 * k + (lane >> 3);
            const v4i lo = buf[16 * r + (c ^ (r & 15))], hi = buf[16 * r + ((c + 1) ^ (r & 15))];
            top = max(top, finish8<T, decltype(ac)::value, LINEAR>(lo, hi, ep, e2, bias, int64_t(m0) + wm + r, n, M, N));
        }
    });
    if (!LINEAR && ep.absmax) {
        top = wave_max_u32(top);
        if (lane == 0) publish_max_u32(ep.absmax, top);
    }
}

template <class T>
__global__ __launch_bounds__(NT) void tile128_kernel(Product p) {
    __shared__ __attribute__((aligned(1024))) int8_t lds[kStages * kStage128];
    run_tile128<T, true, true, false>(p, int(blockIdx.x), lds);
}

// dX's product d and G's g in one grid, where each alone is a single round (2048^3:
// 44 us for the backward pass in two launches, 38 in one; one of blocks = 0 is not
// asked for).
template <class T>
__global__ __launch_bounds__(NT) void tile128_pair_kernel(Product d, Product g) {
    __shared__ __attribute__((aligned(1024))) int8_t lds[kStages * kStage128];
    const int id = int(blockIdx.x);
    if (id < d.blocks) run_tile128<T, true, false, true>(d, id, lds);
    else run_tile128<T, false, false, true>(g, id - d.blocks, lds);
}

}  // namespace dfp8
}  // namespace ionn
