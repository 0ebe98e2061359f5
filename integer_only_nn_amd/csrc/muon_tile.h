// Products of matrices held as pairs of float16 terms, for the orthogonalisation
// of an update (muon.hip): float32-like precision on the float16 matrix cores
// (gfx950, v_mfma_f32_32x32x16_f16).
//
// A value x is hi + lo, hi = fl16(x), lo = fl16(x - hi): 22 bits.  A product is
// hi hi + hi lo + lo hi (lo lo is below float32's last bit), three matrix
// instructions where a float32 product of the library takes the time of nine.  32 values of a row
// lie as 64 bytes of hi and 64 of lo, so that a 128-byte K step of the int8
// kernels' loaders (gemm256.h, dfp8_tile128.h) brings both terms of both operands
// and LDS hands out each fragment once for three products.
//
// Both operands are K-major, their rows padded with zeros to whole tiles, so no
// edge is checked.  A product is blocks of up to eight neighbouring tiles of S
// double steps (64 values of K) each; lanes of as many workgroups take runs of
// `chunk` double steps of the sequence of blocks, across blocks, a workgroup one
// tile of each, and leave each piece's float32 sums in a slot of their own in the
// order of the registers.  So all compute units end together, and a lane's
// workgroups, on one XCD, are at the same place of K and find each other's operands
// in its L2: A of 4096 x 4096 reads 0.44 GB, in runs of single tiles 1.03 (a step
// 3771 against 3830 us, of 4096 x 11008 8258 against 8601).  The pass that follows
// adds a tile's pieces in order (muon.hip), so which workgroup took what decides the
// rounding and nothing else does.
#pragma once

#include "dfp8_tile128.h"

namespace ionn {
namespace muon {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

// C = A B^T by tiles, A [rows][K] and B [cols][K] pairs (4 K bytes a row).
struct Work {
    const int8_t *A, *B;
    float *part;            // [lanes][width][slots][side * side]
    int rows, cols, K;      // rows, cols in tiles' sides, K in 64
    int tri;                // the lower triangle of tiles alone (rows = cols)
    int tiles, S, width;    // width: tiles of a block, workgroups of a lane: 8, 4, 2 or 1
    int chunk, slots, lanes, groups;
};

// Tile t's row and column: in the triangle two rows at a time, else four
// (neighbours in t share operands).
__host__ __device__ __forceinline__ void tile_at(const Work &w, int side, int t, int &ti, int &tj) {
    if (w.tri) {
        // the pair of rows 2 i and 2 i + 1 begins at tile 2 i^2 + i
        int i = int((sqrtf(8.0f * float(t) + 1.0f) - 1.0f) * 0.25f);
        while (2 * i * i + i > t) --i;
        while (2 * (i + 1) * (i + 1) + i + 1 <= t) ++i;
        const int r = t - (2 * i * i + i);
        if (2 * i + 1 == w.rows / side) {  // a last row alone
            ti = 2 * i;
            tj = r;
        } else if (r < 4 * i + 2) {
            ti = 2 * i + (r & 1);
            tj = r >> 1;
        } else {
            ti = tj = 2 * i + 1;
        }
        return;
    }
    const int tm = w.rows / side, tn = w.cols / side, group = t / (4 * tn), first = 4 * group;
    const int size = tm - first < 4 ? tm - first : 4, local = t - group * 4 * tn;
    ti = first + local % size;
    tj = local / size;
}

__device__ __forceinline__ v16f mfma(const v4i &b, const v4i &a, const v16f &c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, b), __builtin_bit_cast(v8h, a), c, 0, 0, 0);
}

// A wavefront's sums to its share of a slot, [i][j][q][lane] of four values.
template <int F>
__device__ __forceinline__ void leave(const v16f (&acc)[F][F], float *to, int lane) {
    v4f *p = reinterpret_cast<v4f *>(to) + lane;
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const v16f &a = acc[i][j];
                p[64 * ((i * F + j) * 4 + q)] = v4f{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
            }
}

// ---- tiles of 128 ----------------------------------------------------------------

// Steps [k0, k1) of tile (ti, tj).
__device__ __forceinline__ void piece128(const Work &w, int ti, int tj, int k0, int k1, float *to, int8_t *lds) {
    using namespace dfp8;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int wm = 64 * (wave >> 1), wn = 64 * (wave & 1), m0 = 128 * ti, n0 = 128 * tj, ld = 4 * w.K;
    Src128<true> sa, sb;
    sa.init(w.A, ld, uint32_t(w.rows) * uint32_t(ld), m0, m0 + 32 * wave, wave, lane);
    sb.init(w.B, ld, uint32_t(w.cols) * uint32_t(ld), n0, n0 + 32 * wave, wave, lane);
    const uint32_t base = g256::lds_addr(lds);
    v16f acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = v16f{};
    const auto load = [&](int kt, int stage) __attribute__((always_inline)) {
        const uint32_t at = base + uint32_t(stage) * uint32_t(kStage128);
        sa.template load<false>(kt, ld, at, wave);
        sb.template load<false>(kt, ld, at + 128 * BK, wave);
    };
    load(k0, 0);
    for (int kt = k0; kt < k1; ++kt) {
        const int stage = (kt - k0) & 1;
        wait_and_meet<0>();
        if (kt + 1 < k1) load(kt + 1, stage ^ 1);
        const int8_t *As = lds + stage * kStage128, *Bs = As + 128 * BK;
        // slices 0 and 1: the high terms of 16 values each, 2 and 3: the low ones
        v4i a[4][2], b[4][2];
#pragma unroll
        for (int sl = 0; sl < 4; ++sl)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[sl][i] = read_frag<128, true>(As, wm + 32 * i, sl, lane);
                b[sl][i] = read_frag<128, true>(Bs, wn + 32 * i, sl, lane);
            }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < 3; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = mfma(b[t == 1 ? 2 + h : h][j], a[t == 2 ? 2 + h : h][i], acc[i][j]);
    }
    leave<2>(acc, to + wave * 4096, lane);
    wait_and_meet<0>();  // the next piece loads over the stages
}

// ---- small tiles -------------------------------------------------------------------

// A tile of 32 F x 32 F by a workgroup of W wavefronts that split the reduction:
// each loads its own 32 values of K at a time, straight into LDS that no other
// wavefront uses (two stages, no barrier), and their sums meet in LDS.  For
// matrices of which tiles of 128 would be few: a product is then about one trip to
// memory, and its epilogue is in the same launch: 784-256-128-10 takes 88 us a step,
// by tiles of 128 and their pieces 243.  (Through registers, four steps in flight,
// 512 x 512 took 106 us against the 101 of its time, 92 today.)
template <int F, int W>
constexpr int kSmallLds = W * 2 * 2 * 32 * F * 128;

// The sums of a wavefront's share of K, of tile (ti, tj).
template <int F, int W>
__device__ __forceinline__ void sums_small(const Work &w, int ti, int tj, int8_t *lds, v16f (&acc)[F][F]) {
    using namespace dfp8;
    constexpr int kOperand = 32 * F * 128, kStage = 2 * kOperand;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int ld = 4 * w.K, steps = w.K / 32, per = (steps + W - 1) / W, k0 = wave * per, k1 = min(steps, k0 + per);
    const auto rsrc = [&](const int8_t *b, int rows) __attribute__((always_inline)) {
        const uint64_t a = uint64_t(uintptr_t(b));
        return v4i{__builtin_amdgcn_readfirstlane(int(uint32_t(a))),
                   __builtin_amdgcn_readfirstlane(int(uint32_t(a >> 32) & 0xffffu)),
                   __builtin_amdgcn_readfirstlane(int(uint32_t(rows) * uint32_t(ld))), 0x00020000};
    };
    const v4i ra = rsrc(w.A, w.rows), rb = rsrc(w.B, w.cols);
    // an instruction takes eight rows of 128 bytes; piece c of row r lies at c ^ fK(r & 15)
    const int sub = lane >> 3, at = lane & 7;
    uint32_t off[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) off[p] = uint32_t(sub) * uint32_t(ld) + 16u * uint32_t(at ^ g256::fK(8 * p + sub));
    const uint32_t base = g256::lds_addr(lds) + uint32_t(wave) * uint32_t(2 * kStage);
    const auto load = [&](int k) __attribute__((always_inline)) {
        const uint32_t to = base + uint32_t((k - k0) & 1) * uint32_t(kStage), kb = 128u * uint32_t(k);
#pragma unroll
        for (int q = 0; q < 4 * F; ++q)
            g256::dma16(ra, off[q & 1] + uint32_t(32 * F * ti + 8 * q) * uint32_t(ld) + kb, 0u, to + 1024u * uint32_t(q));
#pragma unroll
        for (int q = 0; q < 4 * F; ++q)
            g256::dma16(rb, off[q & 1] + uint32_t(32 * F * tj + 8 * q) * uint32_t(ld) + kb, 0u,
                        to + uint32_t(kOperand) + 1024u * uint32_t(q));
    };
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = v16f{};
    if (k0 < k1) load(k0);
    for (int k = k0; k < k1; ++k) {
        // the stage that the next step goes to has been read (lgkmcnt(0)); then this step's loads are in
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xc07f);
        if (k + 1 < k1) {
            load(k + 1);
            __builtin_amdgcn_s_waitcnt(((8 * F) & 15) | (7 << 4) | (15 << 8) | (((8 * F) >> 4) << 14));  // vmcnt(8 F)
        } else {
            __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));  // vmcnt(0)
        }
        asm volatile("" ::: "memory");
        const int8_t *As = lds + wave * (2 * kStage) + ((k - k0) & 1) * kStage, *Bs = As + kOperand;
        v4i a[4][F], b[4][F];
#pragma unroll
        for (int sl = 0; sl < 4; ++sl)
#pragma unroll
            for (int i = 0; i < F; ++i) {
                a[sl][i] = read_frag<32 * F, true>(As, 32 * i, sl, lane);
                b[sl][i] = read_frag<32 * F, true>(Bs, 32 * i, sl, lane);
            }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < 3; ++t)
#pragma unroll
                for (int i = 0; i < F; ++i)
#pragma unroll
                    for (int j = 0; j < F; ++j)
                        acc[i][j] = mfma(b[t == 1 ? 2 + h : h][j], a[t == 2 ? 2 + h : h][i], acc[i][j]);
    }
}

// The tile's sums of all wavefronts: rows of 32 F + 4 floats in LDS, one tile for
// each wavefront, so that a thread adds up neighbouring values of a row.  (The pad
// spreads the rows of a column over the banks.)
template <int F>
constexpr int kSmallPitch = 32 * F + 4;
template <int F>
constexpr int kSmallTile = 32 * F * kSmallPitch<F>;

template <int F>
__device__ __forceinline__ void lay_small(const v16f (&acc)[F][F], float *lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float *to = lds + wave * kSmallTile<F> + (lane & 31) * kSmallPitch<F> + 4 * (lane >> 5);
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const v16f &a = acc[i][j];
                *reinterpret_cast<v4f *>(to + 32 * i * kSmallPitch<F> + 32 * j + 8 * q) =
                    v4f{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
            }
}

// ---- tiles of 256 ----------------------------------------------------------------

// The fragments of 16 values of K: both terms of a wavefront's four row blocks of each operand.
struct Terms {
    v4i a[2][4], b[2][4];  // [term]
    __device__ __forceinline__ void read(int idx, const int8_t *As, const int8_t *Bs, const g256::FragSrc<true> &fa,
                                         const g256::FragSrc<true> &fb, int sl) {
        const int term = idx >> 3, i = idx & 3;
        if (idx & 4) b[term][i] = fb.read(Bs, i, sl + 2 * term);
        else a[term][i] = fa.read(As, i, sl + 2 * term);
    }
};

// Product t (0 .. 47) of 16 values of K: hi hi, then hi lo, then lo hi, each over the 4 x 4 blocks.
__device__ __forceinline__ void product(const Terms &f, int t, v16f (&acc)[4][4]) {
    const int term = t >> 4, i = (t >> 2) & 3, j = t & 3;
    acc[i][j] = mfma(f.b[term == 1][j], f.a[term == 2][i], acc[i][j]);
}

// Steps [k0, k1) of tile (ti, tj), an even number of them, on the operand layouts
// and in the manner of gemm256.h: four wavefronts of 128 x 128, two LDS stages of
// 64 KiB, a step's second half of fragments read while its first half multiplies,
// and the next step's first half behind the barrier in the middle of the second.
__device__ __forceinline__ void piece256(const Work &w, int ti, int tj, int k0, int k1, float *to, int8_t *sA0,
                                         int8_t *sB0, int8_t *sA1, int8_t *sB1) {
    using namespace g256;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int wm = wave >> 1, wn = wave & 1, ld = 4 * w.K;
    TileSrc<true> ta, tb;
    ta.init(w.A, ld, uint32_t(w.rows) * uint32_t(ld), 256 * ti, wave, lane);
    tb.init(w.B, ld, uint32_t(w.cols) * uint32_t(ld), 256 * tj, wave, lane);
    FragSrc<true> fa, fb;
    fa.init(wm * 128, lane);
    fb.init(wn * 128, lane);
    v16f acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v16f{};
    Terms F[2];
    // load pair q (0 .. 7) of step kt
    const auto dma = [&](int q, int kt, int8_t *Ad, int8_t *Bd) __attribute__((always_inline)) {
        if (q < 4) ta.issue_two(kt * g256::BK, Ad, wave, 2 * q);
        else tb.issue_two(kt * g256::BK, Bd, wave, 2 * (q - 4));
    };
#pragma unroll
    for (int q = 0; q < 8; ++q) dma(q, k0, sA0, sB0);
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    dma(0, k0 + 1, sA1, sB1);
    dma(1, k0 + 1, sA1, sB1);
#pragma unroll
    for (int r = 0; r < 16; ++r) F[0].read(r, sA0, sB0, fa, fb, 0);
    const auto step = [&](const int8_t *Ac, const int8_t *Bc, int8_t *An, int8_t *Bn, int kt) __attribute__((always_inline)) {
        const bool more1 = kt + 1 < k1, more2 = kt + 2 < k1;
#pragma unroll
        for (int t = 0; t < 48; ++t) {
            product(F[0], t, acc);
            IONN_SCHED_FENCE();
            if (t % 3 == 0) F[1].read(t / 3, Ac, Bc, fa, fb, 1);
            if (t % 4 == 1 && t / 4 < 6) {
                if (more1) dma(2 + t / 4, kt + 1, An, Bn);
            }
            IONN_SCHED_FENCE();
        }
#pragma unroll
        for (int t = 0; t < 30; ++t) product(F[1], t, acc);
        IONN_SCHED_FENCE();
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        IONN_SCHED_FENCE();
#pragma unroll
        for (int t = 30; t < 48; ++t) {
            product(F[1], t, acc);
            IONN_SCHED_FENCE();
            if (t - 30 < 16) F[0].read(t - 30, An, Bn, fa, fb, 0);
            if (t == 36 || t == 42) {
                if (more2) dma(t == 36 ? 0 : 1, kt + 2, const_cast<int8_t *>(Ac), const_cast<int8_t *>(Bc));
            }
            IONN_SCHED_FENCE();
        }
    };
    for (int kt = k0; kt < k1; kt += 2) {
        step(sA0, sB0, sA1, sB1, kt);
        step(sA1, sB1, sA0, sB0, kt + 1);
    }
    leave<4>(acc, to + wave * 16384, lane);
    __builtin_amdgcn_s_waitcnt(0x0070);
    __builtin_amdgcn_s_barrier();  // the next piece loads over the stages
}

// The pieces of workgroup g of a product: piece(tile row, tile column, first step, last step, slot).
template <int SIDE, class F>
__device__ __forceinline__ void pieces(const Work &w, int g, F &&piece) {
    // (workgroups go to the XCDs in turn: those of a lane to one, neighbouring lanes too)
    const int turn = g >> 3, lane = (g & 7) * (w.groups / (8 * w.width)) + turn / w.width, q = turn % w.width;
    const int total = (w.tiles + w.width - 1) / w.width * w.S;
    int at = lane * w.chunk, slot = 0;
    const int end = min(total, at + w.chunk);
    float *to = w.part + int64_t(lane * w.width + q) * w.slots * (SIDE * SIDE);
    while (at < end) {
        const int block = at / w.S, t = block * w.width + q, from = at - block * w.S, upto = min(w.S, from + end - at);
        if (t < w.tiles) {
            int ti, tj;
            tile_at(w, SIDE, t, ti, tj);
            piece(ti, tj, 2 * from, 2 * upto, to + int64_t(slot) * (SIDE * SIDE));
        }
        at += upto - from;
        ++slot;
    }
}

}  // namespace muon
}  // namespace ionn
