// How a product of the DFP-8 layers is cut, by its sizes: shared by the Linear
// layer (dfp8_linear.hip) and the gated one (dfp8_gated.hip), whose gradients
// are the same two products.
#pragma once

#include "dfp8_rows.h"
#include "dfp8_tile128.h"

namespace ionn {
namespace dfp8 {

constexpr int64_t kMaxSide = int64_t(1) << 30;

inline bool sizes_ok(int64_t B, int64_t IN, int64_t OUT) {
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
    double us;       // of tiles: the time that is expected
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// By the sizes alone (the workspace query knows no addresses); operands whose
// address does not suit TILE256 and TILE128 take TILE.  a_pitch, b_pitch: bytes from
// an operand's row to the next, 0 for rows that follow each other.
template <bool A_KM, bool B_KM>
Plan make_plan(int64_t M, int64_t N, int64_t K, bool forward, int64_t a_pitch = 0, int64_t b_pitch = 0) {
    Plan p{TILE, ceil_div(M, 64) * ceil_div(N, 64), 1, 0, 0, 0.0};
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
    const int64_t lda = a_pitch ? a_pitch : a_side, ldb = b_pitch ? b_pitch : b_side;
    // The tile size that is expected to end first; in us, fitted to
    // measurements: a round of 256 x 256 tiles, one per compute unit, takes 23 (15
    // without an activation) and K / 110; 128 x 128 tiles, two at a time on a
    // compute unit, by the tiles that one gets; 64 x 64 tiles by the share of M N K.
    // Forward in tiles of 64, 128 and 256: 1000 x 1024 x 2048 8.3, 11.2 and 26 us;
    // 2048^3 22.5, 17.6 and 35; 2048 x 4096 x 4096 67, 42 and 54; 4096^3 128, 78
    // and 70.  With both gradients: 512^3 12, 19 and 35; 4096 x 1024 x 4096 110, 81
    // (74 in one grid) and 121.
    const double k = double(K);
    p.us = (forward ? 5.0 : 2.5) + double(M) * double(N) * k / 65536.0 / (forward ? 6800.0 : 6500.0);
    if (tile256_fits<A_KM, B_KM>(nullptr, lda, nullptr, ldb, M, N, K)) {
        const int64_t tiles256 = ceil_div(M, 256) * ceil_div(N, 256), tiles128 = ceil_div(M, 128) * ceil_div(N, 128);
        const double rounds = double(ceil_div(tiles256, 256)), each = double(ceil_div(tiles128, 256));
        const double t128 = forward ? 3.5 + 2.6 * each + k * (0.0022 + 0.0031 * each)
                                    : 2.5 + 1.8 * each + k * (0.0018 + 0.0031 * each);
        const double t256 = rounds * ((forward ? 23.0 : 15.0) + k / 110.0);
        if (t256 < p.us && t256 < t128) p.path = TILE256, p.us = t256;
        else if (t128 < p.us) p.path = TILE128, p.us = t128;
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

inline size_t part_bytes(const Plan &p, int64_t M, int64_t N) {
    return p.split > 1 ? (size_t(p.split) * M * N * sizeof(int32_t) + 15) & ~size_t(15) : 0;
}

inline Product make_product(const Plan &pl, const int8_t *A, int64_t lda, const int8_t *B, int64_t ldb, const Epi &ep,
                     int64_t M, int64_t N, int64_t K, void *part) {
    return Product{A,      B,      lda,      ldb, ep, int(M), int(N), int(K), pl.split, static_cast<int32_t *>(part),
                   int(pl.tiles * pl.split)};
}

inline void as_tiles128(Product &p) { p.blocks = int(ceil_div(p.M, 128) * ceil_div(p.N, 128)); }

// The path a planned product takes with these operands.
inline Path path_of(const Plan &pl, const int8_t *A, const int8_t *B) {
    return (pl.path == TILE256 || pl.path == TILE128) && !(aligned(A, 16) && aligned(B, 16)) ? TILE : pl.path;
}

// (a plan of larger tiles that falls back to 64 x 64 tiles has that many of them)
inline void as_tiles(Product &p) { p.blocks = int(ceil_div(p.M, 64) * ceil_div(p.N, 64) * p.split); }

inline unsigned sum_groups(const Product &p) { return unsigned(ceil_div(int64_t(p.M) * ceil_div(p.N, 4), NT)); }

// The workgroups of a product, on the path that it takes.
inline int64_t groups_of(const Plan &pl, const Product &p) {
    const Path path = path_of(pl, p.A, p.B);
    if (path == ROWS) return ceil_div(p.N, 16 * pl.cols);
    const int side = path == TILE256 ? 256 : path == TILE128 ? 128 : 64;
    return ceil_div(p.M, side) * ceil_div(p.N, side) * (side == 64 ? pl.split : 1);
}

// Whether their launches are within what the runtime takes.
inline bool launches(const Plan &pl, const Product &p) {
    return groups_of(pl, p) <= max_groups(path_of(pl, p.A, p.B) == ROWS ? kRowWaves * 64 : NT);
}
// (products whose tiles can be counted; twice: the two products of a backward
// pass share a grid)
inline bool tiles_ok(int64_t M, int64_t N) { return 2 * ceil_div(M, 64) * ceil_div(N, 64) <= 0x7fffffff; }

// The two gradients' products of a backward pass (dfp8_linear.hip), from the
// error dZ8, edZ that is in place: dX (nullable) [B][IN] and G (nullable)
// [OUT][IN] of type dtype.  IN >= 1.
struct BackwardSizes {
    int64_t B, IN, OUT;
    int64_t ldz, ldx, ldw;  // bytes from a row of dZ8, X, W to the next
};
size_t backward_part_bytes(const BackwardSizes &s);
struct BackwardProducts {
    const int8_t *dZ8, *X, *W;
    const int32_t *edZ, *eX, *eW;
    void *dX, *G;
    BackwardSizes s;
    void *parts;  // backward_part_bytes(s) bytes, 16-byte aligned
};
// How the two products are planned.
void backward_plans(const BackwardSizes &s, Plan &dX, Plan &G);
// Whether their launches are within what the runtime takes.
bool backward_launches(const BackwardProducts &p);
void launch_backward_products(const BackwardProducts &p, int dtype, hipStream_t st);

}  // namespace dfp8
}  // namespace ionn
