// Host-side sizing of the loss head (no HIP dependency; checked on the CPU): tile
// choice, vocabulary pieces, dX splits and the layout of the caller's workspace.
#pragma once

#include <algorithm>
#include <cstdint>

namespace lb {
namespace xent {

constexpr int kCUs = 256;
constexpr int64_t kMaxWidth = (int64_t)1 << 22; // K and V stay below: 256 rows of 2^23 bytes fit a descriptor

inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline int64_t cdiv(int64_t x, int64_t m) { return (x + m - 1) / m; }

// Row tiles: 32, 64 or 128 rows (x 128 columns) for small M, 256 x 256 otherwise.
enum Rows { ROWS32 = 0, ROWS64 = 1, ROWS128 = 2, ROWS256 = 3 };
inline int tile_rows(int r) { return 32 << r; }
inline int tile_cols(int r) { return r == ROWS256 ? 256 : 128; }
inline int choose_rows(int64_t M) { return M <= 32 ? ROWS32 : M <= 64 ? ROWS64 : M <= 128 ? ROWS128 : ROWS256; }

// A packed copy of W's piece (V not a multiple of 8, or W not 16-byte aligned) takes at
// most this.  Large pieces waste fewer part-filled rounds of tiles (pieces of 128 MiB,
// which stay in the last-level cache, were slower).
constexpr int64_t kPackBytes = (int64_t)1 << 30;
// per-tile softmax statistics of a forward piece
constexpr int64_t kPartBytes = (int64_t)128 << 20;
// the piece of dL/dlogits (16 bit) that the backward pass holds
constexpr int64_t kGradBytes = (int64_t)512 << 20;
// fp32 partial sums of dX
constexpr int64_t kSplitBytes = (int64_t)256 << 20;

// widest piece (a multiple of 256 columns, at least 256) with `per_col` bytes a column within `cap`
inline int64_t piece(int64_t V, int64_t per_col, int64_t cap) {
    const int64_t most = std::max<int64_t>(256, cap / std::max<int64_t>(1, per_col) / 256 * 256);
    const int64_t n = cdiv(V, most);
    return up(cdiv(V, n), 256);
}

struct Fwd {
    int rows;          // Rows
    int64_t Kp;        // K rounded up to 8
    int64_t Vc;        // piece width
    int64_t parts;     // statistics entries (tiles) per row and piece
    int join_rows;     // rows per block that joins them
    int64_t off_x, off_w, off_part, off_run, off_zt, off_sum, bytes;
};

inline Fwd forward(int64_t M, int64_t K, int64_t V, bool pack_w) {
    Fwd f;
    f.rows = choose_rows(M);
    f.Kp = up(K, 8);
    const int64_t cols = tile_cols(f.rows);
    f.Vc = piece(V, cdiv(8 * M, cols), kPartBytes);
    if (pack_w)
        f.Vc = std::min(f.Vc, piece(V, 2 * K, kPackBytes));
    f.parts = cdiv(f.Vc, cols);
    f.join_rows = M <= 4096 ? 16 : 64;
    if (M <= 32)
        for (f.join_rows = 1; f.join_rows < M;)
            f.join_rows *= 2;
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t o = at;
        at += up(n, 256);
        return o;
    };
    f.off_x = take(2 * M * f.Kp);
    f.off_w = take(pack_w ? 2 * K * f.Vc : 0);
    f.off_part = take(8 * M * f.parts);
    f.off_run = take(8 * M);
    f.off_zt = take(4 * M);
    f.off_sum = take(16 * cdiv(M, f.join_rows));
    f.bytes = at;
    return f;
}

struct Bwd {
    int rows;
    int64_t Kp, Vc;
    int splits;        // dX's reduction over a piece, in this many ranges
    int64_t split_len; // a multiple of 64
    bool acc;          // dX goes through fp32 memory (several pieces or ranges)
    int64_t off_row, off_x, off_w, off_g, off_acc, bytes;
};

// dX over a piece of Vc columns beside dW over M rows.  A dX tile walks Vc columns, a dW
// tile M rows; where M is small one dX tile would outlast everything else, so its
// reduction is split until a tile is at most half of what a CU gets on average (or
// 1024 columns), within the partial sums' room.
inline int dx_splits(int64_t M, int64_t Kp, int64_t Vc, int rows) {
    const int tr = tile_rows(rows), tc = tile_cols(rows);
    const int dwr = rows == ROWS256 ? 256 : 128;
    const int64_t slots = rows == ROWS256 ? kCUs : 2 * kCUs;
    const int64_t ntx = cdiv(M, tr) * cdiv(Kp, tc);
    const int64_t ntw = cdiv(Kp, dwr) * cdiv(Vc, dwr);
    const int64_t total = ntx * cdiv(Vc, 64) + ntw * cdiv(M, 64);
    const int64_t target = std::max<int64_t>(8, total / slots / 2); // pairs of slabs
    int64_t s = cdiv(cdiv(Vc, 64), target);
    s = std::min<int64_t>(s, std::max<int64_t>(1, kSplitBytes / (4 * M * Kp)));
    s = std::min<int64_t>(s, 64);
    return (int)std::max<int64_t>(1, s);
}

inline Bwd backward(int64_t M, int64_t K, int64_t V, bool pack_w) {
    Bwd b;
    b.rows = choose_rows(M);
    b.Kp = up(K, 8);
    b.Vc = piece(V, 2 * M, kGradBytes);
    if (pack_w)
        b.Vc = std::min(b.Vc, piece(V, 2 * K, kPackBytes));
    b.splits = dx_splits(M, b.Kp, b.Vc, b.rows);
    b.split_len = up(cdiv(b.Vc, b.splits), 64);
    b.splits = (int)cdiv(b.Vc, b.split_len);
    b.acc = b.splits > 1 || b.Vc < V;
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t o = at;
        at += up(n, 256);
        return o;
    };
    b.off_row = take(16 * M + 64);
    b.off_x = take(2 * M * b.Kp);
    b.off_w = take(pack_w ? 2 * K * b.Vc : 0);
    b.off_g = take(2 * M * b.Vc);
    b.off_acc = take(b.acc ? 4 * M * b.Kp * b.splits : 0);
    b.bytes = at;
    return b;
}

// enough for any alignment of W
inline int64_t forward_bytes(int64_t M, int64_t K, int64_t V) {
    return std::max(forward(M, K, V, false).bytes, forward(M, K, V, true).bytes);
}
inline int64_t backward_bytes(int64_t M, int64_t K, int64_t V) {
    return std::max(backward(M, K, V, false).bytes, backward(M, K, V, true).bytes);
}

} // namespace xent
} // namespace lb
