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

// Tile shapes.  Microseconds of a tile over p pairs of slabs (64 reduction indices each),
// measured on the card with single products from 64 x 64 to 4096 x 12288: fixed + p * alone
// with a CU to itself, fixed + p * full with `slots` of them on the card.
struct Shape {
    int ti, tj, slots;
    double fixed, alone, full;
};
enum Rows { ROWS32 = 0, ROWS64 = 1, ROWS128 = 2, ROWS256 = 3, SQUARE64 = 4, WIDE64 = 5 };
inline Shape shape(int r) {
    switch (r) {
    case ROWS32: return {32, 128, 2 * kCUs, 2.9, 0.25, 0.45};
    case ROWS64: return {64, 128, 2 * kCUs, 3.1, 0.30, 0.57};
    case ROWS128: return {128, 128, 2 * kCUs, 3.8, 0.36, 0.65};
    case ROWS256: return {256, 256, kCUs, 11.0, 1.03, 1.03};
    case SQUARE64: return {64, 64, 2 * kCUs, 2.8, 0.24, 0.34};
    default: return {64, 256, 3 * kCUs, 5.0, 0.30, 0.60}; // a reduction of at most 64
    }
}
inline int64_t tiles(int r, int64_t I, int64_t J) { return cdiv(I, shape(r).ti) * cdiv(J, shape(r).tj); }
// a launch of n equal tiles
inline double launch_us(int r, int64_t n, int64_t p) {
    const Shape s = shape(r);
    return n <= kCUs ? s.fixed + s.alone * p : cdiv(n, s.slots) * (s.fixed + s.full * p);
}
// The logits' tiles: X's rows by the vocabulary's columns, over K.
inline int choose_rows(int64_t M, int64_t K, int64_t V) {
    int best = ROWS32;
    for (int r : {ROWS64, ROWS128, ROWS256})
        if (launch_us(r, tiles(r, M, V), cdiv(K, 64)) < launch_us(best, tiles(best, M, V), cdiv(K, 64)))
            best = r;
    return best;
}

// Rows of W at any alignment (V no multiple of 8, or W not 16-byte aligned) are read as they
// are, through registers, or copied to padded rows first.  The copy costs 0.75 ps an
// element, reading as it is 18-28% of a product on 256x256 tiles: forward, M = 2048 776 us
// against about 830, M = 6000 (K = 4096, V = 30001) 1330 against 1220.  Backward the two
// products pay: M = 100 97 against 113, M = 777 697 against 614.
inline bool pack_forward(int64_t M) { return M >= 2560; }
inline bool pack_backward(int64_t M) { return M > 256; }
// The copy of W's piece takes at most this.  Large pieces waste fewer part-filled rounds of
// tiles (M = 2048, K = 4096, V = 50257 backward in pieces of 128 MiB 2559 us, whole 2387);
// where V is a multiple of 8 only a pointer off 16 bytes needs the copy, and every call's
// workspace has room for it: 128 MiB.
inline int64_t pack_bytes(int64_t V) { return V % 8 == 0 ? (int64_t)128 << 20 : (int64_t)1 << 30; }
// per-tile softmax statistics of a forward piece
constexpr int64_t kPartBytes = (int64_t)128 << 20;
// the piece of dL/dlogits (16 bit) that the backward pass holds
constexpr int64_t kGradBytes = (int64_t)512 << 20;
// fp32 partial sums of dX
constexpr int64_t kSplitBytes = (int64_t)256 << 20;

// blocks that look for the largest row factor of the backward pass
constexpr int kPeaks = 255;

// widest piece (a multiple of 256 columns, at least 256) with `per_col` bytes a column within `cap`
inline int64_t piece(int64_t V, int64_t per_col, int64_t cap) {
    const int64_t most = std::max<int64_t>(256, cap / std::max<int64_t>(1, per_col) / 256 * 256);
    const int64_t n = cdiv(V, most);
    return up(cdiv(V, n), 256);
}

struct Fwd {
    int rows;          // Rows
    int64_t Kp;        // rows of the copy of X: K rounded up to 64 (whole 128-byte lines)
    int64_t Vc;        // piece width
    int64_t parts;     // statistics entries (tiles) per row and piece
    int join_rows;     // rows per block that joins them
    int64_t off_x, off_w, off_part, off_run, off_zt, off_sum, bytes;
};

inline Fwd forward(int64_t M, int64_t K, int64_t V, bool pack_w) {
    Fwd f;
    f.rows = choose_rows(M, K, V);
    f.Kp = up(K, 64);
    const int64_t cols = shape(f.rows).tj;
    f.Vc = piece(V, cdiv(8 * M, cols), kPartBytes);
    if (pack_w)
        f.Vc = std::min(f.Vc, piece(V, 2 * K, pack_bytes(V)));
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

// The tiles of dX (rows of X by K, over a piece of Vc columns, in ranges) and dW (K by Vc,
// over the rows) share a launch.
struct Pair {
    int x, w;  // Rows
    int slots; // blocks of the launch on the card
};
// X32_ONCE and X64_ONCE: up to 64 rows, where dW is bound by writing it.  Its tiles take
// their whole reduction at once, and small rings let three blocks share a CU (M = 15,
// K = 1792, V = 109976: 267 us with 128x128 tiles, two to a CU).
enum Both { X32_ONCE = 0, X64_ONCE = 1, X128_W128 = 2, X256_W256 = 3, X64_W64 = 4, X64_W128 = 5 };
inline Pair pair(int both) {
    switch (both) {
    case X32_ONCE: return {ROWS32, WIDE64, 3 * kCUs};
    case X64_ONCE: return {ROWS64, WIDE64, 3 * kCUs};
    case X128_W128: return {ROWS128, ROWS128, 2 * kCUs};
    case X256_W256: return {ROWS256, ROWS256, kCUs};
    case X64_W128: return {ROWS64, ROWS128, 2 * kCUs};
    default: return {SQUARE64, SQUARE64, 2 * kCUs};
    }
}

struct Bwd {
    int rows;          // Rows of the logits' tiles
    int both;          // Both
    int64_t Kp, Vc;
    int splits;        // dX's reduction over a piece, in this many ranges
    int64_t split_len; // a multiple of 64
    bool acc;          // dX goes through fp32 memory (several pieces or ranges)
    int64_t off_row, off_x, off_w, off_g, off_acc, bytes;
};

// A dX tile walks Vc columns, a dW tile M rows; where M is small one dX tile would outlast
// everything else, so its reduction is split until a tile takes at most half of what a
// slot gets on average (or 8 pairs of slabs), within the partial sums' room.
inline int dx_splits(int64_t M, int64_t Kp, int64_t Vc, int both) {
    const Pair c = pair(both);
    const int64_t ntx = tiles(c.x, M, Kp), ntw = tiles(c.w, Kp, Vc);
    const Shape x = shape(c.x), w = shape(c.w);
    const int64_t px = cdiv(Vc, 64), pw = cdiv(M, 64);
    const double per_slot = (ntx * (px * x.full) + ntw * (pw * w.full + w.fixed)) / c.slots;
    const int64_t target = std::max<int64_t>(8, (int64_t)(per_slot / 2 / x.full));
    int64_t s = cdiv(px, target);
    s = std::min<int64_t>(s, std::max<int64_t>(1, kSplitBytes / (4 * M * Kp)));
    return (int)std::max<int64_t>(1, std::min<int64_t>(s, 64));
}
inline double both_us(int64_t M, int64_t Kp, int64_t Vc, int both) {
    const Pair c = pair(both);
    const int s = dx_splits(M, Kp, Vc, both);
    const int64_t nx = tiles(c.x, M, Kp) * s, nw = tiles(c.w, Kp, Vc);
    const Shape x = shape(c.x), w = shape(c.w);
    const double px = (double)cdiv(cdiv(Vc, s), 64), pw = (double)cdiv(M, 64);
    // partial sums written and read back at 5 TB/s
    const double sums = s > 1 ? 3.5 + 8.0 * M * Kp * s / 5e6 : 0.0;
    if (nx + nw <= kCUs)
        return std::max(x.fixed + x.alone * px, w.fixed + w.alone * pw) + sums;
    const double tx = x.fixed + x.full * px, tw = w.fixed + w.full * pw;
    return (nx * tx + nw * tw) / c.slots + 0.5 * std::max(tx, tw) + sums;
}
// (dX's 256x256 tile does not read W at any alignment: its epilogue would spill)
inline int choose_both(int64_t M, int64_t Kp, int64_t Vc) {
    int best = X64_W64;
    for (int b : {X32_ONCE, X64_ONCE, X64_W128, X128_W128, X256_W256})
        if ((b > X64_ONCE || M <= 64) && (b != X256_W256 || pack_backward(M)) &&
            both_us(M, Kp, Vc, b) < both_us(M, Kp, Vc, best))
            best = b;
    return best;
}

inline Bwd backward(int64_t M, int64_t K, int64_t V, bool pack_w) {
    Bwd b;
    b.rows = choose_rows(M, K, V);
    b.Kp = up(K, 64);
    b.Vc = piece(V, 2 * M, kGradBytes);
    if (pack_w)
        b.Vc = std::min(b.Vc, piece(V, 2 * K, pack_bytes(V)));
    b.both = choose_both(M, b.Kp, b.Vc);
    b.splits = dx_splits(M, b.Kp, b.Vc, b.both);
    b.split_len = up(cdiv(b.Vc, b.splits), 64);
    b.splits = (int)cdiv(b.Vc, b.split_len);
    b.acc = b.splits > 1 || b.Vc < V;
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t o = at;
        at += up(n, 256);
        return o;
    };
    b.off_row = take(16 * M + 4 * (1 + kPeaks)); // row parameters, the outputs' factor, kPeaks maxima
    b.off_x = take(2 * M * b.Kp);
    b.off_w = take(pack_w ? 2 * K * b.Vc : 0);
    b.off_g = take(2 * M * b.Vc);
    b.off_acc = take(b.acc ? 4 * M * b.Kp * b.splits : 0);
    b.bytes = at;
    return b;
}

// enough for any alignment of W
inline int64_t forward_bytes(int64_t M, int64_t K, int64_t V) {
    return std::max(forward(M, K, V, false).bytes, forward(M, K, V, pack_forward(M)).bytes);
}
inline int64_t backward_bytes(int64_t M, int64_t K, int64_t V) {
    return std::max(backward(M, K, V, false).bytes, backward(M, K, V, pack_backward(M)).bytes);
}

} // namespace xent
} // namespace lb
