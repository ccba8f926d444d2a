// Host-side sizing of the Newton-Schulz orthogonalisation (no HIP dependency; checked
// on the CPU): tile choice and the layout of the caller's workspace.
#pragma once

#include <algorithm>
#include <cstdint>

namespace lb {
namespace muon {

constexpr int kCUs = 256;
constexpr int64_t kMaxSide = (int64_t)1 << 20; // K and N: rows and slabs stay within a buffer descriptor
constexpr int64_t kMaxBatch = 65535;           // grid dimension
constexpr int kMaxParts = 1024;                // blocks (partial sums) per matrix for the norm
constexpr int64_t kNormBlocks = 4096;          // ... and about as many in all

inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline int64_t cdiv(int64_t x, int64_t m) { return (x + m - 1) / m; }

// Tiles of a product [I, J] over a batch, with a reduction of R.
enum Tile { TILE256 = 0, TILE128 = 1, TILE128_DEEP = 2, TILE64 = 3 };
inline int64_t tiles(int64_t batch, int64_t I, int64_t J, int T, bool sym) {
    const int64_t ti = cdiv(I, T), tj = cdiv(J, T);
    return batch * (sym ? ti * (ti + 1) / 2 : ti * tj);
}
// Microseconds of a launch of n tiles, fixed + per 64 reduction indices, from the products
// themselves on the card (sides 96 to 4096 over 256 to 12288, batches of 1 to 12, random
// operands).  256x256: 8.4 + 1.04, rising to 1.4 with every CU at work (the power limit's
// clock).  128x128, two to a CU: 5 + 0.57 for up to 256 tiles, 4.6 + 0.8 beyond; one to a CU
// (a ring of four slots keeps it so): 4 + 0.36, rising to 0.54.  64x64: 2.8 + 0.25, 0.37 two
// to a CU.  Tiles past whole rounds run as a launch of their own.
inline double microseconds(Tile t, int64_t n, int64_t R) {
    const double p = (double)cdiv(R, 64);
    const bool one = t == TILE256 || t == TILE128_DEEP; // to a CU
    const int64_t slots = one ? kCUs : 2 * kCUs, rounds = n / slots, rem = n % slots;
    const double share = (double)rem / kCUs;
    double first, full, fixed, last; // a full round, and what is left
    switch (t) {
    case TILE256: first = fixed = 8.4, full = 1.4, last = 1.04 + 0.36 * std::max(0.0, share - 0.5) * 2; break;
    case TILE128: first = 4.6, full = 0.8, fixed = 5.0, last = rem <= kCUs ? 0.57 : 0.8; break;
    case TILE128_DEEP: first = fixed = 4.0, full = 0.54, last = 0.36 + 0.18 * share; break;
    default: first = fixed = 2.8, full = 0.37, last = rem <= kCUs ? 0.25 : 0.37; break;
    }
    return rounds * (first + full * p) + (rem ? fixed + last * p : 0.0);
}
struct Choice {
    Tile tile;
    bool lower; // of a symmetric product: the tiles on and below the diagonal only
    double us;
};
// The tiles on and below the diagonal of a symmetric product each store their mirror image
// too: 7 us for 256x256 tiles, 2 for 128x128, 0.4 for 64x64.
inline Choice choose(int64_t batch, int64_t I, int64_t J, int64_t R, bool symmetric) {
    Choice best{TILE256, false, 1e30};
    for (Tile t : {TILE256, TILE128, TILE128_DEEP, TILE64})
        for (int lower = 0; lower <= (symmetric ? 1 : 0); ++lower) {
            const int T = t == TILE256 ? 256 : t == TILE64 ? 64 : 128;
            const double mirror = !lower ? 0.0 : t == TILE256 ? 7.0 : t == TILE64 ? 0.4 : 2.0;
            const double c = microseconds(t, tiles(batch, I, J, T, lower), R) + mirror;
            if (c < best.us)
                best = Choice{t, lower != 0, c};
        }
    return best;
}

// A matrix whose shorter side fits one tile has A and B = bA + cA² made by one block in one
// launch: 64 or 128 wide.  0: two launches.  (128: against 64x64 tiles and a launch more.)
inline int one_tile(int64_t batch, int64_t s, int64_t R) {
    if (s <= 64)
        return 64;
    if (s > 128)
        return 0;
    return microseconds(TILE128_DEEP, batch, R) + 1.0 <= choose(batch, s, s, R, true).us + 3.5 ? 128 : 0;
}

// The reduction of that one tile in ranges, one block each, where it is long: their fp32
// sums are added by the block that makes B, a launch more (4.5 us) and 0.25 us a range.
constexpr int kMaxSplits = 16;
inline int one_tile_splits(int64_t batch, int T, int64_t R) {
    const Tile t = T == 64 ? TILE64 : TILE128_DEEP;
    int best = 1;
    double least = microseconds(t, batch, R);
    for (int s = 2; s <= kMaxSplits; s *= 2) {
        const double c = microseconds(t, batch * s, cdiv(R, s)) + 4.5 + 0.25 * s * (T / 64);
        if (c < least) {
            best = s;
            least = c;
        }
    }
    return best;
}

struct Plan {
    // the shorter side; it and N rounded up to 64: rows of whole 128-byte lines (ragged rows
    // cost a product a quarter of its time: every 128-byte fetch touched two lines)
    int64_t s, sp, Np;
    bool tall;         // K > N: the products run on the columns
    int parts;
    int one, splits; // one_tile() and its ranges (1: none)
    int64_t off_x0, off_x1, off_a, off_b, off_part, off_sums, bytes;
};

inline Plan plan(int64_t batch, int64_t K, int64_t N) {
    Plan p;
    p.tall = K > N;
    p.s = std::min(K, N);
    p.sp = up(p.s, 64);
    p.Np = up(N, 64);
    p.parts = (int)std::min<int64_t>({kMaxParts, cdiv(K * N, 4096), std::max<int64_t>(1, kNormBlocks / batch)});
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t o = at;
        at += up(n, 256);
        return o;
    };
    p.off_x0 = take(2 * batch * K * p.Np);
    p.off_x1 = take(2 * batch * K * p.Np);
    p.off_a = take(2 * batch * p.s * p.sp);
    p.off_b = take(2 * batch * p.s * p.sp);
    p.off_part = take(8 * batch * p.parts);
    const int64_t R = std::max(K, N);
    p.one = one_tile(batch, p.s, R);
    p.splits = p.one ? one_tile_splits(batch, p.one, R) : 1;
    p.off_sums = take(p.splits > 1 ? 4 * batch * p.splits * p.one * p.one : 0);
    p.bytes = at;
    return p;
}

} // namespace muon
} // namespace lb
