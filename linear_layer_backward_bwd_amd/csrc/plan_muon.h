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
// Microseconds of a launch: rounds of (fixed + per 64 reduction indices), from single
// products on the card (64x64 to 4096x12288, R from 64 to 4096; a tile alone on its CU and
// two to a CU): 256x256 7.5 + 1.03, 128x128 3.8 + 0.36 alone (the deep ring keeps it so)
// and 0.65 two to a CU, 64x64 2.8 + 0.24 alone and 0.34.
inline double microseconds(Tile t, int64_t n, int64_t R) {
    const double p = (double)cdiv(R, 64);
    switch (t) {
    case TILE256: return cdiv(n, kCUs) * (7.5 + 1.03 * p);
    case TILE128: return cdiv(n, 2 * kCUs) * (3.8 + 0.65 * p);
    case TILE128_DEEP: return cdiv(n, kCUs) * (3.9 + 0.36 * p);
    default: return n <= kCUs ? 2.8 + 0.24 * p : cdiv(n, 2 * kCUs) * (2.8 + 0.34 * p);
    }
}
inline Tile choose(int64_t batch, int64_t I, int64_t J, int64_t R, bool sym, double *us = nullptr) {
    Tile best = TILE256;
    double least = 0;
    for (Tile t : {TILE256, TILE128, TILE128_DEEP, TILE64}) {
        const int T = t == TILE256 ? 256 : t == TILE64 ? 64 : 128;
        const double c = microseconds(t, tiles(batch, I, J, T, sym), R);
        if (t == TILE256 || c < least) {
            best = t;
            least = c;
        }
    }
    if (us)
        *us = least;
    return best;
}

// Symmetric products run their tiles on and below the diagonal only, each storing its
// mirror image too (about 3 us: 16-bit stores), where that shortens the launch; at equal
// rounds and long reductions too, as idle CUs leave the others a higher clock (4096 x 4096
// over 12288: 136 tiles 272 us, all 256 300).
inline bool lower_only(int64_t batch, int64_t I, int64_t R) {
    double half, full;
    choose(batch, I, I, R, true, &half);
    choose(batch, I, I, R, false, &full);
    return half + 3.0 < full || (half <= full && full > 40.0);
}

// A matrix whose shorter side fits one tile has A and B = bA + cA² made by one block in one
// launch: 64 or 128 wide.  0: two launches.  (128: against 64x64 tiles and a launch more.)
inline int one_tile(int64_t batch, int64_t s, int64_t R) {
    if (s <= 64)
        return 64;
    if (s > 128)
        return 0;
    double us = 0;
    choose(batch, s, s, R, false, &us);
    return microseconds(TILE128_DEEP, batch, R) + 1.0 <= us + 3.3 ? 128 : 0;
}

struct Plan {
    int64_t s, sp, Np; // shorter side, rounded up to 8; N rounded up to 8
    bool tall;         // K > N: the products run on the columns
    int parts;
    int64_t off_x0, off_x1, off_a, off_b, off_part, bytes;
};

inline Plan plan(int64_t batch, int64_t K, int64_t N) {
    Plan p;
    p.tall = K > N;
    p.s = std::min(K, N);
    p.sp = up(p.s, 8);
    p.Np = up(N, 8);
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
    p.bytes = at;
    return p;
}

} // namespace muon
} // namespace lb
