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

// Tiles of a product [I, J] over a batch.  256x256 tiles run one to a CU, 128x128 ones two;
// with no more of them than CUs, one to a CU with a deeper ring.  The rounds that a launch
// takes are weighed by a round's length (256x256: 10).
enum Tile { TILE256 = 0, TILE128 = 1, TILE128_DEEP = 2 };
inline int64_t tiles(int64_t batch, int64_t I, int64_t J, int T, bool sym) {
    const int64_t ti = cdiv(I, T), tj = cdiv(J, T);
    return batch * (sym ? ti * (ti + 1) / 2 : ti * tj);
}
inline Tile choose(int64_t batch, int64_t I, int64_t J, bool sym) {
    const int64_t n256 = tiles(batch, I, J, 256, sym), n128 = tiles(batch, I, J, 128, sym);
    if (n128 <= kCUs)
        return TILE128_DEEP;
    return 10 * cdiv(n256, kCUs) <= 6 * cdiv(n128, 2 * kCUs) ? TILE256 : TILE128;
}

// Symmetric products run their lower tiles only, unless all tiles fit the CUs at once: then
// time is latency, and the mirror image costs more than the tiles saved (256: 6.4 against
// 9.2 us a product).
inline bool lower_only(int64_t batch, int64_t I) { return tiles(batch, I, I, 128, false) > kCUs; }

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
