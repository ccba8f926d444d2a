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
constexpr int kMaxParts = 256;                 // blocks (partial sums) per matrix for the norm

inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline int64_t cdiv(int64_t x, int64_t m) { return (x + m - 1) / m; }

// 256x256 tiles (one block per CU) where they fill at least half of the CUs, else
// 128x128 (two blocks per CU).
inline bool big_tiles(int64_t batch, int64_t I, int64_t J) { return batch * cdiv(I, 256) * cdiv(J, 256) >= kCUs / 2; }

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
    p.parts = (int)std::min<int64_t>(kMaxParts, cdiv(K * N, 4096));
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
