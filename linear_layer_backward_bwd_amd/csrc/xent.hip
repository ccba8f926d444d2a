// Softmax cross entropy of a Linear head on gfx950, without storing the logits:
//
//     z = X·W             X [M,K], W [K,V]
//     lse[m] = log Σ_v exp z[m,v]          loss[m] = lse[m] − z[m, t(m)]
//     G[m,v] = (exp(z[m,v] − lse[m]) − [v = t(m)]) · s[m]      dX = G·Wᵀ   dW = Xᵀ·G
//
// Rows with a negative target take no part: loss, lse and gradient are 0.
//
// Forward: one product over tiles of the vocabulary whose epilogue keeps, per row and
// wave's columns, the maximum and the sum of exponentials (fp32, base 2), and the
// target's logit; a second kernel joins them in a fixed order.  M·K·V products, 8 bytes
// of statistics per row and 32-128 columns instead of 4 bytes per logit.
//
// Backward: the logits are computed again, a piece of the vocabulary at a time; the
// epilogue turns them into G (16 bit: the operand type of the two products that read
// it), then one launch runs the piece's dX and dW tiles.  G's piece is bounded
// (512 MiB) whatever V is.  dX is summed over pieces in fp32.
//
// Rounding: products of 16-bit operands accumulate in fp32; statistics, lse and the
// sums of dX over pieces are fp32, the mean is summed in fp64; G is rounded once to
// the operands' type, dX and dW once at the end.  G is made with s / max |s|, and the
// epilogues multiply by max |s| in fp32: with s itself every entry −s of the targets
// would be off by the same rounding of s, a bias of the whole gradient by up to half a
// step (dW 3.1e-3 off against 2.3e-3).  For fp16 it is scaled up by 2^14 besides, so
// that the probabilities of a large vocabulary stay above fp16's smallest normal.
#include "kernels.h"
#include "plan_xent.h"
#include "tile.h"

#include <algorithm>

namespace lb {
namespace {

using namespace tile;
using xent::cdiv;

typedef float pair_t __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// What the backward pass needs of a row.
struct RowParam {
    float lse2; // lse·log2(e)
    float s;    // upstream gradient over the factor of the outputs
    int t;      // target, -1: none
    int pad;
};

// ---- copies: zero-padded rows, 16-byte aligned -----------------------------------------
// dst [rows, ldd] (ldd % 8 == 0) from src[r*lds + c], c < cols; columns past cols are
// zero, and so are rows that `keep` leaves out.  One 16-byte chunk per thread; unaligned sources are read as dwords (two
// bytes apart: shifted together), the first and last chunk of such a row by elements.
template <class Keep>
__device__ __forceinline__ void pack_rows(const uint16_t *src, int64_t lds, int64_t rows, int64_t cols, uint16_t *dst,
                                          int64_t ldd, int64_t first, int64_t stride, Keep keep) {
    typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));
    const int64_t per = ldd / 8;
    const int64_t step_r = stride / per, step_q = stride - step_r * per;
    int64_t r = first / per, q = first - r * per; // one division, then steps
    for (; r < rows; r += step_r, q += step_q) {
        if (q >= per) {
            q -= per;
            if (++r >= rows)
                break;
        }
        const int64_t c = q * 8;
        u32x4_t v = {};
        if (c < cols) { // loaded whether kept or not: the two loads do not wait for each other
            const uint16_t *p = src + r * lds + c;
            const uintptr_t a = reinterpret_cast<uintptr_t>(p);
            if (c + 8 <= cols && (a & 15) == 0) {
                v = *reinterpret_cast<const u32x4_t *>(p);
            } else if (c + 8 <= cols && (a & 3) == 0) {
                v = *reinterpret_cast<const u32x4_a4 *>(p);
            } else if (c > 0 && c + 8 < cols) {
                const u32x4_t lo = *reinterpret_cast<const u32x4_a4 *>(p - 1);
                const uint32_t hi = *reinterpret_cast<const uint32_t *>(p + 7);
                v = u32x4_t{(lo[0] >> 16) | (lo[1] << 16), (lo[1] >> 16) | (lo[2] << 16),
                            (lo[2] >> 16) | (lo[3] << 16), (lo[3] >> 16) | (hi << 16)};
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < cols)
                        v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
            }
        }
        if (!keep(r))
            v = u32x4_t{};
        *reinterpret_cast<u32x4_t *>(dst + r * ldd + c) = v;
    }
}

__global__ __launch_bounds__(256) void k_xent_pack(const uint16_t *src, int64_t lds, int64_t rows, int64_t cols,
                                                   uint16_t *dst, int64_t ldd) {
    pack_rows(src, lds, rows, cols, dst, ldd, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256,
              [](int64_t) { return true; });
}

void pack(const void *src, int64_t lds, int64_t rows, int64_t cols, void *dst, int64_t ldd, hipStream_t s) {
    const int64_t blocks = std::min<int64_t>(cdiv(rows * (ldd / 8), 256), 16 * xent::kCUs);
    hipLaunchKernelGGL(k_xent_pack, dim3((unsigned)blocks), dim3(256), 0, s, static_cast<const uint16_t *>(src), lds,
                       rows, cols, static_cast<uint16_t *>(dst), ldd);
}

// ---- forward ---------------------------------------------------------------------------
struct StatsParams {
    Job job;               // A = X (RC), B = W's piece (OC)
    const int64_t *target; // [M]
    int64_t v0;            // first column of the piece
    pair_t *part;          // [tiles][M]: (maximum·log2 e, Σ 2^(z·log2 e − that))
    float *zt;             // [M] target logits
};

__device__ __forceinline__ pair_t join(pair_t a, pair_t b) {
    const float m = fmaxf(a.x, b.x);
    const float r = m == -INFINITY ? 0.0f : m; // nothing yet on either side
    return pair_t{m, a.y * exp2_fast(a.x - r) + b.y * exp2_fast(b.x - r)};
}

template <class C, bool FULL>
__device__ __forceinline__ void stats_epilogue(const StatsParams &p, Acc<C> &acc, int64_t ib, int64_t jb,
                                               pair_t (&st)[C::FI], int lane) {
    const int64_t M = p.job.I;
#pragma unroll
    for (int x = 0; x < C::FI; ++x) {
        pin(acc[x]);
        const int64_t i = ib + 16 * x + (lane & 15);
        const int left = FULL ? 0 : (int)min<int64_t>(p.job.J - jb, C::FJ * 16); // columns inside
        auto in = [&](int y, int e) { return FULL || 16 * y + 4 * (lane >> 4) + e < left; };
        float mx = -INFINITY;
#pragma unroll
        for (int y = 0; y < C::FJ; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                mx = fmaxf(mx, in(y, e) ? acc[x][y][e] : -INFINITY);
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float m2 = mx == -INFINITY ? 0.0f : mx * kLog2e;
        float s = 0.0f;
#pragma unroll
        for (int y = 0; y < C::FJ; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float t = exp2_fast(__builtin_fmaf(acc[x][y][e], kLog2e, -m2));
                s += in(y, e) ? t : 0.0f;
            }
        s += __shfl_xor(s, 16, 64);
        s += __shfl_xor(s, 32, 64);
        const bool row = i < M;
        const int64_t t = row ? p.target[i] - p.v0 - jb : -1;
        if (t >= 0 && t < C::FJ * 16 && jb + t < p.job.J && ((int)t >> 2 & 3) == (lane >> 4)) {
            float z = 0.0f;
#pragma unroll
            for (int y = 0; y < C::FJ; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    z = ((int)t >> 4) == y && ((int)t & 3) == e ? acc[x][y][e] : z;
            p.zt[i] = z;
        }
        st[x] = pair_t{mx == -INFINITY ? -INFINITY : m2, s};
    }
}

// The logits' tile and its statistics.  Up to 64 rows it streams W once: M = 32, K = 4096,
// V = 65536 97 us, 5.5 TB/s (a copy reaches 5.1).  From 256 rows it is MFMA-bound: M = 16384,
// K = 4096, V = 32000 3.1 ms, 1.38 PFLOP/s; the exponentials and the start of a tile cost
// about 8 of its 98 us.
template <class C>
__global__ __launch_bounds__(kThreads, C::TI == 256 ? 1 : 2) void k_xent_stats(StatsParams p) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::kLds];
    LB_LDS char *smem = (LB_LDS char *)smem_raw;
    int ti, tj;
    coords(p.job, gathered(blockIdx.x, gridDim.x), ti, tj);
    Acc<C> acc;
    accumulate<C>(p.job, ti, tj, smem, acc);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t ib = (int64_t)ti * C::TI + (w / C::WJ) * C::FI * 16;
    const int64_t jb = (int64_t)tj * C::TJ + (w % C::WJ) * C::FJ * 16;
    pair_t st[C::FI]; // of this wave's columns
    if (jb + C::FJ * 16 <= p.job.J)
        stats_epilogue<C, true>(p, acc, ib, jb, st, lane);
    else
        stats_epilogue<C, false>(p, acc, ib, jb, st, lane);
    // join the waves that hold the same rows
    LB_LDS pair_t *const sh = (LB_LDS pair_t *)smem; // [WJ][TI]
#pragma unroll
    for (int x = 0; x < C::FI; ++x)
        if (lane < 16)
            sh[(w % C::WJ) * C::TI + (w / C::WJ) * C::FI * 16 + 16 * x + lane] = st[x];
    __syncthreads();
    const int r = threadIdx.x;
    const int64_t i = (int64_t)ti * C::TI + r;
    if (r < C::TI && i < p.job.I) {
        pair_t a = sh[r];
#pragma unroll
        for (int k = 1; k < C::WJ; ++k)
            a = join(a, sh[k * C::TI + r]);
        p.part[(int64_t)tj * p.job.I + i] = a;
    }
}

// Joins a piece's statistics with those of the pieces before (run), and after the last
// piece writes loss and lse, and the block's sum and count of losses.  A block of 1024
// takes rb rows; 1024 / rb threads per row walk the tiles, a fixed tree joins them.  Few
// rows go to one block, which then writes the mean too; otherwise rb is small enough for
// many blocks (one block for 32 rows of 2048 entries took 27 us).
struct Sum {
    double loss;
    int64_t n;
};
struct JoinParams {
    const pair_t *part;
    pair_t *run;
    const float *zt;
    const int64_t *target;
    float *loss, *lse;
    Sum *sum;   // [blocks]
    float *out; // mean written here by the only block, or null
    int64_t M, V, parts;
    int first, last, rb;
};

__device__ __forceinline__ void write_mean(Sum s, float *out) {
    const double inv = s.n ? 1.0 / (double)s.n : 0.0;
    out[0] = s.n ? (float)(s.loss * inv) : 0.0f;
    out[1] = (float)inv;
}
__device__ __forceinline__ Sum wave_sum(Sum s) {
#pragma unroll
    for (int h = 32; h > 0; h >>= 1) {
        s.loss += __shfl_xor(s.loss, h, 64);
        s.n += __shfl_xor(s.n, h, 64);
    }
    return s;
}

__global__ __launch_bounds__(1024) void k_xent_join(JoinParams p) {
    __shared__ pair_t sh[1024];
    const int rb = p.rb, per = 1024 / rb;
    const int r = threadIdx.x % rb, k = threadIdx.x / rb;
    const int64_t i = (int64_t)blockIdx.x * rb + r;
    pair_t a = pair_t{-INFINITY, 0.0f};
    if (i < p.M) {
        if (k == 0 && !p.first)
            a = p.run[i];
        for (int64_t e = k; e < p.parts; e += 4 * per) {
            pair_t q[4]; // four loads in flight
#pragma unroll
            for (int u = 0; u < 4; ++u)
                q[u] = e + u * per < p.parts ? p.part[(e + u * per) * p.M + i] : pair_t{-INFINITY, 0.0f};
#pragma unroll
            for (int u = 0; u < 4; ++u)
                a = join(a, q[u]);
        }
    }
    sh[threadIdx.x] = a;
    __syncthreads();
    for (int h = per / 2; h > 0; h >>= 1) {
        if (k < h)
            sh[threadIdx.x] = join(sh[threadIdx.x], sh[threadIdx.x + h * rb]);
        __syncthreads();
    }
    if (threadIdx.x >= 64) // rb <= 64: the rows' results are the first wave's
        return;
    Sum s{0.0, 0};
    if (k == 0 && i < p.M) {
        a = sh[r];
        p.run[i] = a;
        if (p.last) {
            const int64_t t = p.target[i];
            // the loss from the logarithm's two parts, the target's exponent as it is in the sum:
            // lse − z has lost half a step of |z|, all of the loss of a row that is nearly sure
            const float log2s = __builtin_log2f(a.y);
            const float lse = (a.x + log2s) * kLn2;
            const float own = t < 0 || t >= p.V ? 0.0f : __builtin_fmaf(p.zt[i], kLog2e, -a.x);
            const float loss = t < 0 ? 0.0f : t < p.V ? (log2s - own) * kLn2 : NAN;
            p.lse[i] = t < 0 ? 0.0f : lse;
            p.loss[i] = loss;
            s = Sum{(double)loss, t >= 0};
        }
    }
    if (p.last) {
        s = wave_sum(s);
        if (threadIdx.x == 0) {
            if (p.out)
                write_mean(s, p.out);
            else
                p.sum[blockIdx.x] = s;
        }
    }
}

// mean of the counted losses and 1 / their number (0 of none), from the blocks' sums
__global__ __launch_bounds__(256) void k_xent_mean(const Sum *sum, int64_t n, float *out) {
    __shared__ Sum sh[4];
    Sum s{0.0, 0};
    for (int64_t i = threadIdx.x; i < n; i += 256) {
        s.loss += sum[i].loss;
        s.n += sum[i].n;
    }
    s = wave_sum(s);
    if ((threadIdx.x & 63) == 0)
        sh[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 4; ++w) {
            s.loss += sh[w].loss;
            s.n += sh[w].n;
        }
        write_mean(s, out);
    }
}

template <class T, int ROWS>
struct FwdCfg;
template <class T> struct FwdCfg<T, xent::ROWS32> { using C = Cfg<T, 1, 4, 2, 2, false, true, 4>; };
template <class T> struct FwdCfg<T, xent::ROWS64> { using C = Cfg<T, 1, 4, 4, 2, false, true, 3>; };
template <class T> struct FwdCfg<T, xent::ROWS128> { using C = Cfg<T, 2, 2, 4, 4, false, true, 2>; };
template <class T> struct FwdCfg<T, xent::ROWS256> { using C = Cfg<T, 2, 2, 8, 8, false, true, 2, 3>; };

template <class C>
void set_tiles(Job &j) {
    j.tiles_i = (int)cdiv(j.I, C::TI);
    j.tiles_j = (int)cdiv(j.J, C::TJ);
    j.group = 4;
}

// the tile, with B = W at any alignment if `any`
template <class C, class Fn>
void with_alignment(bool any, Fn fn) {
    if (any)
        fn(typename C::With{});
    else
        fn(C{});
}

template <class C>
void run_stats(StatsParams &p, hipStream_t s) {
    set_tiles<C>(p.job);
    hipLaunchKernelGGL((k_xent_stats<C>), dim3((unsigned)(p.job.tiles_i * p.job.tiles_j)), dim3(kThreads), 0, s, p);
}

// fn(Cfg): the logits' tile
template <class T, class Fn>
void logits_tile(int rows, bool any, Fn fn) {
    switch (rows) {
    case xent::ROWS32: with_alignment<typename FwdCfg<T, xent::ROWS32>::C>(any, fn); break;
    case xent::ROWS64: with_alignment<typename FwdCfg<T, xent::ROWS64>::C>(any, fn); break;
    case xent::ROWS128: with_alignment<typename FwdCfg<T, xent::ROWS128>::C>(any, fn); break;
    default: with_alignment<typename FwdCfg<T, xent::ROWS256>::C>(any, fn); break;
    }
}
template <class T>
void stats(int rows, bool any, StatsParams &p, hipStream_t s) {
    logits_tile<T>(rows, any, [&](auto c) { run_stats<decltype(c)>(p, s); });
}

bool aligned(const void *p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// ---- backward --------------------------------------------------------------------------
// Row parameters, by the first `params` blocks, and X's copy (rows that take no part as zeros:
// theirs may hold anything), by the others.  factor[0] is what both outputs are multiplied
// by: max |s| (or 1 if that is 0, infinite or NaN), over 2^14 for fp16.  Without row_scale
// that is every row's |s|; with it each of the `params` blocks takes the maximum itself, over
// the rows up to kPeakRows, else over k_xent_peak's blocks (with one block for all rows the
// backward pass at M = 65536, K = 256, V = 1024 took 580 us in place of 399).
struct PrepParams {
    const int64_t *target;
    const float *lse, *row_scale, *d_scale;
    float scale;
    int64_t M, K, V, Kp;
    int f16, params, peaks; // peaks: 0, or the number of entries of `peak`
    RowParam *row;
    float *factor;
    float *peak; // [xent::kPeaks]
    const uint16_t *X;
    uint16_t *x;

    __device__ __forceinline__ float base() const { return scale * (d_scale ? d_scale[0] : 1.0f); }
    // the copy of X by n blocks, of which this is b
    __device__ __forceinline__ void copy(int b, int n, float base_) const {
        pack_rows(X, K, M, K, x, Kp, (int64_t)b * 256 + threadIdx.x, (int64_t)n * 256, [&](int64_t r) {
            return target[r] >= 0 && (row_scale ? base_ * row_scale[r] : base_) != 0.0f;
        });
    }
    // what the rows' s are divided by, from the largest of them
    static __device__ __forceinline__ float unit_of(float mx) { return mx > 0.0f && mx < INFINITY ? mx : 1.0f; }
    __device__ __forceinline__ float up() const { return f16 ? 16384.0f : 1.0f; }
    __device__ __forceinline__ RowParam param(int64_t t, float lse_, float s, float mx) const {
        if (t >= V)
            return RowParam{0.0f, NAN, -1, 0}; // no such class: the gradients say so
        if (t >= 0 && s != 0.0f)
            return RowParam{lse_ * kLog2e, s / mx * up(), (int)t, 0};
        return RowParam{0.0f, 0.0f, -1, 0}; // takes no part
    }
};
constexpr int64_t kPeakRows = 1024;

__device__ __forceinline__ float block_max(float v, float (&sh)[4]) {
#pragma unroll
    for (int h = 32; h > 0; h >>= 1)
        v = fmaxf(v, __shfl_xor(v, h, 64));
    if ((threadIdx.x & 63) == 0)
        sh[threadIdx.x >> 6] = v;
    __syncthreads();
    return fmaxf(fmaxf(sh[0], sh[1]), fmaxf(sh[2], sh[3]));
}

// largest |s| of the rows that take part, each block over a share of them
__global__ __launch_bounds__(256) void k_xent_peak(PrepParams p) {
    __shared__ float sh[4];
    const float base = p.base();
    float mx = 0.0f;
#pragma unroll 4
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.M; i += (int64_t)gridDim.x * 256)
        mx = fmaxf(mx, p.target[i] >= 0 ? fabsf(base * p.row_scale[i]) : 0.0f);
    mx = block_max(mx, sh);
    if (threadIdx.x == 0)
        p.peak[blockIdx.x] = mx;
}

__global__ __launch_bounds__(256) void k_xent_prep(PrepParams p) {
    __shared__ float sh[4];
    const float base = p.base();
    auto s_of = [&](int64_t i) { return p.row_scale ? base * p.row_scale[i] : base; };
    if ((int)blockIdx.x >= p.params) {
        p.copy(blockIdx.x - p.params, gridDim.x - p.params, base);
        return;
    }
    float mx = fabsf(base);
    if (p.row_scale) {
        mx = 0.0f;
        if (p.peaks) {
            if ((int)threadIdx.x < p.peaks)
                mx = p.peak[threadIdx.x];
        } else {
            for (int64_t i = threadIdx.x; i < p.M; i += 256)
                mx = fmaxf(mx, p.target[i] >= 0 ? fabsf(s_of(i)) : 0.0f);
        }
        mx = block_max(mx, sh);
    }
    mx = PrepParams::unit_of(mx);
    if (blockIdx.x == 0 && threadIdx.x == 0)
        p.factor[0] = mx / p.up();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.M; i += (int64_t)p.params * 256)
        p.row[i] = p.param(p.target[i], p.lse[i], s_of(i), mx);
}

struct GradParams {
    Job job; // A = X (RC), B = W's piece (OC)
    const RowParam *row;
    int64_t v0, Vg; // first column of the piece; columns of G (a multiple of 64, zero past J)
    uint16_t *g;    // [M, Vg]
    PrepParams prep; // OWN
    int tiles;       // OWN: blocks of tiles; the others copy X
};

// OWN, up to 64 rows, saves the launch that prepares them (40.6 -> 37.9 us at M = 16, K = 1024,
// V = 32000): each wave takes its rows' parameters and the largest |s| from the arrays
// while its first operands are on their way, X is read as it is (a row out of the loss is
// dropped by its s), and blocks behind the tiles make the copy that dW needs.
// The piece of G = (exp(z − lse) − onehot)·s; the row parameters are loaded once the sums
// stand, 16 bytes a row and lane, and G leaves through LDS in whole lines (M = 8192,
// K = 4096, a piece of 32768 columns: 1.62 ms, 1.36 PFLOP/s).
template <class C, bool OWN>
__global__ __launch_bounds__(kThreads, C::TI == 256 ? 1 : 2) void k_xent_grad(GradParams p) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::kLds];
    LB_LDS char *smem = (LB_LDS char *)smem_raw;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int ti, tj;
    if constexpr (OWN) {
        if ((int)blockIdx.x >= p.tiles) {
            p.prep.copy(blockIdx.x - p.tiles, gridDim.x - p.tiles, p.prep.base());
            return;
        }
        coords(p.job, gathered(blockIdx.x, p.tiles), ti, tj);
    } else {
        coords(p.job, gathered(blockIdx.x, gridDim.x), ti, tj);
    }
    const int64_t ib = (int64_t)ti * C::TI + (w / C::WJ) * C::FI * 16;
    const int64_t jb = (int64_t)tj * C::TJ + (w % C::WJ) * C::FJ * 16;
    RowParam rp[C::FI];
    if constexpr (OWN) {
        const PrepParams &q = p.prep;
        const float base = q.base();
        auto s_of = [&](int64_t i) { return q.row_scale ? base * q.row_scale[i] : base; };
        float mx = fabsf(base);
        if (q.row_scale) { // M <= 64: a row a lane
            mx = lane < q.M && q.target[lane] >= 0 ? fmaxf(0.0f, fabsf(s_of(lane))) : 0.0f;
#pragma unroll
            for (int h = 32; h > 0; h >>= 1)
                mx = fmaxf(mx, __shfl_xor(mx, h, 64));
        }
        mx = PrepParams::unit_of(mx);
        if (blockIdx.x == 0 && threadIdx.x == 0)
            q.factor[0] = mx / q.up();
#pragma unroll
        for (int x = 0; x < C::FI; ++x) {
            const int64_t i = ib + 16 * x + (lane & 15);
            rp[x] = i < q.M ? q.param(q.target[i], q.lse[i], s_of(i), mx) : RowParam{0.0f, 0.0f, -1, 0};
        }
    }
    Acc<C> acc;
    accumulate<C>(p.job, ti, tj, smem, acc);
    if constexpr (!OWN) {
#pragma unroll
        for (int x = 0; x < C::FI; ++x) {
            const int64_t i = ib + 16 * x + (lane & 15);
            rp[x] = i < p.job.I ? p.row[i] : RowParam{0.0f, 0.0f, -1, 0};
        }
    }
    const int j0 = (int)jb + 4 * (lane >> 4);
    store16<C>(acc, p.g, p.Vg, p.job.I, p.Vg, ib, jb, true, false, smem, [](int) {}, [&](int x, int y) {
        const int t = rp[x].t < 0 ? -1 : rp[x].t - (int)p.v0;
        float g[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = j0 + 16 * y + e;
            const float pr = exp2_fast(__builtin_fmaf(acc[x][y][e], kLog2e, -rp[x].lse2));
            g[e] = (j == t ? pr - 1.0f : pr) * rp[x].s;
            g[e] = j < (int)p.job.J && !(OWN && rp[x].s == 0.0f) ? g[e] : 0.0f;
        }
        return u32x2_t{C::T::pack2(g[0], g[1]), C::T::pack2(g[2], g[3])};
    });
}

struct BothParams {
    Job dx;            // A = G (RC), B = W's piece (RC); R = the piece's columns
    int splits;        // ranges of dx.R
    int64_t split_len;
    float *acc;        // [splits][M][Kp] fp32, or null: one range and one piece
    int64_t Kp;
    int first, last;   // piece
    uint16_t *dX;      // written after the last piece when splits == 1
    int dx_vec;
    Job dw;            // A = X (OC), B = G (OC); J = the piece's columns
    uint16_t *dW;      // at the piece's first column
    int64_t ldw;
    int dw_vec, dw_nt; // rows 16-byte aligned; of whole 128-byte lines
    const float *factor; // of both outputs
    int dw_tiles;      // blocks of dW; 0: not wanted
    int dx_tiles;      // blocks of dX
    int dx_first;      // the longer tiles are launched first
    int want_dx;
};

template <class C>
__device__ __forceinline__ void dx_tile(const BothParams &p, int b, LB_LDS char *smem) {
    const int per = p.dx.tiles_i * p.dx.tiles_j;
    b = gathered(b, p.dx_tiles); // neighbours share a range too
    const int sp = b / per;
    Job j = p.dx;
    const int64_t k0 = (int64_t)sp * p.split_len;
    j.a += k0;
    j.b += k0;
    j.R = min<int64_t>(p.split_len, p.dx.R - k0);
    int ti, tj;
    coords(j, b - sp * per, ti, tj);
    Acc<C> acc;
    accumulate<C>(j, ti, tj, smem, acc);
    const int64_t i0 = (int64_t)ti * C::TI, j0 = (int64_t)tj * C::TJ;
    const int64_t M = j.I, K = j.J;
    float *const part = p.acc ? p.acc + (int64_t)sp * M * p.Kp : nullptr;
    const float f = p.factor[0];
    const bool out = p.splits == 1 && p.last;
    staged<C>(acc, i0, j0, smem, [](int, int64_t, int, int64_t) {}, [&](int, int64_t i, int rows, int64_t j, f32x4_t (&v)[C::FJ]) {
        if (!p.first) {
            f32x4_t old[C::FJ];
#pragma unroll
            for (int q = 0; q < C::FJ; ++q)
                old[q] = i + q * rows < M && j < p.Kp
                             ? *reinterpret_cast<const f32x4_t *>(part + (i + q * rows) * p.Kp + j)
                             : f32x4_t{};
#pragma unroll
            for (int q = 0; q < C::FJ; ++q)
                v[q] = old[q] + v[q];
        }
#pragma unroll
        for (int q = 0; q < C::FJ; ++q) {
            const int64_t r = i + q * rows;
            if (r >= M || j >= p.Kp)
                continue;
            if (!out) {
                *reinterpret_cast<f32x4_t *>(part + r * p.Kp + j) = v[q];
            } else if (p.dx_vec && j < K) {
                const u32x2_t h = {C::T::pack2(v[q][0] * f, v[q][1] * f), C::T::pack2(v[q][2] * f, v[q][3] * f)};
                *reinterpret_cast<u32x2_t *>(p.dX + r * K + j) = h;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < K)
                        p.dX[r * K + j + e] = C::T::one(v[q][e] * f);
            }
        }
    });
}

template <class C>
__device__ __forceinline__ void dw_tile(const BothParams &p, int b, LB_LDS char *smem) {
    int ti, tj;
    coords(p.dw, gathered(b, p.dw_tiles), ti, tj);
    Acc<C> acc;
    if constexpr (C::S == 1)
        accumulate_once<C>(p.dw, ti, tj, smem, acc);
    else
        accumulate<C>(p.dw, ti, tj, smem, acc);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t ib = (int64_t)ti * C::TI + (w / C::WJ) * C::FI * 16;
    const int64_t jb = (int64_t)tj * C::TJ + (w % C::WJ) * C::FJ * 16;
    const float f = p.factor[0];
    store16<C>(acc, p.dW, p.ldw, p.dw.I, p.dw.J, ib, jb, p.dw_vec, p.dw_nt, smem, [](int) {}, [&](int x, int y) {
        const f32x4_t &a = acc[x][y];
        return u32x2_t{C::T::pack2(a[0] * f, a[1] * f), C::T::pack2(a[2] * f, a[3] * f)};
    });
}

// dX and dW of a piece in one launch, the longer tiles first, so that the shorter ones fill
// the CUs that the longer leave (the same piece: 3.0 ms, 1.45 PFLOP/s).  At M = 16, K = 1024,
// V = 32000 23 us for 131 MB, dX reading W and dW written side by side.
template <class CX, class CW>
__global__ __launch_bounds__(kThreads, CX::TI == 256 ? 1 : CW::S == 1 ? 3 : 2) void k_xent_both(BothParams p) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[CX::kLds > CW::kLds ? CX::kLds : CW::kLds];
    LB_LDS char *smem = (LB_LDS char *)smem_raw;
    const int b = blockIdx.x;
    const int lead = p.dx_first ? p.dx_tiles : p.dw_tiles;
    if ((b < lead) == (p.dx_first != 0))
        dx_tile<CX>(p, p.dx_first ? b : b - lead, smem);
    else
        dw_tile<CW>(p, p.dx_first ? b - lead : b, smem);
}

// dX from the ranges' partial sums: 64 groups of four columns per block, each wave a
// quarter of the ranges (in turn), the four sums added in wave order.
template <class T>
__global__ __launch_bounds__(256) void k_xent_dx_sum(const float *acc, int splits, int64_t M, int64_t K, int64_t Kp,
                                                     const float *factor, uint16_t *dX, int vec) {
    __shared__ f32x4_t sh[4][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const float f = factor[0];
    const int64_t n = M * Kp / 4;
    for (int64_t q0 = (int64_t)blockIdx.x * 64; q0 < n; q0 += (int64_t)gridDim.x * 64) {
        const int64_t q = q0 + lane;
        f32x4_t v = {};
        if (q < n) {
#pragma unroll 4
            for (int s = w; s < splits; s += 4)
                v += *reinterpret_cast<const f32x4_t *>(acc + (int64_t)s * M * Kp + 4 * q);
        }
        sh[w][lane] = v;
        __syncthreads();
        if (w == 0 && q < n) {
            v = ((v + sh[1][lane]) + sh[2][lane]) + sh[3][lane];
            const int64_t r = 4 * q / Kp, c = 4 * q - r * Kp;
            if (vec && c < K) {
                *reinterpret_cast<u32x2_t *>(dX + r * K + c) =
                    u32x2_t{T::pack2(v[0] * f, v[1] * f), T::pack2(v[2] * f, v[3] * f)};
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < K)
                        dX[r * K + c + e] = T::one(v[e] * f);
            }
        }
        __syncthreads();
    }
}

template <class T, int BOTH>
struct BwdCfg;
template <class T> struct BwdCfg<T, xent::X32_ONCE> {
    using X = Cfg<T, 1, 4, 2, 2, false, false, 2>;
    using W = Cfg<T, 1, 4, 4, 4, true, true, 1>;
};
template <class T> struct BwdCfg<T, xent::X64_ONCE> {
    using X = Cfg<T, 1, 4, 4, 2, false, false, 2>;
    using W = Cfg<T, 1, 4, 4, 4, true, true, 1>;
};
template <class T> struct BwdCfg<T, xent::X64_W128> {
    using X = Cfg<T, 1, 4, 4, 2, false, false, 3>;
    using W = Cfg<T, 2, 2, 4, 4, true, true, 2>;
};
template <class T> struct BwdCfg<T, xent::X128_W128> {
    using X = Cfg<T, 2, 2, 4, 4, false, false, 2>;
    using W = Cfg<T, 2, 2, 4, 4, true, true, 2>;
};
template <class T> struct BwdCfg<T, xent::X256_W256> {
    using X = Cfg<T, 2, 2, 8, 8, false, false, 2, 3>;
    using W = Cfg<T, 2, 2, 8, 8, true, true, 2, 3>;
};
template <class T> struct BwdCfg<T, xent::X64_W64> {
    using X = Cfg<T, 2, 2, 2, 2, false, false, 4>;
    using W = Cfg<T, 2, 2, 2, 2, true, true, 4>;
};

template <class C>
void run_grad(GradParams &g, hipStream_t s) {
    set_tiles<C>(g.job);
    // G's padding columns (up to a multiple of 64) are zeroed by the tiles that own them
    g.job.tiles_j = (int)cdiv(g.Vg, C::TJ);
    const int tiles = g.job.tiles_i * g.job.tiles_j;
    if constexpr (C::TI <= 64) {
        if (g.tiles) { // OWN: up to a block per CU copies X
            g.tiles = tiles;
            const int64_t copies = std::min<int64_t>(cdiv(g.prep.M * (g.prep.Kp / 8), 256), xent::kCUs);
            hipLaunchKernelGGL((k_xent_grad<C, true>), dim3((unsigned)(tiles + copies)), dim3(kThreads), 0, s, g);
            return;
        }
    }
    hipLaunchKernelGGL((k_xent_grad<C, false>), dim3((unsigned)tiles), dim3(kThreads), 0, s, g);
}
template <class T>
void grad(int rows, bool any, GradParams &g, hipStream_t s) {
    logits_tile<T>(rows, any, [&](auto c) { run_grad<decltype(c)>(g, s); });
}
template <class CX, class CW>
void run_both(BothParams &p, hipStream_t s) {
    set_tiles<CX>(p.dx);
    set_tiles<CW>(p.dw);
    p.dx_tiles = p.want_dx ? p.dx.tiles_i * p.dx.tiles_j * p.splits : 0;
    p.dw_tiles = p.dW ? p.dw.tiles_i * p.dw.tiles_j : 0;
    p.dx_first = p.split_len * CX::TI * CX::TJ >= p.dw.R * CW::TI * CW::TJ;
    hipLaunchKernelGGL((k_xent_both<CX, CW>), dim3((unsigned)(p.dx_tiles + p.dw_tiles)), dim3(kThreads), 0, s, p);
}
template <class T, int BOTH>
void both_as(bool any, BothParams &p, hipStream_t s) {
    with_alignment<typename BwdCfg<T, BOTH>::X>(
        any, [&](auto c) { run_both<decltype(c), typename BwdCfg<T, BOTH>::W>(p, s); });
}
template <class T>
void both(int which, bool any, BothParams &p, hipStream_t s) {
    switch (which) {
    case xent::X32_ONCE: both_as<T, xent::X32_ONCE>(any, p, s); break;
    case xent::X64_ONCE: both_as<T, xent::X64_ONCE>(any, p, s); break;
    case xent::X64_W128: both_as<T, xent::X64_W128>(any, p, s); break;
    case xent::X128_W128: both_as<T, xent::X128_W128>(any, p, s); break;
    case xent::X256_W256: // never with `any`
        run_both<typename BwdCfg<T, xent::X256_W256>::X, typename BwdCfg<T, xent::X256_W256>::W>(p, s);
        break;
    default: both_as<T, xent::X64_W64>(any, p, s); break;
    }
}

template <class T>
hipError_t backward(const XentBwdArgs &a, hipStream_t s) {
    const bool ragged = a.V % 8 != 0 || !aligned(a.W, 16), pack_w = ragged && xent::pack_backward(a.M);
    const xent::Bwd b = xent::backward(a.M, a.K, a.V, pack_w);
    char *const ws = static_cast<char *>(a.ws);
    RowParam *const row = reinterpret_cast<RowParam *>(ws + b.off_row);
    float *const factor = reinterpret_cast<float *>(ws + b.off_row + 16 * a.M);
    uint16_t *const x = reinterpret_cast<uint16_t *>(ws + b.off_x);
    uint16_t *const wp = reinterpret_cast<uint16_t *>(ws + b.off_w);
    PrepParams pp{a.target, a.lse, a.row_scale, a.d_scale, a.scale, a.M, a.K, a.V, b.Kp, a.f16,
                  (int)std::min<int64_t>(cdiv(a.M, 256), xent::kCUs), 0, row, factor, factor + 1,
                  static_cast<const uint16_t *>(a.X), x};
    // the logits' kernel prepares the rows itself
    const bool own = a.M <= 64 && b.rows <= xent::ROWS64 && b.Vc >= a.V && a.K % 8 == 0 && aligned(a.X, 16);
    if (a.row_scale && a.M > kPeakRows) {
        pp.peaks = (int)std::min<int64_t>(cdiv(a.M, 1024), xent::kPeaks);
        hipLaunchKernelGGL(k_xent_peak, dim3((unsigned)pp.peaks), dim3(256), 0, s, pp);
    }
    const int64_t copies = std::min<int64_t>(cdiv(a.M * (b.Kp / 8), 256), 8 * xent::kCUs);
    if (!own)
        hipLaunchKernelGGL(k_xent_prep, dim3((unsigned)(pp.params + copies)), dim3(256), 0, s, pp);
    const bool dx_vec = a.K % 4 == 0 && aligned(a.dX, 8);
    for (int64_t v0 = 0; v0 < a.V; v0 += b.Vc) {
        const int64_t vc = std::min(b.Vc, a.V - v0);
        const uint16_t *w = static_cast<const uint16_t *>(a.W) + v0;
        int64_t ldw = a.V;
        if (pack_w) {
            pack(w, a.V, a.K, vc, wp, b.Vc, s);
            w = wp;
            ldw = b.Vc;
        }
        GradParams g{};
        g.job.a = own ? static_cast<const uint16_t *>(a.X) : x;
        g.job.lda = own ? a.K : b.Kp;
        g.prep = pp;
        g.tiles = own;
        g.job.b = w;
        g.job.ldb = ldw;
        g.job.I = a.M;
        g.job.J = vc;
        g.job.R = a.K;
        g.row = row;
        g.v0 = v0;
        g.Vg = xent::up(vc, 64);
        g.g = reinterpret_cast<uint16_t *>(ws + b.off_g);
        BothParams p{};
        p.dx.a = g.g;
        p.dx.lda = g.Vg;
        p.dx.b = w;
        p.dx.ldb = ldw;
        p.dx.I = a.M;
        p.dx.J = a.K;
        p.dx.R = vc;
        p.split_len = std::min(b.split_len, xent::up(p.dx.R, 64));
        p.splits = b.splits;
        p.acc = b.acc ? reinterpret_cast<float *>(ws + b.off_acc) : nullptr;
        p.Kp = b.Kp;
        p.first = v0 == 0;
        p.last = v0 + b.Vc >= a.V;
        p.dX = static_cast<uint16_t *>(a.dX);
        p.dx_vec = dx_vec;
        p.dw.a = x;
        p.dw.lda = b.Kp;
        p.dw.b = g.g;
        p.dw.ldb = g.Vg;
        p.dw.I = a.K;
        p.dw.J = vc;
        p.dw.R = a.M;
        p.dW = a.dW ? static_cast<uint16_t *>(a.dW) + v0 : nullptr;
        p.ldw = a.V;
        p.dw_vec = a.V % 8 == 0 && aligned(a.dW, 16);
        p.dw_nt = a.V % 64 == 0 && aligned(a.dW, 128);
        p.factor = factor;
        p.want_dx = a.dX != nullptr;
        grad<T>(b.rows, ragged && !pack_w, g, s);
        both<T>(b.both, ragged && !pack_w, p, s);
    }
    if (a.dX && b.splits > 1) {
        const int64_t blocks = std::min<int64_t>(cdiv(a.M * b.Kp / 4, 64), 32 * xent::kCUs);
        hipLaunchKernelGGL((k_xent_dx_sum<T>), dim3((unsigned)blocks), dim3(256), 0, s,
                           reinterpret_cast<const float *>(ws + b.off_acc), b.splits, a.M, a.K, b.Kp, factor,
                           static_cast<uint16_t *>(a.dX), (int)dx_vec);
    }
    return hipGetLastError();
}

template <class T>
hipError_t forward(const XentArgs &a, hipStream_t s) {
    const bool ragged = a.V % 8 != 0 || !aligned(a.W, 16), pack_w = ragged && xent::pack_forward(a.M);
    const xent::Fwd f = xent::forward(a.M, a.K, a.V, pack_w);
    char *const ws = static_cast<char *>(a.ws);
    StatsParams p{};
    p.job.a = static_cast<const uint16_t *>(a.X);
    p.job.lda = a.K;
    // also where rows are no whole 128-byte lines and the product is large: ragged rows cost
    // a quarter of its time
    if (a.K % 8 != 0 || !aligned(a.X, 16) || (a.K % 64 != 0 && (double)a.M * a.K * a.V > 5e10)) {
        uint16_t *const x = reinterpret_cast<uint16_t *>(ws + f.off_x);
        pack(a.X, a.K, a.M, a.K, x, f.Kp, s);
        p.job.a = x;
        p.job.lda = f.Kp;
    }
    p.job.I = a.M;
    p.job.R = a.K;
    p.target = a.target;
    p.part = reinterpret_cast<pair_t *>(ws + f.off_part);
    p.zt = reinterpret_cast<float *>(ws + f.off_zt);
    JoinParams j{};
    j.part = p.part;
    j.run = reinterpret_cast<pair_t *>(ws + f.off_run);
    j.zt = p.zt;
    j.target = a.target;
    j.loss = a.loss;
    j.lse = a.lse;
    j.M = a.M;
    j.V = a.V;
    j.sum = reinterpret_cast<Sum *>(ws + f.off_sum);
    j.rb = f.join_rows;
    const int64_t blocks = cdiv(a.M, j.rb);
    j.out = blocks == 1 ? a.out : nullptr;
    for (int64_t v0 = 0; v0 < a.V; v0 += f.Vc) {
        const int64_t vc = std::min(f.Vc, a.V - v0);
        const uint16_t *w = static_cast<const uint16_t *>(a.W) + v0;
        p.job.ldb = a.V;
        if (pack_w) {
            uint16_t *const wp = reinterpret_cast<uint16_t *>(ws + f.off_w);
            pack(w, a.V, a.K, vc, wp, f.Vc, s);
            w = wp;
            p.job.ldb = f.Vc;
        }
        p.job.b = w;
        p.job.J = vc;
        p.v0 = v0;
        stats<T>(f.rows, ragged && !pack_w, p, s);
        j.parts = cdiv(vc, xent::shape(f.rows).tj);
        j.first = v0 == 0;
        j.last = v0 + f.Vc >= a.V;
        hipLaunchKernelGGL(k_xent_join, dim3((unsigned)blocks), dim3(1024), 0, s, j);
    }
    if (blocks > 1)
        hipLaunchKernelGGL(k_xent_mean, dim3(1), dim3(256), 0, s, j.sum, blocks, a.out);
    return hipGetLastError();
}

// dW = 0 when there are no rows (a kernel, not a memset: calls may be captured into a graph)
__global__ __launch_bounds__(256) void k_xent_zero(uint16_t *p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        p[i] = 0;
}

} // namespace

hipError_t launch_lin_xent(const XentArgs &a, hipStream_t s) {
    if (a.M == 0) { // nothing counted: mean 0
        hipLaunchKernelGGL(k_xent_mean, dim3(1), dim3(256), 0, s, (const Sum *)nullptr, (int64_t)0, a.out);
        return hipGetLastError();
    }
    return a.f16 ? forward<F16>(a, s) : forward<BF16>(a, s);
}

hipError_t launch_lin_xent_bwd(const XentBwdArgs &a, hipStream_t s) {
    if (!a.dX && !a.dW)
        return hipSuccess;
    if (a.M == 0) {
        if (a.dW)
            hipLaunchKernelGGL(k_xent_zero, dim3(1024), dim3(256), 0, s, static_cast<uint16_t *>(a.dW), a.K * a.V);
        return hipGetLastError();
    }
    return a.f16 ? backward<F16>(a, s) : backward<BF16>(a, s);
}

} // namespace lb
