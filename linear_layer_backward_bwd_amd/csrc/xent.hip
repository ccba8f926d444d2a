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
// the operands' type, dX and dW once at the end.  For fp16, G is scaled by a power of
// two that brings max |s| to [2^14, 2^15), so that the probabilities of a large
// vocabulary stay above fp16's smallest normal; the epilogues take it out again.
#include "kernels.h"
#include "plan_xent.h"
#include "tile.h"

#include <algorithm>

namespace lb {
namespace {

using namespace tile;
using xent::cdiv;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// What the backward pass needs of a row.
struct RowParam {
    float lse2; // lse·log2(e)
    float s;    // upstream gradient · power of two
    int t;      // target, -1: none
    int pad;
};

// ---- copies: zero-padded rows, 16-byte aligned -----------------------------------------
// dst [rows, ldd] (ldd % 8 == 0) from src[r*lds + c], c < cols; columns past cols are
// zero, and so are the rows that `row` (if given) says take no part (their X may hold
// anything).  One 16-byte chunk per thread; unaligned sources are read as dwords (two
// bytes apart: shifted together), the first and last chunk of such a row by elements.
__global__ __launch_bounds__(256) void k_xent_pack(const uint16_t *src, int64_t lds, int64_t rows, int64_t cols,
                                                   uint16_t *dst, int64_t ldd, const RowParam *row) {
    typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));
    const int64_t per = ldd / 8, n = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per, c = (i - r * per) * 8;
        u32x4_t v = {};
        if (c < cols && !(row && row[r].t < 0 && row[r].s == 0.0f)) {
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
        *reinterpret_cast<u32x4_t *>(dst + r * ldd + c) = v;
    }
}

void pack(const void *src, int64_t lds, int64_t rows, int64_t cols, void *dst, int64_t ldd, const RowParam *row,
          hipStream_t s) {
    const int64_t blocks = std::min<int64_t>(cdiv(rows * (ldd / 8), 256), 16 * xent::kCUs);
    hipLaunchKernelGGL(k_xent_pack, dim3((unsigned)blocks), dim3(256), 0, s, static_cast<const uint16_t *>(src), lds,
                       rows, cols, static_cast<uint16_t *>(dst), ldd, row);
}

// ---- forward ---------------------------------------------------------------------------
struct StatsParams {
    Job job;               // A = X (RC), B = W's piece (OC)
    const int64_t *target; // [M]
    int64_t v0;            // first column of the piece
    float2 *part;          // [parts][M]: (maximum·log2 e, Σ 2^(z·log2 e − that))
    float *zt;             // [M] target logits
};

template <class C, bool FULL>
__device__ __forceinline__ void stats_epilogue(const StatsParams &p, Acc<C> &acc, int64_t ib, int64_t jb,
                                               int64_t slot, int lane) {
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
        if (lane < 16 && row)
            p.part[slot * M + i] = make_float2(mx == -INFINITY ? -INFINITY : m2, s);
    }
}

template <class C>
__global__ __launch_bounds__(kThreads, C::TI == 256 ? 1 : 2) void k_xent_stats(StatsParams p) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::kLds];
    LB_LDS char *smem = (LB_LDS char *)smem_raw;
    int ti, tj;
    coords(p.job, blockIdx.x, ti, tj);
    Acc<C> acc;
    accumulate<C>(p.job, ti, tj, smem, acc);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t ib = (int64_t)ti * C::TI + (w / C::WJ) * C::FI * 16;
    const int64_t jb = (int64_t)tj * C::TJ + (w % C::WJ) * C::FJ * 16;
    const int64_t slot = (int64_t)tj * C::WJ + w % C::WJ;
    if (jb + C::FJ * 16 <= p.job.J)
        stats_epilogue<C, true>(p, acc, ib, jb, slot, lane);
    else
        stats_epilogue<C, false>(p, acc, ib, jb, slot, lane);
}

// Joins a piece's statistics with those of the pieces before (run), and after the last
// piece writes loss and lse.  A block takes RB rows, 1024 / RB threads per row walk the
// entries, then a fixed tree joins them.
struct JoinParams {
    const float2 *part;
    float2 *run;
    const float *zt;
    const int64_t *target;
    float *loss, *lse;
    float *out; // mean written here when one block holds every row, or null
    int64_t M, V, parts;
    int first, last, rb;
};

__device__ __forceinline__ float2 join(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x);
    const float r = m == -INFINITY ? 0.0f : m; // nothing yet on either side
    return make_float2(m, a.y * exp2_fast(a.x - r) + b.y * exp2_fast(b.x - r));
}

// mean of the counted losses and 1 / their number (0 of none) by one block of 1024
__device__ __forceinline__ void mean_of(const float *loss, const int64_t *target, int64_t M, float *out, double *sd,
                                        int64_t *sn) {
    double d = 0.0;
    int64_t n = 0;
    for (int64_t i = threadIdx.x; i < M; i += 1024)
        if (target[i] >= 0) {
            d += (double)loss[i];
            ++n;
        }
    sd[threadIdx.x] = d;
    sn[threadIdx.x] = n;
    __syncthreads();
    for (int h = 512; h > 0; h >>= 1) {
        if ((int)threadIdx.x < h) {
            sd[threadIdx.x] += sd[threadIdx.x + h];
            sn[threadIdx.x] += sn[threadIdx.x + h];
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        const double inv = sn[0] ? 1.0 / (double)sn[0] : 0.0;
        out[0] = sn[0] ? (float)(sd[0] * inv) : 0.0f;
        out[1] = (float)inv;
    }
}

__global__ __launch_bounds__(1024) void k_xent_join(JoinParams p) {
    __shared__ float2 sh[1024];
    __shared__ double sd[1024];
    __shared__ int64_t sn[1024];
    const int rb = p.rb, per = 1024 / rb;
    const int r = threadIdx.x % rb, k = threadIdx.x / rb;
    const int64_t i = (int64_t)blockIdx.x * rb + r;
    float2 a = make_float2(-INFINITY, 0.0f);
    if (i < p.M) {
        if (k == 0 && !p.first)
            a = p.run[i];
        for (int64_t e = k; e < p.parts; e += per)
            a = join(a, p.part[e * p.M + i]);
    }
    sh[threadIdx.x] = a;
    __syncthreads();
    for (int h = per / 2; h > 0; h >>= 1) {
        if (k < h)
            sh[threadIdx.x] = join(sh[threadIdx.x], sh[threadIdx.x + h * rb]);
        __syncthreads();
    }
    if (k == 0 && i < p.M) {
        a = sh[r];
        p.run[i] = a;
        if (p.last) {
            const int64_t t = p.target[i];
            const float lse = (a.x + __builtin_log2f(a.y)) * kLn2;
            p.lse[i] = t < 0 ? 0.0f : lse;
            p.loss[i] = t < 0 ? 0.0f : t < p.V ? lse - p.zt[i] : NAN;
        }
    }
    if (p.last && p.out) {
        __syncthreads(); // one block: its losses are visible to it
        mean_of(p.loss, p.target, p.M, p.out, sd, sn);
    }
}

__global__ __launch_bounds__(1024) void k_xent_mean(const float *loss, const int64_t *target, int64_t M, float *out) {
    __shared__ double sd[1024];
    __shared__ int64_t sn[1024];
    mean_of(loss, target, M, out, sd, sn);
}

template <class T, int ROWS>
struct FwdCfg;
template <class T> struct FwdCfg<T, xent::ROWS32> { using C = Cfg<T, 1, 4, 2, 2, false, true, 4>; };
template <class T> struct FwdCfg<T, xent::ROWS64> { using C = Cfg<T, 1, 4, 4, 2, false, true, 3>; };
template <class T> struct FwdCfg<T, xent::ROWS128> { using C = Cfg<T, 2, 2, 4, 4, false, true, 2>; };
template <class T> struct FwdCfg<T, xent::ROWS256> { using C = Cfg<T, 2, 2, 8, 8, false, true, 2>; };

template <class C>
void set_tiles(Job &j) {
    j.tiles_i = (int)cdiv(j.I, C::TI);
    j.tiles_j = (int)cdiv(j.J, C::TJ);
    j.group = 4;
}

template <class C>
void run_stats(StatsParams &p, hipStream_t s) {
    set_tiles<C>(p.job);
    hipLaunchKernelGGL((k_xent_stats<C>), dim3((unsigned)(p.job.tiles_i * p.job.tiles_j)), dim3(kThreads), 0, s, p);
}

template <class T>
void stats(int rows, StatsParams &p, hipStream_t s) {
    switch (rows) {
    case xent::ROWS32: run_stats<typename FwdCfg<T, xent::ROWS32>::C>(p, s); break;
    case xent::ROWS64: run_stats<typename FwdCfg<T, xent::ROWS64>::C>(p, s); break;
    case xent::ROWS128: run_stats<typename FwdCfg<T, xent::ROWS128>::C>(p, s); break;
    default: run_stats<typename FwdCfg<T, xent::ROWS256>::C>(p, s); break;
    }
}

bool aligned(const void *p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// ---- backward --------------------------------------------------------------------------
// Row parameters (one block).  fp16: the power of two that brings max |s| to
// [2^14, 2^15); bf16 has fp32's range and takes 1.  scale[0], scale[1]: it and its inverse.
struct RowsParams {
    const int64_t *target;
    const float *lse, *row_scale, *d_scale;
    float scale;
    int64_t M, V;
    int f16;
    RowParam *row;
    float *pow2;
};

__global__ __launch_bounds__(1024) void k_xent_rows(RowsParams p) {
    __shared__ float sh[1024];
    const float base = p.scale * (p.d_scale ? p.d_scale[0] : 1.0f);
    auto s_of = [&](int64_t i) { return p.row_scale ? base * p.row_scale[i] : base; };
    float f = 1.0f;
    if (p.f16) {
        float mx = 0.0f;
        for (int64_t i = threadIdx.x; i < p.M; i += 1024)
            if (p.target[i] >= 0)
                mx = fmaxf(mx, fabsf(s_of(i)));
        sh[threadIdx.x] = mx;
        __syncthreads();
        for (int h = 512; h > 0; h >>= 1) {
            if ((int)threadIdx.x < h)
                sh[threadIdx.x] = fmaxf(sh[threadIdx.x], sh[threadIdx.x + h]);
            __syncthreads();
        }
        mx = sh[0];
        if (mx > 0.0f && mx < INFINITY) {
            int e;
            (void)frexpf(mx, &e); // mx in [2^(e-1), 2^e)
            f = ldexpf(1.0f, max(-100, min(100, 15 - e)));
        }
    }
    if (threadIdx.x == 0) {
        p.pow2[0] = f;
        p.pow2[1] = 1.0f / f;
    }
    for (int64_t i = threadIdx.x; i < p.M; i += 1024) {
        const int64_t t = p.target[i];
        const float s = s_of(i);
        RowParam r{0.0f, 0.0f, -1, 0}; // takes no part
        if (t >= p.V)
            r = RowParam{0.0f, NAN, -1, 0}; // no such class: the gradients say so
        else if (t >= 0 && s != 0.0f)
            r = RowParam{p.lse[i] * kLog2e, s * f, (int)t, 0};
        p.row[i] = r;
    }
}

// 16-bit output through LDS: 32 rows of a wave at a time, whole 16-byte chunks per lane.
// value(x, y) gives the 4 packed values of acc[x][y].  VEC: rows of dst 16-byte aligned.
template <class C, class Fn>
__device__ __forceinline__ void store16(Acc<C> &acc, uint16_t *dst, int64_t ld, int64_t I, int64_t J, int64_t ib, int64_t jb,
                                        bool vec, LB_LDS char *smem, Fn value) {
    constexpr int FJ = C::FJ, kRowB = FJ * 32, kChunks = 2 * FJ, kRows = 64 / kChunks;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    LB_LDS char *const reg = smem + w * (FJ * 1024);
#pragma unroll
    for (int h = 0; h < C::FI / 2; ++h) {
        pin(acc[2 * h]);
        pin(acc[2 * h + 1]);
#pragma unroll
        for (int xx = 0; xx < 2; ++xx)
#pragma unroll
            for (int y = 0; y < FJ; ++y) {
                const int r = 16 * xx + (lane & 15);
                const int c = 2 * y + (lane >> 5); // 16-byte chunk: 8 columns
                *reinterpret_cast<LB_LDS u32x2_t *>(reg + r * kRowB + ((c ^ (r & (kChunks - 1))) << 4) +
                                                    ((lane >> 4) & 1) * 8) = value(2 * h + xx, y);
            }
        const int64_t i0 = ib + 32 * h;
        if (vec) {
            u32x4_t v[FJ];
#pragma unroll
            for (int q = 0; q < FJ; ++q) {
                const int r = q * kRows + lane / kChunks, c = lane % kChunks;
                v[q] = *reinterpret_cast<const LB_LDS u32x4_t *>(reg + r * kRowB + ((c ^ (r & (kChunks - 1))) << 4));
            }
            __builtin_amdgcn_sched_barrier(0); // all reads before the first store
            const int64_t j = jb + 8 * (lane % kChunks);
#pragma unroll
            for (int q = 0; q < FJ; ++q) {
                const int64_t i = i0 + q * kRows + lane / kChunks;
                if (i < I && j < J)
                    __builtin_nontemporal_store(v[q], reinterpret_cast<u32x4_t *>(dst + i * ld + j));
            }
        } else {
            // rows of any alignment: 64 lanes store 64 neighbouring elements
            for (int q = 0; q < 32 * FJ * 16 / 64; ++q) {
                const int e = q * 64 + lane;
                const int r = e / (FJ * 16), c = e % (FJ * 16);
                const uint16_t v = *reinterpret_cast<const LB_LDS uint16_t *>(
                    reg + r * kRowB + (((c >> 3) ^ (r & (kChunks - 1))) << 4) + (c & 7) * 2);
                if (i0 + r < I && jb + c < J)
                    dst[(i0 + r) * ld + jb + c] = v;
            }
        }
    }
}

struct GradParams {
    Job job; // A = X (RC), B = W's piece (OC)
    const RowParam *row;
    int64_t v0, Vg; // first column of the piece; columns of G (a multiple of 64, zero past J)
    uint16_t *g;    // [M, Vg]
};

// the piece of G = (exp(z − lse) − onehot)·s
template <class C>
__global__ __launch_bounds__(kThreads, C::TI == 256 ? 1 : 2) void k_xent_grad(GradParams p) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::kLds];
    LB_LDS char *smem = (LB_LDS char *)smem_raw;
    int ti, tj;
    coords(p.job, blockIdx.x, ti, tj);
    Acc<C> acc;
    accumulate<C>(p.job, ti, tj, smem, acc);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t ib = (int64_t)ti * C::TI + (w / C::WJ) * C::FI * 16;
    const int64_t jb = (int64_t)tj * C::TJ + (w % C::WJ) * C::FJ * 16;
    RowParam rp[C::FI];
#pragma unroll
    for (int x = 0; x < C::FI; ++x) {
        const int64_t i = ib + 16 * x + (lane & 15);
        rp[x] = i < p.job.I ? p.row[i] : RowParam{0.0f, 0.0f, -1, 0};
    }
    const int j0 = (int)jb + 4 * (lane >> 4);
    store16<C>(acc, p.g, p.Vg, p.job.I, p.Vg, ib, jb, true, smem, [&](int x, int y) {
        const int t = rp[x].t < 0 ? -1 : rp[x].t - (int)p.v0;
        float g[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = j0 + 16 * y + e;
            const float pr = exp2_fast(__builtin_fmaf(acc[x][y][e], kLog2e, -rp[x].lse2));
            g[e] = (j == t ? pr - 1.0f : pr) * rp[x].s;
            g[e] = j < (int)p.job.J ? g[e] : 0.0f;
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
    int dw_vec;
    const float *pow2; // [1]: factor of both outputs
    int dw_tiles;      // blocks of dW; 0: not wanted
    int dx_tiles;      // blocks of dX
    int dx_first;      // the longer tiles are launched first
};

template <class C>
__device__ __forceinline__ void dx_tile(const BothParams &p, int b, LB_LDS char *smem) {
    const int per = p.dx.tiles_i * p.dx.tiles_j;
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
    const float f = p.pow2[1];
    const bool out = p.splits == 1 && p.last;
    staged<C>(acc, i0, j0, smem, [&](int64_t i, int rows, int64_t j, f32x4_t (&v)[C::FJ]) {
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
                __builtin_nontemporal_store(h, reinterpret_cast<u32x2_t *>(p.dX + r * K + j));
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
    coords(p.dw, b, ti, tj);
    Acc<C> acc;
    accumulate<C>(p.dw, ti, tj, smem, acc);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t ib = (int64_t)ti * C::TI + (w / C::WJ) * C::FI * 16;
    const int64_t jb = (int64_t)tj * C::TJ + (w % C::WJ) * C::FJ * 16;
    const float f = p.pow2[1];
    store16<C>(acc, p.dW, p.ldw, p.dw.I, p.dw.J, ib, jb, p.dw_vec, smem, [&](int x, int y) {
        const f32x4_t &a = acc[x][y];
        return u32x2_t{C::T::pack2(a[0] * f, a[1] * f), C::T::pack2(a[2] * f, a[3] * f)};
    });
}

template <class CX, class CW>
__global__ __launch_bounds__(kThreads, CX::TI == 256 ? 1 : 2) void k_xent_both(BothParams p) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[CX::kLds > CW::kLds ? CX::kLds : CW::kLds];
    LB_LDS char *smem = (LB_LDS char *)smem_raw;
    const int b = blockIdx.x;
    const int lead = p.dx_first ? p.dx_tiles : p.dw_tiles;
    if ((b < lead) == (p.dx_first != 0))
        dx_tile<CX>(p, p.dx_first ? b : b - lead, smem);
    else
        dw_tile<CW>(p, p.dx_first ? b - lead : b, smem);
}

// dX from the ranges' partial sums, in range order
template <class T>
__global__ __launch_bounds__(256) void k_xent_dx_sum(const float *acc, int splits, int64_t M, int64_t K, int64_t Kp,
                                                     const float *pow2, uint16_t *dX, int vec) {
    const float f = pow2[1];
    const int64_t n = M * Kp / 4;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < n; q += (int64_t)gridDim.x * 256) {
        f32x4_t v = *reinterpret_cast<const f32x4_t *>(acc + 4 * q);
        for (int s = 1; s < splits; ++s)
            v += *reinterpret_cast<const f32x4_t *>(acc + (int64_t)s * M * Kp + 4 * q);
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
}

template <class T, int ROWS>
struct BwdCfg;
template <class T> struct BwdCfg<T, xent::ROWS32> {
    using X = Cfg<T, 1, 4, 2, 2, false, false, 4>;
    using W = Cfg<T, 2, 2, 4, 4, true, true, 2>;
};
template <class T> struct BwdCfg<T, xent::ROWS64> {
    using X = Cfg<T, 1, 4, 4, 2, false, false, 3>;
    using W = Cfg<T, 2, 2, 4, 4, true, true, 2>;
};
template <class T> struct BwdCfg<T, xent::ROWS128> {
    using X = Cfg<T, 2, 2, 4, 4, false, false, 2>;
    using W = Cfg<T, 2, 2, 4, 4, true, true, 2>;
};
template <class T> struct BwdCfg<T, xent::ROWS256> {
    using X = Cfg<T, 2, 2, 8, 8, false, false, 2>;
    using W = Cfg<T, 2, 2, 8, 8, true, true, 2>;
};

template <class T, int ROWS>
void piece_bwd(GradParams &g, BothParams &p, bool want_dx, bool want_dw, hipStream_t s) {
    using CG = typename FwdCfg<T, ROWS>::C;
    using CX = typename BwdCfg<T, ROWS>::X;
    using CW = typename BwdCfg<T, ROWS>::W;
    set_tiles<CG>(g.job);
    // G's padding columns (up to a multiple of 64) are zeroed by the tiles that own them
    g.job.tiles_j = (int)cdiv(g.Vg, CG::TJ);
    hipLaunchKernelGGL((k_xent_grad<CG>), dim3((unsigned)(g.job.tiles_i * g.job.tiles_j)), dim3(kThreads), 0, s, g);
    set_tiles<CX>(p.dx);
    set_tiles<CW>(p.dw);
    p.dx_tiles = want_dx ? p.dx.tiles_i * p.dx.tiles_j * p.splits : 0;
    p.dw_tiles = want_dw ? p.dw.tiles_i * p.dw.tiles_j : 0;
    p.dx_first = p.split_len * CX::TI * CX::TJ >= p.dw.R * CW::TI * CW::TJ;
    hipLaunchKernelGGL((k_xent_both<CX, CW>), dim3((unsigned)(p.dx_tiles + p.dw_tiles)), dim3(kThreads), 0, s, p);
}

template <class T>
hipError_t backward(const XentBwdArgs &a, hipStream_t s) {
    const bool pack_w = a.V % 8 != 0 || !aligned(a.W, 16);
    const xent::Bwd b = xent::backward(a.M, a.K, a.V, pack_w);
    char *const ws = static_cast<char *>(a.ws);
    RowParam *const row = reinterpret_cast<RowParam *>(ws + b.off_row);
    float *const pow2 = reinterpret_cast<float *>(ws + b.off_row + 16 * a.M);
    uint16_t *const x = reinterpret_cast<uint16_t *>(ws + b.off_x);
    uint16_t *const wp = reinterpret_cast<uint16_t *>(ws + b.off_w);
    RowsParams rows{a.target, a.lse, a.row_scale, a.d_scale, a.scale, a.M, a.V, a.f16, row, pow2};
    hipLaunchKernelGGL(k_xent_rows, dim3(1), dim3(1024), 0, s, rows);
    pack(a.X, a.K, a.M, a.K, x, b.Kp, row, s);
    const bool dx_vec = a.K % 4 == 0 && aligned(a.dX, 8);
    for (int64_t v0 = 0; v0 < a.V; v0 += b.Vc) {
        const int64_t vc = std::min(b.Vc, a.V - v0);
        const uint16_t *w = static_cast<const uint16_t *>(a.W) + v0;
        int64_t ldw = a.V;
        if (pack_w) {
            pack(w, a.V, a.K, vc, wp, b.Vc, nullptr, s);
            w = wp;
            ldw = b.Vc;
        }
        GradParams g{};
        g.job.a = x;
        g.job.lda = b.Kp;
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
        p.pow2 = pow2;
        switch (b.rows) {
        case xent::ROWS32: piece_bwd<T, xent::ROWS32>(g, p, a.dX, a.dW, s); break;
        case xent::ROWS64: piece_bwd<T, xent::ROWS64>(g, p, a.dX, a.dW, s); break;
        case xent::ROWS128: piece_bwd<T, xent::ROWS128>(g, p, a.dX, a.dW, s); break;
        default: piece_bwd<T, xent::ROWS256>(g, p, a.dX, a.dW, s); break;
        }
    }
    if (a.dX && b.splits > 1) {
        const int64_t blocks = std::min<int64_t>(cdiv(a.M * b.Kp / 4, 256), 8 * xent::kCUs);
        hipLaunchKernelGGL((k_xent_dx_sum<T>), dim3((unsigned)blocks), dim3(256), 0, s,
                           reinterpret_cast<const float *>(ws + b.off_acc), b.splits, a.M, a.K, b.Kp, pow2,
                           static_cast<uint16_t *>(a.dX), (int)dx_vec);
    }
    return hipGetLastError();
}

template <class T>
hipError_t forward(const XentArgs &a, hipStream_t s) {
    const bool pack_w = a.V % 8 != 0 || !aligned(a.W, 16);
    const xent::Fwd f = xent::forward(a.M, a.K, a.V, pack_w);
    char *const ws = static_cast<char *>(a.ws);
    StatsParams p{};
    p.job.a = static_cast<const uint16_t *>(a.X);
    p.job.lda = a.K;
    if (a.K % 8 != 0 || !aligned(a.X, 16)) {
        uint16_t *const x = reinterpret_cast<uint16_t *>(ws + f.off_x);
        pack(a.X, a.K, a.M, a.K, x, f.Kp, nullptr, s);
        p.job.a = x;
        p.job.lda = f.Kp;
    }
    p.job.I = a.M;
    p.job.R = a.K;
    p.target = a.target;
    p.part = reinterpret_cast<float2 *>(ws + f.off_part);
    p.zt = reinterpret_cast<float *>(ws + f.off_zt);
    JoinParams j{};
    j.part = p.part;
    j.run = reinterpret_cast<float2 *>(ws + f.off_run);
    j.zt = p.zt;
    j.target = a.target;
    j.loss = a.loss;
    j.lse = a.lse;
    j.M = a.M;
    j.V = a.V;
    j.rb = 64;
    while (j.rb > 1 && j.rb / 2 >= a.M)
        j.rb /= 2;
    const bool one = a.M <= j.rb; // one block joins every row and can write the mean
    j.out = one ? a.out : nullptr;
    for (int64_t v0 = 0; v0 < a.V; v0 += f.Vc) {
        const int64_t vc = std::min(f.Vc, a.V - v0);
        const uint16_t *w = static_cast<const uint16_t *>(a.W) + v0;
        p.job.ldb = a.V;
        if (pack_w) {
            uint16_t *const wp = reinterpret_cast<uint16_t *>(ws + f.off_w);
            pack(w, a.V, a.K, vc, wp, f.Vc, nullptr, s);
            w = wp;
            p.job.ldb = f.Vc;
        }
        p.job.b = w;
        p.job.J = vc;
        p.v0 = v0;
        stats<T>(f.rows, p, s);
        j.parts = xent::up(vc, xent::tile_cols(f.rows)) / f.wcols;
        j.first = v0 == 0;
        j.last = v0 + f.Vc >= a.V;
        hipLaunchKernelGGL(k_xent_join, dim3((unsigned)cdiv(a.M, j.rb)), dim3(1024), 0, s, j);
    }
    if (!one)
        hipLaunchKernelGGL(k_xent_mean, dim3(1), dim3(1024), 0, s, a.loss, a.target, a.M, a.out);
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
        hipLaunchKernelGGL(k_xent_mean, dim3(1), dim3(1024), 0, s, a.loss, a.target, (int64_t)0, a.out);
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
