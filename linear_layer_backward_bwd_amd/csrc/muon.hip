// Muon on gfx950: momentum, Newton-Schulz orthogonalisation, weight update.
//
//     g = float(grad)·inv_scale·clip      mom = β·mom + g
//     u = g + β·mom (Nesterov) or mom     X = u / ‖u‖_F
//     repeat: A = X·Xᵀ   B = b·A + c·A²   X = a·X + B·X       (a, b, c below)
//     W = W − lr·(scale·X + wd·W)
//
// The polynomial a·σ + b·σ³ + c·σ⁵ acts on the singular values of X and moves all of
// them towards 1.  The products run on the shorter side: A = X·Xᵀ for K <= N, XᵀX and
// X·B for K > N; with the tile's two operand layouts no transpose is stored.
//
// Numbers.  All operands of the products are fp16 (11 bits; bf16's 8 gave errors of 1%
// after five steps on noise, fp16 0.13%), scaled by fixed powers of two: singular
// values stay in [0, 1.21] (the polynomial's maximum on that interval is 1.202), so
// |X| <= 1.21, |A| <= 1.47 and |B| <= 2.81 entry by entry, and 2^15·X, 2^14·A, 2^14·B stay
// below 65504 while entries down to 2^-29 of the largest singular value keep 11 bits.
// Sums are fp32; the norm is summed in fp64; momentum and W are fp32 throughout.
// Each X, A and B is rounded once.
#include "kernels.h"
#include "plan_muon.h"
#include "tile.h"

#include <algorithm>

namespace lb {
namespace {

using namespace tile;
using muon::cdiv;

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kX = 32768.0f; // 2^15: stored X / X
constexpr float kG = 16384.0f; // 2^14: stored A / A, stored B / B

// ---- momentum and norm -------------------------------------------------------------------
template <int GT>
__device__ __forceinline__ float grad_at(const void *g, int64_t i) {
    if constexpr (GT == GRAD_F32)
        return static_cast<const float *>(g)[i];
    else if constexpr (GT == GRAD_F16)
        return f16_bits_to_f32(static_cast<const uint16_t *>(g)[i]);
    else
        return bf16_bits_to_f32(static_cast<const uint16_t *>(g)[i]);
}
// Vectors at any alignment of their elements: one instruction where a scalar loop takes four
// (3 x 2050 rows of 515 floats: momentum and norm 10.6 -> 7.6 us, scaling 15.9 -> 8.6,
// as with rows of 512).
typedef f32x4_t f32x4_any __attribute__((aligned(4)));
typedef u32x2_t u32x2_any __attribute__((aligned(2)));
template <int GT>
__device__ __forceinline__ f32x4_t grad4_at(const void *g, int64_t i) {
    if constexpr (GT == GRAD_F32) {
        return *reinterpret_cast<const f32x4_any *>(static_cast<const float *>(g) + i);
    } else {
        const u32x2_t h = *reinterpret_cast<const u32x2_any *>(static_cast<const uint16_t *>(g) + i);
        if constexpr (GT == GRAD_F16)
            return f32x4_t{F16::f32(h[0]), F16::f32(h[0] >> 16), F16::f32(h[1]), F16::f32(h[1] >> 16)};
        else
            return f32x4_t{BF16::f32(h[0]), BF16::f32(h[0] >> 16), BF16::f32(h[1]), BF16::f32(h[1] >> 16)};
    }
}

struct PrepParams {
    const void *g;
    float *mom; // or null: u = g
    int64_t K, N, Np;
    float inv_scale, beta;
    const float *clip;
    const int32_t *skip;
    int nesterov, parts;
    double *part; // [batch][parts]
    uint16_t *x;  // [batch][K][Np]
};

__device__ __forceinline__ float unscaled(float g, float inv_scale, float clip) {
    return __fmul_rn(__fmul_rn(g, inv_scale), clip);
}
__device__ __forceinline__ float update_of(float g, float mom, const PrepParams &p) {
    return !p.mom ? g : p.nesterov ? __fadd_rn(g, __fmul_rn(p.beta, mom)) : mom;
}

// mom is updated in place; block j of a matrix sums u² over its share (fixed order).
// HBM-bound: one read of grad, one read and write of mom (4096 x 12288, bf16: 86 us, 5.8 TB/s
// with 1024 blocks; 256 blocks took 150).
template <int GT>
__global__ __launch_bounds__(256) void k_muon_norm(PrepParams p) {
    if (p.skip && *p.skip)
        return;
    __shared__ double sh[256];
    const float clip = p.clip ? *p.clip : 1.0f;
    const int64_t n = p.K * p.N, base = (int64_t)blockIdx.y * n;
    double s = 0.0;
    auto add = [&](float &g, float &m) {
        g = unscaled(g, p.inv_scale, clip);
        m = __fadd_rn(__fmul_rn(p.beta, m), g);
        const double u = (double)update_of(g, m, p);
        s += u * u;
    };
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i + 4 <= n; i += (int64_t)p.parts * 256 * 4) {
        f32x4_t g = grad4_at<GT>(p.g, base + i), m{};
        if (p.mom)
            m = *reinterpret_cast<const f32x4_any *>(p.mom + base + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float ge = g[e], me = m[e];
            add(ge, me);
            m[e] = me;
        }
        if (p.mom)
            *reinterpret_cast<f32x4_any *>(p.mom + base + i) = m;
    }
    if (blockIdx.x == 0 && (int)threadIdx.x < (int)(n & 3)) { // what four elements at a time leave
        const int64_t i = base + n - 1 - threadIdx.x;
        float g = grad_at<GT>(p.g, i), m = p.mom ? p.mom[i] : 0.0f;
        add(g, m);
        if (p.mom)
            p.mom[i] = m;
    }
    sh[threadIdx.x] = s;
    __syncthreads();
    for (int h = 128; h > 0; h >>= 1) {
        if ((int)threadIdx.x < h)
            sh[threadIdx.x] += sh[threadIdx.x + h];
        __syncthreads();
    }
    if (threadIdx.x == 0)
        p.part[(int64_t)blockIdx.y * p.parts + blockIdx.x] = sh[0];
}

// X = u / ‖u‖_F in fp16, rows padded with zeros to a multiple of 64.  ‖u‖ = 0 gives 0, a
// norm that is infinite or NaN gives NaN throughout.  HBM-bound (4096 x 12288: 88 us, 4.6
// TB/s); rows and columns are walked without a division per element, which took as long as
// the memory.
template <int GT, bool TAIL> // TAIL: N is no multiple of 4
__global__ __launch_bounds__(256) void k_muon_scale(PrepParams p) {
    if (p.skip && *p.skip)
        return;
    __shared__ double sh[256];
    double mine = 0.0;
    for (int i = threadIdx.x; i < p.parts; i += 256)
        mine += p.part[(int64_t)blockIdx.y * p.parts + i];
    sh[threadIdx.x] = mine;
    __syncthreads();
    for (int h = 128; h > 0; h >>= 1) {
        if ((int)threadIdx.x < h)
            sh[threadIdx.x] += sh[threadIdx.x + h];
        __syncthreads();
    }
    // 2^15 / ‖u‖ as a float in [0.5, 1) and a power of two: no intermediate leaves fp32's range
    const double norm = sqrt(sh[0]);
    int e = 0;
    const float f = norm == 0.0 ? 0.0f : norm < INFINITY ? (float)frexp((double)kX / norm, &e) : NAN;
    const float clip = p.clip ? *p.clip : 1.0f;
    const int64_t base = (int64_t)blockIdx.y * p.K * p.N;
    uint16_t *const x = p.x + (int64_t)blockIdx.y * p.K * p.Np;
    const int64_t per = p.Np / 8, first = (int64_t)blockIdx.x * 256 + threadIdx.x, stride = (int64_t)gridDim.x * 256;
    const int64_t step_r = stride / per, step_q = stride - step_r * per;
    int64_t r = first / per, q = first - r * per; // one division, then steps
    for (; r < p.K; r += step_r, q += step_q) {
        if (q >= per) {
            q -= per;
            if (++r >= p.K)
                break;
        }
        const int64_t c = q * 8, i = base + r * p.N + c;
        f32x4_t g[2] = {}, m[2] = {};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t left = p.N - (c + 4 * k);
            if (left >= (TAIL ? 4 : 1)) {
                g[k] = grad4_at<GT>(p.g, i + 4 * k);
                if (p.mom)
                    m[k] = *reinterpret_cast<const f32x4_any *>(p.mom + i + 4 * k);
            } else if (TAIL) {
#pragma unroll
                for (int d = 0; d < 3; ++d)
                    if (d < left) {
                        g[k][d] = grad_at<GT>(p.g, i + 4 * k + d);
                        m[k][d] = p.mom ? p.mom[i + 4 * k + d] : 0.0f;
                    }
            }
        }
        u32x4_t h;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float u[2];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const int n = 2 * k + d;
                const float v = update_of(unscaled(g[n >> 2][n & 3], p.inv_scale, clip), m[n >> 2][n & 3], p);
                u[d] = c + n < p.N ? ldexpf(v, e) * f : 0.0f; // a padding column stays 0 whatever f is
            }
            h[k] = F16::pack2(u[0], u[1]);
        }
        *reinterpret_cast<u32x4_t *>(x + r * p.Np + c) = h;
    }
}

// ---- the products -------------------------------------------------------------------------
enum Step {
    GRAM,   // out = f·sum
    ADD,    // out = f·sum + fa·add
    ORTH,   // o = (f·sum + fa·add), 16 bit, the caller's matrix
    UPDATE, // W -= lr·(scale·(f·sum + fa·add) + wd·W), and its 16-bit copy
};

struct ProductParams {
    Job job;
    int tiles;              // of one matrix
    int64_t step_a, step_b; // elements from one matrix to the next
    float f, fa;
    const uint16_t *add; // fp16
    int64_t ld_add, step_add;
    uint16_t *out; // fp16, ld a multiple of 64
    int64_t ld_out, step_out;
    // the caller's matrices, [batch][I][J]
    uint16_t *o;
    float *W;
    uint16_t *W16;
    int o_bf16; // type of o / W16
    float lr, scale, wd;
    const int32_t *skip;
};

__device__ __forceinline__ f32x4_t f16x4(const u32x2_t &h) {
    return f32x4_t{F16::f32(h[0]), F16::f32(h[0] >> 16), F16::f32(h[1]), F16::f32(h[1] >> 16)};
}

// A 4 x 4 block of 16-bit values held by four neighbouring lanes (lane q: row q) transposed:
// lane q gets the values of column mirror_row(q).  Two exchanges within the quad.
__device__ __forceinline__ int mirror_row(int lane) { return ((lane & 1) << 1) | ((lane >> 1) & 1); }
__device__ __forceinline__ u32x2_t transposed4(const u32x2_t &h, int lane) {
    const bool odd = lane & 1, upper = lane & 2;
    const uint32_t own = odd ? h[1] : h[0];
    const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)(odd ? h[0] : h[1]), 0xB1, 0xf, 0xf, true); // lane ^ 1
    const uint32_t lo = odd ? got : own, hi = odd ? own : got;
    const uint32_t d0 = (lo & 0xffffu) | (hi << 16), d1 = (lo >> 16) | (hi & 0xffff0000u);
    const uint32_t far = (uint32_t)__builtin_amdgcn_mov_dpp((int)(upper ? d0 : d1), 0x4E, 0xf, 0xf, true); // lane ^ 2
    return upper ? u32x2_t{far, d1} : u32x2_t{d0, far};
}

// GRAM and the ADD that makes B are symmetric (SYM): only the tiles on and below
// the diagonal run, and each stores its mirror image too.  What is added is loaded one
// round of the epilogue ahead (the first before the main loop): with the loads in the
// round that uses them, A² at 4096 took 120 us.
template <class C, int STEP, bool SYM>
__device__ __forceinline__ void store_small(const ProductParams &p, const Job &job, int64_t b, int ti, int tj,
                                            LB_LDS char *smem) {
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t I = job.I, Jp = (job.J + 7) / 8 * 8;
    const int64_t ib = (int64_t)ti * C::TI + (w / C::WJ) * C::FI * 16;
    const int64_t jb = (int64_t)tj * C::TJ + (w % C::WJ) * C::FJ * 16;
    const uint16_t *const add = p.add + b * p.step_add;
    uint16_t *const out = p.out + b * p.step_out;
    u32x2_t next[2][C::FJ], cur[2][C::FJ];
    // rows past I read zero, columns past the padding are another row's and not stored
    const uint32_t add_off = (uint32_t)((lane & 15) * p.ld_add + 4 * (lane >> 4)) * 2;
    auto load = [&](int h) {
        if constexpr (STEP == ADD) {
            const int64_t i0 = ib + 32 * h, rows = max<int64_t>(0, min<int64_t>(32, I - i0));
            const __amdgpu_buffer_rsrc_t rs =
                rsrc(add + i0 * p.ld_add + jb, rows && jb < Jp ? (uint32_t)((rows * p.ld_add - jb) * 2) : 0u);
#pragma unroll
            for (int xx = 0; xx < 2; ++xx)
#pragma unroll
                for (int y = 0; y < C::FJ; ++y)
                    next[xx][y] = __builtin_bit_cast(
                        u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(
                                     rs, (int)(add_off + 32 * xx * (uint32_t)p.ld_add + 32 * y), 0, 0));
        }
    };
    load(0);
    Acc<C> acc;
    accumulate<C>(job, ti, tj, smem, acc);
    const bool mirror = SYM && ti != tj;
    // the wave's mirror image: FJ*16 rows from row jb, from column ib on
    const int64_t mrows = max<int64_t>(0, min<int64_t>(C::FJ * 16, I - jb));
    const __amdgpu_buffer_rsrc_t mrs = rsrc(out + jb * p.ld_out + ib, (uint32_t)(mrows * p.ld_out * 2));
    const uint32_t mirror_off =
        (uint32_t)((4 * (lane >> 4) + mirror_row(lane)) * p.ld_out + (lane & 12)) * 2;
    store16<C>(
        acc, out, p.ld_out, I, Jp, ib, jb, true, false, smem,
        [&](int h) {
#pragma unroll
            for (int xx = 0; xx < 2; ++xx)
#pragma unroll
                for (int y = 0; y < C::FJ; ++y)
                    cur[xx][y] = next[xx][y];
            if (h + 1 < C::FI / 2)
                load(h + 1);
        },
        [&](int x, int y) {
            f32x4_t t;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                t[e] = p.f * acc[x][y][e];
            if constexpr (STEP == ADD) {
                const f32x4_t a = f16x4(cur[x & 1][y]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    t[e] = __builtin_fmaf(p.fa, a[e], t[e]);
            }
            const u32x2_t h = {F16::pack2(t[0], t[1]), F16::pack2(t[2], t[3])};
            if (mirror) {
                const uint32_t skip = (uint32_t)!(ib + 16 * x + (lane & 12) < Jp) << 31; // padding columns: zero
                __builtin_amdgcn_raw_buffer_store_b64(
                    transposed4(h, lane), mrs,
                    (int)((mirror_off + 32 * y * (uint32_t)p.ld_out + 32 * x) | skip), 0, 0);
            }
            return h;
        });
}

// The last product, on the caller's matrices.  What a round combines with (X, and W of
// UPDATE) is loaded a round ahead through descriptors of the round's 16 rows, which drop the
// rows past I (a chunk over a row's end reads into the next row and does not use it).  VEC:
// rows take 4 elements at a time, and the stores go through such descriptors too.
template <class C, int STEP, bool VEC>
__device__ __forceinline__ void store_last(const ProductParams &p, const Job &job, int64_t b, int ti, int tj,
                                           LB_LDS char *smem) {
    Acc<C> acc;
    accumulate<C>(job, ti, tj, smem, acc);
    constexpr int kChunks = 4 * C::FJ;
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t i0 = (int64_t)ti * C::TI, j0 = (int64_t)tj * C::TJ;
    const int64_t I = job.I, J = job.J, mine = b * I * J;
    const int64_t iw = i0 + (wv / C::WJ) * C::FI * 16, jw = j0 + (wv % C::WJ) * C::FJ * 16; // the wave's corner
    const uint16_t *const add = p.add + b * p.step_add;
    const int lr = lane / kChunks, lc = 4 * (lane % kChunks);
    const uint32_t skip = (uint32_t)!(jw + lc < J) << 31;
    const uint32_t off_x = (uint32_t)(lr * p.ld_add + lc) * 2 | skip, off_w = (uint32_t)(lr * J + lc) * 4 | skip;
    // bytes of the round's rows from the wave's first column on, `cols` columns a row
    auto window = [&](int k, int64_t ld, int bytes, int64_t cols) {
        const int64_t rows = max<int64_t>(0, min<int64_t>(16, I - (iw + 16 * k)));
        return rows && jw < J ? (uint32_t)(((rows - 1) * ld + cols - jw) * bytes) : 0u;
    };
    u32x2_t x[2][C::FJ];
    f32x4_t w[2][C::FJ];
    auto load = [&](int k, int rows) {
        const int64_t i = iw + 16 * k;
        const __amdgpu_buffer_rsrc_t rx = rsrc(add + i * p.ld_add + jw, window(k, p.ld_add, 2, (J + 3) / 4 * 4));
        const __amdgpu_buffer_rsrc_t rw =
            rsrc(STEP == UPDATE ? p.W + mine + i * J + jw : nullptr, STEP == UPDATE ? window(k, J, 4, J) : 0u);
#pragma unroll
        for (int q = 0; q < C::FJ; ++q) {
            x[k & 1][q] = __builtin_bit_cast(
                u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(rx, (int)(off_x + (uint32_t)(q * rows * p.ld_add * 2)),
                                                              0, 0));
            if constexpr (STEP == UPDATE)
                w[k & 1][q] = __builtin_bit_cast(
                    f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, (int)(off_w + (uint32_t)(q * rows * J * 4)),
                                                                   0, 0));
        }
    };
    auto stepped = [&](float old, float o) { return old - p.lr * (p.scale * o + p.wd * old); };
    staged<C>(
        acc, i0, j0, smem,
        [&](int k, int64_t, int rows, int64_t) {
            if (k == 0)
                load(0, rows);
            if (k + 1 < C::FI)
                load(k + 1, rows);
        },
        [&](int k, int64_t i, int rows, int64_t j, f32x4_t (&v)[C::FJ]) {
            if constexpr (VEC) {
                const int64_t r0 = iw + 16 * k;
                const __amdgpu_buffer_rsrc_t ro = rsrc(STEP == ORTH ? p.o + mine + r0 * J + jw : nullptr,
                                                       STEP == ORTH ? window(k, J, 2, J) : 0u);
                const __amdgpu_buffer_rsrc_t rw = rsrc(STEP == UPDATE ? p.W + mine + r0 * J + jw : nullptr,
                                                       STEP == UPDATE ? window(k, J, 4, J) : 0u);
                const bool copy = STEP == UPDATE && p.W16;
                const __amdgpu_buffer_rsrc_t rc =
                    rsrc(copy ? p.W16 + mine + r0 * J + jw : nullptr, copy ? window(k, J, 2, J) : 0u);
#pragma unroll
                for (int q = 0; q < C::FJ; ++q) {
                    const f32x4_t a = f16x4(x[k & 1][q]);
                    f32x4_t t;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        t[e] = __builtin_fmaf(p.fa, a[e], p.f * v[q][e]);
                    const uint32_t o4 = off_w + (uint32_t)(q * rows * J * 4);
                    const uint32_t o2 = (uint32_t)((lr + q * rows) * J + lc) * 2 | skip;
                    if constexpr (STEP == UPDATE) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            t[e] = stepped(w[k & 1][q][e], t[e]);
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, t), rw, (int)o4, 0, 0);
                    }
                    const u32x2_t h = p.o_bf16 ? u32x2_t{BF16::pack2(t[0], t[1]), BF16::pack2(t[2], t[3])}
                                               : u32x2_t{F16::pack2(t[0], t[1]), F16::pack2(t[2], t[3])};
                    if constexpr (STEP == ORTH)
                        __builtin_amdgcn_raw_buffer_store_b64(h, ro, (int)o2, 0, 0);
                    else
                        __builtin_amdgcn_raw_buffer_store_b64(h, rc, (int)o2, 0, 0); // dropped without a copy
                }
            } else { // rows at any element: the chunk over a row's end element by element
#pragma unroll
                for (int q = 0; q < C::FJ; ++q) {
                    const int64_t r = i + q * rows;
                    if (r >= I || j >= J)
                        continue;
                    const f32x4_t a = f16x4(x[k & 1][q]);
                    f32x4_t t;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        t[e] = __builtin_fmaf(p.fa, a[e], p.f * v[q][e]);
                        if constexpr (STEP == UPDATE)
                            t[e] = stepped(w[k & 1][q][e], t[e]);
                    }
                    const u32x2_t h = p.o_bf16 ? u32x2_t{BF16::pack2(t[0], t[1]), BF16::pack2(t[2], t[3])}
                                               : u32x2_t{F16::pack2(t[0], t[1]), F16::pack2(t[2], t[3])};
                    const int64_t at = mine + r * J + j;
                    uint16_t *const o = STEP == ORTH ? p.o : p.W16; // W16 may be null
                    if (j + 4 <= J) {
                        if constexpr (STEP == UPDATE)
                            *reinterpret_cast<f32x4_any *>(p.W + at) = t;
                        if (o)
                            *reinterpret_cast<u32x2_any *>(o + at) = h;
                    } else {
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            if (j + e < J) {
                                if constexpr (STEP == UPDATE)
                                    p.W[at + e] = t[e];
                                if (o)
                                    o[at + e] = (uint16_t)(h[e >> 1] >> (16 * (e & 1)));
                            }
                    }
                }
            }
        });
}

// FLAG: SYM of GRAM and ADD, VEC of ORTH and UPDATE.  At 4096 x 12288: A 260 us (lower tiles:
// 136 of 256 CUs, 2.2 GHz), B 105, X 335 (1.23 PFLOP/s), the last one with W, mom's update and
// the 16-bit copy 381.  At 12 x 1024 x 1024: 23, 26, 37 and 45 us.
template <class C, int STEP, bool FLAG>
__global__ __launch_bounds__(kThreads, C::kLds > 80 * 1024 ? 1 : 2) void k_muon_product(ProductParams p) {
    if (p.skip && *p.skip)
        return;
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::kLds];
    LB_LDS char *smem = (LB_LDS char *)smem_raw;
    const int u = gathered(blockIdx.x, gridDim.x); // over the whole batch
    const int64_t b = u / p.tiles;
    Job job = p.job;
    job.a += b * p.step_a;
    job.b += b * p.step_b;
    int ti, tj;
    if constexpr ((STEP == GRAM || STEP == ADD) && FLAG)
        coords_lower(u - (int)b * p.tiles, ti, tj);
    else
        coords(job, u - (int)b * p.tiles, ti, tj);
    if constexpr (STEP == GRAM || STEP == ADD)
        store_small<C, STEP, FLAG>(p, job, b, ti, tj, smem);
    else
        store_last<C, STEP, FLAG>(p, job, b, ti, tj, smem);
}

template <class C, int STEP, bool FLAG>
void launch(ProductParams &p, int64_t batch, hipStream_t s) {
    p.job.tiles_i = (int)cdiv(p.job.I, C::TI);
    p.job.tiles_j = (int)cdiv(p.job.J, C::TJ);
    p.job.group = 4;
    const int64_t tiles = (STEP == GRAM || STEP == ADD) && FLAG
                              ? (int64_t)p.job.tiles_i * (p.job.tiles_i + 1) / 2
                              : (int64_t)p.job.tiles_i * p.job.tiles_j;
    p.tiles = (int)tiles;
    hipLaunchKernelGGL((k_muon_product<C, STEP, FLAG>), dim3((unsigned)(tiles * batch)), dim3(kThreads), 0, s, p);
}
template <bool AOC, bool BOC, int STEP, bool FLAG>
void product_with(muon::Tile tile, ProductParams &p, int64_t batch, hipStream_t s) {
    switch (tile) {
    case muon::TILE256: launch<Cfg<F16, 2, 2, 8, 8, AOC, BOC, 2, 3>, STEP, FLAG>(p, batch, s); break;
    case muon::TILE128: launch<Cfg<F16, 2, 2, 4, 4, AOC, BOC, 2>, STEP, FLAG>(p, batch, s); break;
    case muon::TILE128_DEEP: launch<Cfg<F16, 2, 2, 4, 4, AOC, BOC, 4>, STEP, FLAG>(p, batch, s); break;
    default: launch<Cfg<F16, 2, 2, 2, 2, AOC, BOC, 4>, STEP, FLAG>(p, batch, s); break;
    }
}
template <bool AOC, bool BOC, int STEP, bool FLAG>
void product(ProductParams &p, int64_t batch, hipStream_t s) {
    product_with<AOC, BOC, STEP, FLAG>(muon::choose(batch, p.job.I, p.job.J, p.job.R, false).tile, p, batch, s);
}
template <bool AOC, bool BOC, int STEP>
void symmetric_product(ProductParams &p, int64_t batch, hipStream_t s) {
    const muon::Choice c = muon::choose(batch, p.job.I, p.job.J, p.job.R, true);
    if (c.lower)
        product_with<AOC, BOC, STEP, true>(c.tile, p, batch, s);
    else
        product_with<AOC, BOC, STEP, false>(c.tile, p, batch, s);
}
// A and B = bA + cA² of a matrix whose shorter side fits one tile: the block writes A, in
// fp16, to LDS as RC pairs (the ring is free by then), multiplies it by itself from there
// and adds bA from its own registers.  Neither A nor a second launch touches memory.
// PARTS: A's sums come from `sums`, p.tiles ranges per matrix (k_muon_gram_part), added in
// range order.
template <class C, bool PARTS>
__global__ __launch_bounds__(kThreads, C::kLds > 80 * 1024 ? 1 : 2) void k_muon_poly(ProductParams p, float f2,
                                                                                     const f32x4_t *sums) {
    static_assert(C::TI == C::TJ && C::FI == C::FJ && C::WI == 2, "one square tile");
    if (p.skip && *p.skip)
        return;
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::kLds];
    LB_LDS char *smem = (LB_LDS char *)smem_raw;
    constexpr int T = C::TI, F = C::FI;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Job job = p.job;
    Acc<C> acc;
    if constexpr (PARTS) {
#pragma unroll
        for (int x = 0; x < F; ++x)
#pragma unroll
            for (int y = 0; y < F; ++y) {
                const f32x4_t *q = sums + ((int64_t)blockIdx.x * p.tiles * F * F + x * F + y) * 256 + threadIdx.x;
                f32x4_t t = *q;
                for (int r = 1; r < p.tiles; ++r)
                    t += q[(int64_t)r * F * F * 256];
                acc[x][y] = t;
            }
    } else {
        job.a += blockIdx.x * p.step_a;
        job.b += blockIdx.x * p.step_b;
        accumulate<C>(job, 0, 0, smem, acc);
    }
    // A as T/64 pairs of T rows of 128 bytes, chunk c of row o at c ^ (o % 8)
    u32x2_t a[F][F];
#pragma unroll
    for (int x = 0; x < F; ++x) {
        pin(acc[x]);
#pragma unroll
        for (int y = 0; y < F; ++y) {
            const int i = (w / 2) * F * 16 + 16 * x + (lane & 15), j = (w % 2) * F * 16 + 16 * y + 4 * (lane >> 4);
            const f32x4_t &t = acc[x][y];
            a[x][y] = u32x2_t{F16::pack2(p.f * t[0], p.f * t[1]), F16::pack2(p.f * t[2], p.f * t[3])};
            *reinterpret_cast<LB_LDS u32x2_t *>(smem + (j >> 6) * (T * 128) + i * 128 +
                                                ((((j & 63) >> 3) ^ (i & 7)) << 4) + (j & 4) * 2) = a[x][y];
            acc[x][y] = f32x4_t{};
        }
    }
    __syncthreads();
    Frags<T, false, F, 2> fa, fb;
    fa.init(smem, (w / 2) * F * 16, lane);
    fb.init(smem, (w % 2) * F * 16, lane);
    frag_half_t unused[F][2];
#pragma unroll
    for (int h = 0; h < T / 32; ++h) {
        u32x4_t af[F], bf[F];
#pragma unroll
        for (int k = 0; k < F; ++k) {
            if (h & 1) {
                fa.template read<0, 1>(k, (h >> 1) * (T * 128), af, unused);
                fb.template read<0, 1>(k, (h >> 1) * (T * 128), bf, unused);
            } else {
                fa.template read<0, 0>(k, (h >> 1) * (T * 128), af, unused);
                fb.template read<0, 0>(k, (h >> 1) * (T * 128), bf, unused);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        Frags<T, false, F, 2>::settle(af, unused);
        Frags<T, false, F, 2>::settle(bf, unused);
#pragma unroll
        for (int x = 0; x < F; ++x)
#pragma unroll
            for (int y = 0; y < F; ++y)
                F16::mfma(acc[x][y], bf[y], af[x]);
    }
    mfma_drain();
    __syncthreads(); // every wave has read A: the epilogue may stage over it
    store16<C>(
        acc, p.out + blockIdx.x * p.step_out, p.ld_out, job.I, (job.J + 7) / 8 * 8, (w / 2) * F * 16, (w % 2) * F * 16,
        true, false, smem, [](int) {},
        [&](int x, int y) {
            const f32x4_t old = f16x4(a[x][y]);
            f32x4_t t;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                t[e] = __builtin_fmaf(p.fa, old[e], f2 * acc[x][y][e]);
            return u32x2_t{F16::pack2(t[0], t[1]), F16::pack2(t[2], t[3])};
        });
}

// One range of that tile's reduction: its sums in fragment order, 16 bytes a lane.
template <class C>
__global__ __launch_bounds__(kThreads, C::kLds > 80 * 1024 ? 1 : 2) void k_muon_gram_part(ProductParams p, int64_t len,
                                                                                          f32x4_t *sums) {
    if (p.skip && *p.skip)
        return;
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::kLds];
    constexpr int F = C::FI;
    Job job = p.job;
    const int64_t r0 = blockIdx.x * len; // a multiple of 64
    job.a += blockIdx.y * p.step_a + (C::AOC ? r0 * job.lda : r0);
    job.b = job.a;
    job.R = min<int64_t>(len, p.job.R - r0);
    Acc<C> acc;
    accumulate<C>(job, 0, 0, (LB_LDS char *)smem_raw, acc);
    f32x4_t *const q = sums + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * F * F * 256 + threadIdx.x;
#pragma unroll
    for (int x = 0; x < F; ++x) {
        pin(acc[x]);
#pragma unroll
        for (int y = 0; y < F; ++y)
            q[(x * F + y) * 256] = acc[x][y];
    }
}

template <class C>
void one_tile_as(int splits, ProductParams &p, float f2, f32x4_t *sums, int64_t batch, hipStream_t s) {
    if (splits > 1) {
        const int64_t len = muon::up(cdiv(p.job.R, splits), 64);
        p.tiles = (int)cdiv(p.job.R, len);
        hipLaunchKernelGGL((k_muon_gram_part<C>), dim3((unsigned)p.tiles, (unsigned)batch), dim3(kThreads), 0, s, p,
                           len, sums);
        hipLaunchKernelGGL((k_muon_poly<C, true>), dim3((unsigned)batch), dim3(kThreads), 0, s, p, f2,
                           (const f32x4_t *)sums);
    } else {
        hipLaunchKernelGGL((k_muon_poly<C, false>), dim3((unsigned)batch), dim3(kThreads), 0, s, p, f2,
                           (const f32x4_t *)nullptr);
    }
}
template <bool OC>
void one_tile_poly(const muon::Plan &pl, ProductParams &p, float f2, f32x4_t *sums, int64_t batch, hipStream_t s) {
    p.job.tiles_i = p.job.tiles_j = p.job.group = 1;
    if (pl.one == 64)
        one_tile_as<Cfg<F16, 2, 2, 2, 2, OC, OC, 4>>(pl.splits, p, f2, sums, batch, s);
    else
        one_tile_as<Cfg<F16, 2, 2, 4, 4, OC, OC, 4>>(pl.splits, p, f2, sums, batch, s);
}

template <int STEP>
void last_product(ProductParams &p, int64_t batch, bool tall, bool vec, hipStream_t s) {
    if (tall)
        vec ? product<false, false, STEP, true>(p, batch, s) : product<false, false, STEP, false>(p, batch, s);
    else
        vec ? product<false, true, STEP, true>(p, batch, s) : product<false, true, STEP, false>(p, batch, s);
}

template <int GT>
void prepare(PrepParams &p, int64_t batch, hipStream_t s) {
    const dim3 norm((unsigned)p.parts, (unsigned)batch);
    const dim3 scale((unsigned)std::min<int64_t>(cdiv(p.K * p.Np / 8, 256), std::max<int64_t>(16 * muon::kCUs / batch, 64)), (unsigned)batch);
    hipLaunchKernelGGL(k_muon_norm<GT>, norm, dim3(256), 0, s, p);
    if (p.N % 4)
        hipLaunchKernelGGL((k_muon_scale<GT, true>), scale, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((k_muon_scale<GT, false>), scale, dim3(256), 0, s, p);
}

bool aligned(const void *p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

} // namespace

hipError_t launch_muon(const MuonArgs &a, hipStream_t s) {
    if (a.batch == 0 || a.K == 0 || a.N == 0)
        return hipSuccess;
    const muon::Plan pl = muon::plan(a.batch, a.K, a.N);
    char *const ws = static_cast<char *>(a.ws);
    uint16_t *x = reinterpret_cast<uint16_t *>(ws + pl.off_x0), *y = reinterpret_cast<uint16_t *>(ws + pl.off_x1);
    uint16_t *const ga = reinterpret_cast<uint16_t *>(ws + pl.off_a);
    uint16_t *const gb = reinterpret_cast<uint16_t *>(ws + pl.off_b);
    PrepParams pp{a.grad, a.mom, a.K, a.N, pl.Np, a.inv_scale, a.beta, a.clip, a.skip, a.nesterov ? 1 : 0, pl.parts,
                  reinterpret_cast<double *>(ws + pl.off_part), x};
    if (a.gt == GRAD_F32)
        prepare<GRAD_F32>(pp, a.batch, s);
    else if (a.gt == GRAD_F16)
        prepare<GRAD_F16>(pp, a.batch, s);
    else
        prepare<GRAD_BF16>(pp, a.batch, s);

    const int64_t nx = a.K * pl.Np, ng = pl.s * pl.sp;
    ProductParams gram{}, poly{}, upd{};
    gram.job = Job{nullptr, nullptr, pl.Np, pl.Np, pl.s, pl.s, pl.tall ? a.K : a.N, 0, 0, 0};
    gram.step_a = gram.step_b = nx;
    gram.f = kG / (kX * kX);
    gram.out = ga;
    gram.ld_out = pl.sp;
    gram.step_out = ng;
    gram.skip = a.skip;
    poly.job = Job{ga, ga, pl.sp, pl.sp, pl.s, pl.s, pl.s, 0, 0, 0};
    poly.step_a = poly.step_b = poly.step_add = poly.step_out = ng;
    poly.f = kC / kG;
    poly.fa = kB;
    poly.add = ga;
    poly.ld_add = poly.ld_out = pl.sp;
    poly.out = gb;
    poly.skip = a.skip;
    upd.job = Job{nullptr, nullptr, 0, 0, a.K, a.N, pl.s, 0, 0, 0};
    upd.job.lda = pl.tall ? pl.Np : pl.sp;
    upd.job.ldb = pl.tall ? pl.sp : pl.Np;
    upd.step_a = pl.tall ? nx : ng;
    upd.step_b = pl.tall ? ng : nx;
    upd.ld_add = upd.ld_out = pl.Np;
    upd.step_add = upd.step_out = nx;
    upd.o = static_cast<uint16_t *>(a.O);
    upd.W = a.W;
    upd.W16 = static_cast<uint16_t *>(a.W16);
    upd.o_bf16 = a.o_bf16 ? 1 : 0;
    const bool rows4 = a.N % 4 == 0 && aligned(a.O, 8) && aligned(a.W, 16) && aligned(a.W16, 8);
    upd.lr = a.lr;
    upd.scale = a.scale;
    upd.wd = a.wd;
    upd.skip = a.skip;
    f32x4_t *const sums = reinterpret_cast<f32x4_t *>(ws + pl.off_sums);
    for (int t = 0; t < a.steps; ++t) {
        gram.job.a = gram.job.b = x;
        if (pl.one) { // A stays in LDS, B comes out
            gram.fa = kB;
            gram.out = gb;
            pl.tall ? one_tile_poly<true>(pl, gram, poly.f, sums, a.batch, s)
                    : one_tile_poly<false>(pl, gram, poly.f, sums, a.batch, s);
        } else if (pl.tall)
            symmetric_product<true, true, GRAM>(gram, a.batch, s);
        else
            symmetric_product<false, false, GRAM>(gram, a.batch, s);
        if (!pl.one)
            symmetric_product<false, false, ADD>(poly, a.batch, s);
        const bool last = t + 1 == a.steps;
        upd.job.a = pl.tall ? x : gb;
        upd.job.b = pl.tall ? gb : x;
        upd.add = x;
        upd.out = y;
        // stored X is 2^15·X, the sum 2^29·B·X; the last step leaves the powers of two
        upd.f = last ? 1.0f / (kX * kG) : 1.0f / kG;
        upd.fa = last ? kA / kX : kA;
        if (!last)
            pl.tall ? product<false, false, ADD, false>(upd, a.batch, s)
                    : product<false, true, ADD, false>(upd, a.batch, s);
        else if (a.W)
            last_product<UPDATE>(upd, a.batch, pl.tall, rows4, s);
        else
            last_product<ORTH>(upd, a.batch, pl.tall, rows4, s);
        std::swap(x, y);
    }
    return hipGetLastError();
}

} // namespace lb
