// A 16-bit MFMA product tile for gfx950, shared by the loss-head and Muon kernels:
//
//     C[i,j] = Σ_r A(i,r)·B(j,r)        bf16 or fp16 operands, fp32 accumulation
//
// One block of four waves owns a TI x TJ tile of C and hands its fp32 sums to an
// epilogue.  Each operand is stored in memory in one of two ways:
//
//   RC  reduction contiguous: A(i,r) = a[i*lda + r]
//   OC  outer contiguous:     A(i,r) = a[r*lda + i]
//
// so that X·W, G·Wᵀ, Xᵀ·G, X·Xᵀ, Xᵀ·X and B·X all run without a transposed copy.
//
// Pipeline.  The reduction runs in pairs of 32-deep slabs (64 reduction indices).
// An operand's pair is T x 64 elements in LDS, T*128 bytes, filled by global->LDS
// DMA (buffer_load_dwordx4 ... lds) through a ring of S pair slots per operand:
//
//   RC  T rows of 128 B (whole cache lines); 16-byte chunk c of row o sits at
//       chunk c ^ (o % 8); a 16x16x32 fragment is one ds_read_b128.
//   OC  64 rows (r) of 2T bytes; chunk c of row r sits at c ^ swz_oc(r); a fragment is two
//       transposing reads (ds_read_b64_tr_b16), each a 4-row x 16-column block per 16 lanes.
//
// Both patterns read without bank conflicts (the layouts of the Linear backward's
// tile kernel).  While the MFMAs of one slab run on fragments in registers, the
// next slab's fragments are read; in a pair's second slab every fragment of the
// pair is in registers, so after one barrier its slot takes the DMA of the pair S
// ahead.  One barrier per 64 reduction indices.  Pairs past the reduction's end are
// issued too, through an empty buffer descriptor (they read zero), so the loop has
// no tail: only one wait count and one branch.
//
// Bound.  256x256 (8x8 fragments per wave, 256 LDS bytes per MFMA): MFMA and the power
// limit; 1.36-1.42 PFLOP/s over whole calls, matrix pipes 66-73% busy at 1.7-1.9 GHz.  B has
// three slots there, A two (160 KiB of LDS): B's DMA, issued after A's, gets a pair more to
// land (Muon's A at 4096 x 4096 over 12288: 272 -> 256 us).  128x128 (512 LDS bytes per MFMA):
// LDS, 1536 cycles of reads and DMA for 1024 of MFMA with two blocks on a CU; it fills the
// card where there are few tiles.  64x64 and the 32- and 64-row tiles: latency (0.25 us a
// pair) or HBM.
#pragma once

#include "device.h"

#include <type_traits>

namespace lb {
namespace tile {

#define LB_LDS __attribute__((address_space(3)))

constexpr uint32_t kOutOfRange = 0x80000000u; // buffer offset past every descriptor used here
constexpr int kThreads = 256;                 // four waves

// Two stored 16-bit types, told apart at compile time.
struct BF16 {
    static __device__ __forceinline__ uint32_t pack2(float a, float b) { return pack_bf16x2(a, b); }
    static __device__ __forceinline__ uint16_t one(float a) { return f32_to_bf16_bits(a); }
    static __device__ __forceinline__ float f32(uint32_t h) { return bf16_bits_to_f32(h & 0xffffu); }
    static __device__ __forceinline__ void mfma(f32x4_t &acc, const u32x4_t &a, const u32x4_t &b) {
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    }
};
struct F16 {
    static __device__ __forceinline__ uint16_t one(float a) {
        return __builtin_bit_cast(uint16_t, (_Float16)a); // nearest even; overflow to infinity
    }
    static __device__ __forceinline__ uint32_t pack2(float a, float b) {
        return (uint32_t)one(a) | ((uint32_t)one(b) << 16);
    }
    static __device__ __forceinline__ float f32(uint32_t h) { return f16_bits_to_f32((uint16_t)(h & 0xffffu)); }
    static __device__ __forceinline__ void mfma(f32x4_t &acc, const u32x4_t &a, const u32x4_t &b) {
        asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    }
};

// Four waves as WI x WJ, each FI x FJ fragments of 16 x 16; S pair slots for A, SB for B.
// BANY: B's rows may start at any element (2-byte alignment): they come through registers.
template <class T_, int WI_, int WJ_, int FI_, int FJ_, bool AOC_, bool BOC_, int S_, int SB_ = S_, bool BANY_ = false>
struct Cfg {
    using T = T_;
    static constexpr int WI = WI_, WJ = WJ_, FI = FI_, FJ = FJ_, S = S_, SB = SB_;
    static constexpr bool AOC = AOC_, BOC = BOC_, BANY = BANY_;
    static constexpr int TI = WI * FI * 16, TJ = WJ * FJ * 16;
    static constexpr int kPairA = TI * 128, kPairB = TJ * 128; // bytes of an operand's pair
    static constexpr int kOffB = S * kPairA;                   // A's slots first, then B's
    static constexpr int kLds = S * kPairA + SB * kPairB;
    static constexpr int kDmaA = TI / 32, kDmaB = TJ / 32; // DMA instructions per wave per pair
    static constexpr int kDma = kDmaA + kDmaB;
    static_assert(WI * WJ == 4, "four waves");
    static_assert(TI % 32 == 0 && TJ % 32 == 0, "whole DMA instructions per wave");
    static_assert(!AOC || TI == 64 || TI == 128 || TI == 256, "OC rows of 128, 256 or 512 bytes");
    static_assert(!BOC || TJ == 64 || TJ == 128 || TJ == 256, "OC rows of 128, 256 or 512 bytes");
    static_assert(4 * FJ * 1024 <= kLds, "the epilogue stages 16 rows per wave in the ring");
    // memory instructions that may be in flight while A's next pair (and B's, if it is
    // DMA'd too) has landed; a chunk of B that comes through registers is two loads
    static constexpr int kAhead =
        BANY ? (S - 2) * (kDmaA + 2 * kDmaB) + 2 * kDmaB : (S - 2) * kDma + (SB - S) * kDmaB;
    static_assert(SB >= S && kAhead + kDma < 64, "vmcnt is 6 bits");
    using With = Cfg<T_, WI_, WJ_, FI_, FJ_, AOC_, BOC_, S_, SB_, true>; // the same, B at any alignment
};

// One product.  lda, ldb multiples of 8 elements, a and b 16-byte aligned.  Operands are
// fetched in 16-byte chunks along their contiguous index: where that extent (RC: R, OC: I
// or J) is no multiple of 8, the rest of the last chunk is memory of the operand's own,
// and zero (or only reaches sums that the epilogue drops).  2*256*ld < 2^31 for RC
// operands and 2*64*ld < 2^31 for OC ones, checked on the host.  With BANY, b and ldb are
// free; what follows a row's end in its last chunk is then the next row (the columns of C
// it reaches are dropped, or A is zero there).
struct Job {
    const uint16_t *a, *b;
    int64_t lda, ldb;
    int64_t I, J, R;
    int tiles_i, tiles_j;
    int group; // tile rows per raster group
};

typedef uint32_t frag_half_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t rs, LB_LDS char *dst, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LB_LDS void *)dst, 16, (int)off, 0, 0, 0);
}
template <int N>
__device__ __forceinline__ void vm_wait() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Publishes landed DMA and retires this wave's LDS reads; no fence, so DMA stays in flight.
__device__ __forceinline__ void ring_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// XOR on an OC row's chunk index: the rows r..r+3 and r+8..r+11 of one 32-lane read land on
// eight different 32-byte segments of the 256 bytes of banks (rows of 128 bytes alternate
// between two halves by themselves, so four segments are left to choose).
template <int T>
__device__ __forceinline__ int swz_oc(int row) {
    if constexpr (T >= 128)
        return 2 * ((row & 3) | (((row >> 3) & 1) << 2));
    else
        return 2 * (((row >> 1) & 1) | (((row >> 3) & 1) << 1));
}

// Blocks are dealt to the 8 XCDs in turn: block t of n -> its place when each XCD's blocks
// are gathered into one contiguous range (any n), so that tiles that run together on an
// XCD are neighbours and share operand panels in its L2.
__device__ __forceinline__ int gathered(int t, int n) {
    const int x = t & 7, rem = n & 7;
    return x * (n >> 3) + (x < rem ? x : rem) + (t >> 3);
}
// place -> tile, rastered in groups of `group` tile rows
__device__ __forceinline__ void coords(const Job &jb, int u, int &ti, int &tj) {
    const int per = jb.group * jb.tiles_j;
    const int g = u / per;
    const int first = g * jb.group;
    const int rows = min(jb.tiles_i - first, jb.group);
    u -= g * per;
    ti = first + u % rows;
    tj = u / rows;
}
// The same for a symmetric product: the tiles on and below the diagonal only (tj <= ti),
// row by row.
__device__ __forceinline__ void coords_lower(int u, int &ti, int &tj) {
    ti = (int)((__builtin_sqrtf(8.0f * (float)u + 1.0f) - 1.0f) * 0.5f);
    while (ti * (ti + 1) / 2 > u)
        --ti;
    while ((ti + 1) * (ti + 2) / 2 <= u)
        ++ti;
    ti = __builtin_amdgcn_readfirstlane(ti);
    tj = u - ti * (ti + 1) / 2;
}

// One operand of a tile: T outer indices from o0 on.
template <int T, bool OC, int kDmaN, int S>
struct Side {
    static constexpr int kPair = T * 128;
    static constexpr int kRowB = 2 * T; // OC row bytes
    uint32_t off[kDmaN];                // DMA source offsets, fixed for the tile
    const uint16_t *cur;                // first element of the next pair to fetch
    int64_t step;                       // elements from one pair to the next
    int64_t left;                       // reduction indices from `cur` on (may be <= 0)
    int64_t ld, span;                   // RC: rows; OC: columns of the window
    int kchunk;                         // RC: this lane's first r within a pair

    __device__ __forceinline__ void init(const uint16_t *p, int64_t ld_, int64_t O, int64_t R, int64_t o0, int w,
                                         int lane) {
        ld = ld_;
        if constexpr (OC) {
            left = R;
            constexpr int kChunks = T / 8;       // 16-byte chunks per row
            constexpr int kRows = 64 / kChunks;  // rows per DMA instruction
            cur = p + o0;
            step = 64 * ld;
            span = (O - o0 + 7) / 8 * 8; // whole chunks
            kchunk = 0;
#pragma unroll
            for (int d = 0; d < kDmaN; ++d) {
                const int row = (w * kDmaN + d) * kRows + lane / kChunks;
                const int c = (lane % kChunks) ^ swz_oc<T>(row);
                off[d] = (uint32_t)((row * ld + 8 * c) * 2) | ((uint32_t)!(8 * c < span) << 31);
            }
        } else {
            left = (R + 7) / 8 * 8; // whole chunks
            cur = p + o0 * ld;
            step = 64;
            span = min<int64_t>(T, O - o0);
            kchunk = 8 * ((lane & 7) ^ (lane >> 3)); // row % 8 is lane / 8 in every instruction
#pragma unroll
            for (int d = 0; d < kDmaN; ++d) {
                const int row = (w * kDmaN + d) * 8 + (lane >> 3);
                off[d] = (uint32_t)((row * ld + kchunk) * 2) | ((uint32_t)!(row < span) << 31);
            }
        }
    }
    struct Src {
        __amdgpu_buffer_rsrc_t rs;
        uint32_t mask; // RC: bit 31 for lanes past the reduction's end
    };
    // the descriptor of the next pair; advances
    __device__ __forceinline__ Src next() {
        Src s;
        if constexpr (OC) {
            const int64_t rows = min<int64_t>(64, left);
            s.rs = rsrc(cur, left > 0 ? (uint32_t)(((rows - 1) * ld + span) * 2) : 0u);
            s.mask = 0;
        } else {
            s.rs = rsrc(cur, left > 0 ? (uint32_t)(((span - 1) * ld + left) * 2) : 0u);
            s.mask = (uint32_t)(kchunk >= left) << 31;
        }
        cur += step;
        left -= 64;
        return s;
    }
    __device__ __forceinline__ void dma(const Src &s, LB_LDS char *slot, int w, int d) const {
        dma16(s.rs, slot + (w * kDmaN + d) * 1024, off[d] | s.mask);
    }
};

// The same for rows at any alignment of 2 bytes.  A 16-byte chunk is fetched as the aligned
// dwords that hold it, four and one more, shifted together (a row's chunks all by 0 or by
// 16 bits) and written to the ring by ds_write.  The stage holds the pair after those in
// the ring, so a load has a pair's time to land.  No load passes the dword that holds the
// matrix' last element.
template <int T, bool OC, int kDmaN>
struct AnySide {
    uint32_t off[kDmaN], dst[kDmaN];
    u32x4_t v[kDmaN];  // stage
    uint32_t e[kDmaN]; // the fifth dwords
    uint32_t shift;
    const uint16_t *cur; // aligned down to a dword
    int64_t step, left, ld, span;
    int half, kchunk; // elements that aligning skipped back; RC: this lane's first r

    __device__ __forceinline__ void init(const uint16_t *p, int64_t ld_, int64_t O, int64_t R, int64_t o0, int w,
                                         int lane) {
        ld = ld_;
        left = R;
        const uint16_t *first = OC ? p + o0 : p + o0 * ld;
        half = (int)((reinterpret_cast<uintptr_t>(first) >> 1) & 1);
        cur = first - half;
        constexpr int kChunks = OC ? T / 8 : 8, kRows = 64 / kChunks; // per instruction
        const int c = lane % kChunks;
        kchunk = OC ? 0 : 8 * c;
        step = OC ? 64 * ld : 64; // whole dwords: the shifts stay
        span = OC ? O - o0 : min<int64_t>(T, O - o0);
        shift = (uint32_t)((half + (lane / kChunks) * ld) & 1) * 16; // kRows is even
#pragma unroll
        for (int d = 0; d < kDmaN; ++d) {
            const int row = (w * kDmaN + d) * kRows + lane / kChunks;
            const bool in = OC ? 8 * c < span : row < span;
            off[d] = ((uint32_t)((half + row * ld + 8 * c) * 2) & ~3u) | ((uint32_t)!in << 31);
            dst[d] = (uint32_t)(row * (16 * kChunks) + ((c ^ (OC ? swz_oc<T>(row) : row & 7)) << 4));
        }
    }
    struct Src {
        __amdgpu_buffer_rsrc_t rs;
        uint32_t mask;
    };
    __device__ __forceinline__ Src next() {
        Src s;
        const int64_t rows = OC ? min<int64_t>(64, left) : span;
        const int64_t last = OC ? span : left; // elements of the last row
        s.rs = rsrc(cur, left > 0 ? (uint32_t)((half + (rows - 1) * ld + last) * 2 + 3) & ~3u : 0u);
        s.mask = OC ? 0u : (uint32_t)(kchunk >= left) << 31;
        cur += step;
        left -= 64;
        return s;
    }
    __device__ __forceinline__ void load(const Src &s, int d) {
        const int o = (int)(off[d] | s.mask);
        v[d] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(s.rs, o, 0, 0));
        e[d] = __builtin_amdgcn_raw_buffer_load_b32(s.rs, o + 16, 0, 0);
    }
    __device__ __forceinline__ void write(LB_LDS char *slot, int d) const {
        u32x4_t x;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x[k] = __builtin_amdgcn_alignbit(k == 3 ? e[d] : v[d][k + 1], v[d][k], shift);
        asm volatile("ds_write_b128 %0, %1" ::"v"(slot + dst[d]), "v"(x) : "memory");
    }
};

// LDS fragment addresses of one operand for a wave, and the reads.  Inline asm: the
// compiler would wait for the DMA in flight (it may alias) before every read.  Callers
// wait with settle(), which also keeps every output in use until the data has landed.
template <int T, bool OC, int F, int S>
struct Frags {
    static constexpr int kPair = T * 128;
    static constexpr int kReads = OC ? 2 * F : F;
    LB_LDS char *base[OC ? F : 2];

    __device__ __forceinline__ void init(LB_LDS char *region, int ob, int lane) {
        if constexpr (OC) {
            const int g = lane >> 4, s = lane & 15;
            const int row = 8 * g + (s >> 2);
#pragma unroll
            for (int x = 0; x < F; ++x) {
                const int col = ob + 16 * x + 4 * (s & 3);
                base[x] = region + row * (2 * T) + (((col >> 3) ^ swz_oc<T>(row)) << 4) + (col & 7) * 2;
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                base[h] = region + (ob + (lane & 15)) * 128 + (((4 * h + (lane >> 4)) ^ (lane & 7)) << 4);
        }
    }
    // read number k (0..kReads-1) of slab half H; the slot is a compile-time constant
    // where its offset fits the instruction's 16 bits (two slots), else SLOT is 0 and `add` holds it
    template <int SLOT, int H>
    __device__ __forceinline__ void read(int k, int add, u32x4_t (&f)[F], frag_half_t (&h)[F][2]) const {
        if constexpr (OC) {
            const int x = k >> 1;
            if (k & 1)
                read_tr<SLOT * kPair + H * 64 * T + 8 * T>(base[x] + add, h[x][1]);
            else
                read_tr<SLOT * kPair + H * 64 * T>(base[x] + add, h[x][0]);
        } else {
            read_rc<SLOT * kPair, F>(base[H] + add, k, f);
        }
    }
    template <int OFF>
    static __device__ __forceinline__ void read_tr(const LB_LDS char *p, frag_half_t &v) {
        static_assert(OFF >= 0 && OFF < 65536, "ds offset is 16 bits");
        asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(v) : "v"(p), "n"(OFF));
    }
    template <int OFF, int N>
    static __device__ __forceinline__ void read_rc(const LB_LDS char *p, int x, u32x4_t (&f)[N]) {
        static_assert(OFF + 2048 * (N - 1) < 65536, "ds offset is 16 bits");
        switch (x) { // x is a constant after unrolling
        case 0: asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(f[0]) : "v"(p), "n"(OFF)); break;
#define LB_RC(X)                                                                                                     \
    case X:                                                                                                          \
        if constexpr (X < N)                                                                                         \
            asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(f[X < N ? X : 0]) : "v"(p), "n"(OFF + 2048 * X));    \
        break;
            LB_RC(1) LB_RC(2) LB_RC(3) LB_RC(4) LB_RC(5) LB_RC(6) LB_RC(7)
#undef LB_RC
        }
    }
    // after the wait: the reads' outputs exist from here on
    static __device__ __forceinline__ void settle(u32x4_t (&f)[F], frag_half_t (&h)[F][2]) {
        if constexpr (OC) {
#pragma unroll
            for (int x = 0; x < F; ++x) {
                asm volatile("" : "+v"(h[x][0]), "+v"(h[x][1]));
                f[x] = __builtin_shufflevector(h[x][0], h[x][1], 0, 1, 2, 3);
            }
        } else {
#pragma unroll
            for (int x = 0; x < F; ++x)
                asm volatile("" : "+v"(f[x]));
        }
    }
};

// Wait states between the last MFMA and another instruction that reads its accumulator.
__device__ __forceinline__ void mfma_drain() { asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory"); }

template <class C>
using Acc = f32x4_t[C::FI][C::FJ];

// Keeps a row of accumulators in its AGPRs up to this point (the compiler otherwise
// copies all of them to VGPRs before an epilogue's first branch, and spills).
template <int N>
__device__ __forceinline__ void pin(f32x4_t (&a)[N]) {
#pragma unroll
    for (int y = 0; y < N; ++y)
        asm volatile("" : "+a"(a[y]));
}

// The sums of tile (ti, tj): acc[x][y] of lane l of wave w holds C[i][j..j+3] for
// i = i0 + (w / WJ)*FI*16 + 16x + l % 16, j = j0 + (w % WJ)*FJ*16 + 16y + 4*(l / 16).
// On return the ring is free (a barrier has passed) and may stage the epilogue.
template <class C>
__device__ __forceinline__ void accumulate(const Job &jb, int ti, int tj, LB_LDS char *smem, Acc<C> &acc) {
    using SA = Side<C::TI, C::AOC, C::kDmaA, C::S>;
    using SB = std::conditional_t<C::BANY, AnySide<C::TJ, C::BOC, C::kDmaB>, Side<C::TJ, C::BOC, C::kDmaB, C::SB>>;
    using FA = Frags<C::TI, C::AOC, C::FI, C::S>;
    using FB = Frags<C::TJ, C::BOC, C::FJ, C::SB>;
    constexpr int FI = C::FI, FJ = C::FJ, NM = FI * FJ;
    constexpr int NR = FA::kReads + FB::kReads;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    SA sa;
    SB sb;
    sa.init(jb.a, jb.lda, jb.I, jb.R, (int64_t)ti * C::TI, w, lane);
    sb.init(jb.b, jb.ldb, jb.J, jb.R, (int64_t)tj * C::TJ, w, lane);
    FA fa;
    FB fb;
    fa.init(smem, (w / C::WJ) * FI * 16, lane);
    fb.init(smem + C::kOffB, (w % C::WJ) * FJ * 16, lane);
#pragma unroll
    for (int x = 0; x < FI; ++x)
#pragma unroll
        for (int y = 0; y < FJ; ++y)
            acc[x][y] = f32x4_t{};

    const int npair = (int)((jb.R + 63) / 64);
    u32x4_t a0[FI], b0[FJ], a1[FI], b1[FJ];
    frag_half_t ha[FI][2], hb[FJ][2];

    // DMA instruction d of a pair: A's, then B's (which may have a slot more, and time)
    auto issue = [&](const typename SA::Src &xa, const typename SB::Src &xb, int slot_a, int slot_b, int d) {
        if (d < C::kDmaA) {
            sa.dma(xa, smem + slot_a * C::kPairA, w, d);
        } else if constexpr (C::BANY) { // the staged pair to its slot, the one after it to the stage
            sb.write(smem + C::kOffB + slot_b * C::kPairB, d - C::kDmaA);
            sb.load(xb, d - C::kDmaA);
        } else {
            sb.dma(xb, smem + C::kOffB + slot_b * C::kPairB, w, d - C::kDmaA);
        }
    };
    auto settle = [&](u32x4_t (&af)[FI], u32x4_t (&bf)[FJ]) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        FA::settle(af, ha);
        FB::settle(bf, hb);
        __builtin_amdgcn_sched_barrier(0);
    };
    // MFMAs of one slab on (af, bf), the LDS reads of slab half H of the pair in slot
    // SLOT (+ adds) into (an, bn) after the first of them, `other(i)` after each
    auto slab = [&](auto slot_c, auto slotb_c, auto half_c, int add_a, int add_b, u32x4_t (&af)[FI], u32x4_t (&bf)[FJ],
                    u32x4_t (&an)[FI], u32x4_t (&bn)[FJ], auto other) {
        constexpr int SLOT = decltype(slot_c)::value, SLOTB = decltype(slotb_c)::value;
        constexpr int H = decltype(half_c)::value;
        constexpr int kPer = (NR + NM - 1) / NM;                             // reads per MFMA
        constexpr int kEvery = NR <= NM ? (NM / 2 / NR > 0 ? NM / 2 / NR : 1) : 1; // MFMAs per read
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            C::T::mfma(acc[i / FJ][i % FJ], bf[i % FJ], af[i / FJ]);
            __builtin_amdgcn_sched_barrier(0);
            if (i % kEvery == 0) {
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    const int k = i / kEvery * kPer + e;
                    if (k < FA::kReads)
                        fa.template read<SLOT, H>(k, add_a, an, ha);
                    else if (k < NR)
                        fb.template read<SLOTB, H>(k - FA::kReads, add_b, bn, hb);
                }
            }
            other(i);
            __builtin_amdgcn_sched_barrier(0);
        }
        settle(an, bn);
    };
    using Z = std::integral_constant<int, 0>;
    using O = std::integral_constant<int, 1>;

    // prologue: every slot on its way; the first slab's fragments
    typename SA::Src xa;
    typename SB::Src xb;
    if constexpr (C::BANY) {
        xb = sb.next();
#pragma unroll
        for (int d = 0; d < C::kDmaB; ++d)
            sb.load(xb, d);
    }
#pragma unroll
    for (int s = 0; s < C::SB; ++s) {
        if (s < C::S)
            xa = sa.next();
        xb = sb.next();
#pragma unroll
        for (int d = s < C::S ? 0 : C::kDmaA; d < C::kDma; ++d)
            issue(xa, xb, s, s, d);
    }
    vm_wait<C::BANY ? 2 * C::kDmaB : C::kAhead + C::kDma>();
    ring_barrier();
#pragma unroll
    for (int k = 0; k < FA::kReads; ++k)
        fa.template read<0, 0>(k, 0, a0, ha);
#pragma unroll
    for (int k = 0; k < FB::kReads; ++k)
        fb.template read<0, 0>(k, 0, b0, hb);
    settle(a0, b0);

    // One pair.  A slot is a compile-time constant (PAR, of two) or `ia`; so is B's where
    // both have two, else `ib`.
    constexpr bool fixa = C::S == 2, fixb = C::S == 2 && C::SB == 2;
    int ia = 0, ib = 0; // the pair's slots where they are not constants
    auto pair = [&](auto par, auto next) {
        using PB = std::integral_constant<int, fixb ? decltype(par)::value : 0>;
        using NB = std::integral_constant<int, fixb ? decltype(next)::value : 0>;
        const int ja = ia + 1 == C::S ? 0 : ia + 1, jb = ib + 1 == C::SB ? 0 : ib + 1;
        // first half; the descriptors of the pairs to fetch are made between its MFMAs
        slab(par, PB{}, O{}, fixa ? 0 : ia * C::kPairA, fixb ? 0 : ib * C::kPairB, a0, b0, a1, b1, [&](int i) {
            if (i == NM - 2) {
                xa = sa.next();
                xb = sb.next();
            }
        });
        vm_wait<C::kAhead>(); // the next pair has landed
        ring_barrier();       // everyone's; and this pair's slots are free
        slab(next, NB{}, Z{}, fixa ? 0 : ja * C::kPairA, fixb ? 0 : jb * C::kPairB, a1, b1, a0, b0, [&](int i) {
#pragma unroll
            for (int d = i * C::kDma / NM; d < (i + 1) * C::kDma / NM; ++d)
                issue(xa, xb, fixa ? decltype(par)::value : ia, fixb ? decltype(par)::value : ib, d);
        });
        ia = ja;
        ib = jb;
    };
    if constexpr (fixa) {
        // an odd count runs one pair of zeros more: with an exit between the two the
        // compiler copied the accumulators out of the AGPRs on every turn
        for (int q = 0; q < npair; q += 2) {
            pair(Z{}, O{});
            pair(O{}, Z{});
        }
    } else {
        for (int q = 0; q < npair; ++q)
            pair(Z{}, Z{});
    }
    mfma_drain();
    vm_wait<0>();
    ring_barrier();
}

// The same for a reduction of at most 64 indices: one pair, one slot per operand, nothing
// to pipeline.  The small ring lets three blocks share a CU, whose loads and stores then
// cover each other's latency.
template <class C>
__device__ __forceinline__ void accumulate_once(const Job &jb, int ti, int tj, LB_LDS char *smem, Acc<C> &acc) {
    static_assert(C::S == 1 && C::SB == 1 && !C::BANY, "one pair");
    using FA = Frags<C::TI, C::AOC, C::FI, 1>;
    using FB = Frags<C::TJ, C::BOC, C::FJ, 1>;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Side<C::TI, C::AOC, C::kDmaA, 1> sa;
    Side<C::TJ, C::BOC, C::kDmaB, 1> sb;
    sa.init(jb.a, jb.lda, jb.I, jb.R, (int64_t)ti * C::TI, w, lane);
    sb.init(jb.b, jb.ldb, jb.J, jb.R, (int64_t)tj * C::TJ, w, lane);
    const auto xa = sa.next();
    const auto xb = sb.next();
#pragma unroll
    for (int d = 0; d < C::kDmaA; ++d)
        sa.dma(xa, smem, w, d);
#pragma unroll
    for (int d = 0; d < C::kDmaB; ++d)
        sb.dma(xb, smem + C::kOffB, w, d);
    FA fa;
    FB fb;
    fa.init(smem, (w / C::WJ) * C::FI * 16, lane);
    fb.init(smem + C::kOffB, (w % C::WJ) * C::FJ * 16, lane);
#pragma unroll
    for (int x = 0; x < C::FI; ++x)
#pragma unroll
        for (int y = 0; y < C::FJ; ++y)
            acc[x][y] = f32x4_t{};
    vm_wait<0>();
    ring_barrier();
    auto half = [&](auto h) {
        constexpr int H = decltype(h)::value;
        u32x4_t a[C::FI], b[C::FJ];
        frag_half_t ha[C::FI][2], hb[C::FJ][2];
#pragma unroll
        for (int k = 0; k < FA::kReads; ++k)
            fa.template read<0, H>(k, 0, a, ha);
#pragma unroll
        for (int k = 0; k < FB::kReads; ++k)
            fb.template read<0, H>(k, 0, b, hb);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        FA::settle(a, ha);
        FB::settle(b, hb);
#pragma unroll
        for (int x = 0; x < C::FI; ++x)
#pragma unroll
            for (int y = 0; y < C::FJ; ++y)
                C::T::mfma(acc[x][y], b[y], a[x]);
    };
    half(std::integral_constant<int, 0>{});
    half(std::integral_constant<int, 1>{}); // zeros where R <= 32
    mfma_drain();
    ring_barrier();
}

// Passes a wave's sums through its own part of the ring, 16 rows at a time, so that a
// lane holds 4 consecutive columns and 4*FJ lanes a row's FJ*16 columns (direct from the
// accumulators a store instruction would touch 16 rows).  round(x, i, rows, j, v): v[q] is
// C[i + q*rows][j..j+3], q < FJ; begin(x, i, rows, j) comes before the round's LDS traffic
// (to load what a later round combines with).
template <class C, class Begin, class Fn>
__device__ __forceinline__ void staged(Acc<C> &acc, int64_t i0, int64_t j0, LB_LDS char *smem, Begin begin,
                                       Fn round) {
    constexpr int FJ = C::FJ, kChunks = 4 * FJ, kRows = 64 / kChunks;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    LB_LDS char *const reg = smem + w * (FJ * 1024);
    const int64_t ib = i0 + (w / C::WJ) * C::FI * 16, jb = j0 + (w % C::WJ) * FJ * 16;
#pragma unroll
    for (int x = 0; x < C::FI; ++x) {
        asm volatile("" ::: "memory"); // loads of later rounds stay behind this one's stores
        begin(x, ib + 16 * x + lane / kChunks, kRows, jb + 4 * (lane % kChunks));
        pin(acc[x]);
#pragma unroll
        for (int y = 0; y < FJ; ++y) {
            const int r = lane & 15, c = 4 * y + (lane >> 4);
            *reinterpret_cast<LB_LDS f32x4_t *>(reg + r * (FJ * 64) + ((c ^ (r & (kChunks - 1))) << 4)) = acc[x][y];
        }
        f32x4_t v[FJ];
#pragma unroll
        for (int q = 0; q < FJ; ++q) {
            const int r = q * kRows + lane / kChunks, c = lane % kChunks;
            v[q] = *reinterpret_cast<const LB_LDS f32x4_t *>(reg + r * (FJ * 64) + ((c ^ (r & (kChunks - 1))) << 4));
        }
        __builtin_amdgcn_sched_barrier(0); // all reads before the first use
        round(x, ib + 16 * x + lane / kChunks, kRows, jb + 4 * (lane % kChunks), v);
    }
}

// 16-bit output through LDS: 32 rows of a wave at a time, whole 16-byte chunks per lane.
// begin(h) is called before round h, value(x, y) gives the 4 packed values of acc[x][y].
// vec: rows of dst 16-byte aligned and J a multiple of 8; stores then go through a
// descriptor of the round's rows, which drops the rows past I without a branch (with a
// check per store each became a branch of its own).
// nt: non-temporal stores, for data not read again soon in rows of whole 128-byte lines.
// (Where rows start inside a line the caches have to put two waves' parts together: dW for
// M = 15, K = 1792, V = 109976 took 285 us with non-temporal stores, 163 at V = 110080.)
template <class C, class Begin, class Fn>
__device__ __forceinline__ void store16(Acc<C> &acc, uint16_t *dst, int64_t ld, int64_t I, int64_t J, int64_t ib,
                                        int64_t jb, bool vec, bool nt, LB_LDS char *smem, Begin begin, Fn value) {
    constexpr int FJ = C::FJ, kRowB = FJ * 32, kChunks = 2 * FJ, kRows = 64 / kChunks;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    LB_LDS char *const reg = smem + w * (FJ * 1024);
    const uint32_t off = (uint32_t)((lane / kChunks) * ld + 8 * (lane % kChunks)) * 2 |
                         ((uint32_t)!(jb + 8 * (lane % kChunks) < J) << 31);
    const uint32_t step = (uint32_t)(kRows * ld * 2);
#pragma unroll
    for (int h = 0; h < C::FI / 2; ++h) {
        asm volatile("" ::: "memory"); // loads of later rounds stay behind this one's stores
        begin(h);
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
            const int64_t rows = max<int64_t>(0, min<int64_t>(32, I - i0));
            const __amdgpu_buffer_rsrc_t rs = rsrc(dst + i0 * ld + jb, (uint32_t)(rows * ld * 2));
            if (nt) {
#pragma unroll
                for (int q = 0; q < FJ; ++q)
                    __builtin_amdgcn_raw_buffer_store_b128(v[q], rs, (int)(off + q * step), 0, 2);
            } else {
#pragma unroll
                for (int q = 0; q < FJ; ++q)
                    __builtin_amdgcn_raw_buffer_store_b128(v[q], rs, (int)(off + q * step), 0, 0);
            }
        } else {
            // rows of any alignment: 64 lanes store 64 neighbouring elements of a row (two
            // rows of 32), eight stores at a time
            constexpr int kCols = FJ * 16, kSegs = kCols >= 64 ? kCols / 64 : 1, kPer = kCols >= 64 ? 1 : 64 / kCols;
            const int64_t rows = max<int64_t>(0, min<int64_t>(32, I - i0));
            const __amdgpu_buffer_rsrc_t rs =
                rsrc(dst + i0 * ld + jb, rows && jb < J ? (uint32_t)(((rows - 1) * ld + J - jb) * 2) : 0u);
            const int lr = lane / kCols, lc = lane % kCols; // lr = 0 for whole rows
#pragma unroll
            for (int q0 = 0; q0 < 32 * kSegs / kPer; q0 += 8) {
                uint16_t v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int r = (q0 + u) / kSegs * kPer + lr, c = (q0 + u) % kSegs * 64 + lc;
                    v[u] = *reinterpret_cast<const LB_LDS uint16_t *>(
                        reg + r * kRowB + (((c >> 3) ^ (r & (kChunks - 1))) << 4) + (c & 7) * 2);
                }
                __builtin_amdgcn_sched_barrier(0); // all reads before the first store
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int r = (q0 + u) / kSegs * kPer, c = (q0 + u) % kSegs * 64;
                    const uint32_t o = (uint32_t)(lr * ld + lc + c) * 2 + (uint32_t)(r * ld * 2);
                    __builtin_amdgcn_raw_buffer_store_b16(
                        v[u], rs, (int)(o | ((uint32_t)!(jb + c + lc < J) << 31)), 0, 0);
                }
            }
        }
    }
}

} // namespace tile
} // namespace lb
