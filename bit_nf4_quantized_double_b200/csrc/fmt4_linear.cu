// Product of a few tokens with a weight kept in one of the group-scaled 4-bit formats of
// fmt4.cu (page "QLoRA: put the large model in memory, then change it with a small adapter",
// wq-win.github.io/llm/074-qlora, section 4, evidence 1 names the formats):
//   Y[m, n] = (1 / S) sum_b absmax[n, b] sum_{k in block b} v(code[n, k]) X[m, k].
//
// The codes and block constants, 0.5625 bytes per weight, are read once; they bound the
// kernel while the tokens are few. What would bound it next is turning codes into matrix
// operands: the integer pipe takes a warp instruction every two cycles, and at HBM speed 64
// weights per lane have to pass in about 180 cycles of a scheduler.
//
// Weights become fp16 pairs, exactly. E2M1: the conversion instruction of that type, one per
// two codes. E3M0: a code is a six-bit float s eee 00 in bits 5..2 of a byte, whose conversion
// takes two codes as well (seven integer instructions for eight codes with the masks). Int4:
// sign to bit 15, magnitude to bits 8..10, which fp16 reads as m 2^-16 (any bits below 2^11
// are an integer times 2^-24; nine instructions for eight codes). Left shifts are
// multiplications by powers of two that the compiler does not know, which run on the other
// integer pipe. Bits further down would need fewer shifts, but the sum inside mma aligns its
// terms by their exponent fields, so that a small subnormal costs the others low bits
// (measured 2e-6 instead of 1e-7 of the result).
//
// Tokens become fp16 after scaling by 2^-e, set per token and 256 inputs so that the largest
// lies in [2^14, 2^15): exact for every bf16 within 2^-31 of the largest of its 256
// neighbours, off by at most 2^-39 of that largest below.
//
// mma.sync m16n8k16 adds the exact products in fp32; each 64-block's sum is then scaled by
// its constant in fp32, and Y is rounded once at the end. (An fp8 mma.sync needs fewer
// instructions to place the codes, but on this part it runs as two fp16 mma with conversions
// before them: 48 us where a [28672, 8192] weight's bytes take 20.)
//
// Layout. A warp keeps the token operands of one slice of 256 inputs in registers and runs
// down the rows in steps of 16, which it copies into its own ring of stages (stream4.cuh).
// The 16 warps of a CTA hold 16 slices, a cluster of CTAs the whole row; a tile of 16 rows is
// summed over the warps, then over the CTAs, in a fixed order.
#include <algorithm>
#include <atomic>

#include "launch.h"
#include "stream4.cuh"

namespace qnf4 {

using namespace tc;

namespace {

constexpr int kF4Warps = 16;
constexpr int kF4Threads = 32 * kF4Warps;
constexpr int kF4Stages = 4;
constexpr int kF4StageBytes = s4::kCodeBytes + s4::kStepRows * 16;   // codes, four fp32 constants per row
constexpr int kF4Tokens = 16;                                          // tokens per pass over the codes
constexpr int kF4MaxCluster = 8;
constexpr int kF4SegBytes = 16384;                                     // tile sums kept for the cluster's sum

// Shared memory: 256 rows of 256 bytes whose first halves hold the lookup table (a word per
// lane) and whose second halves ("holes", 32 floats each) the warps' sums; the rings; a barrier;
// the tile sums of a cluster's segment.
constexpr int kF4TableBytes = 65536;
constexpr int kF4RingBytes = kF4Warps * kF4Stages * kF4StageBytes;
constexpr int kF4BarBytes = 32;
constexpr int f4_smem(bool cluster) { return kF4TableBytes + kF4RingBytes + kF4BarBytes + (cluster ? kF4SegBytes : 0); }
static_assert(f4_smem(true) <= 232448, "shared memory");

// A round is f4_round(nt) steps of every warp. Its sums go to one of two buffers and are added
// over the warps after the first step of the next round, when the others have mostly written
// theirs. A warp's sums of a tile are a piece of 128 nt floats, [token][row], permuted so that
// the 32 lanes of a store (eight rows of four tokens 2 t, or of four tokens 2 t + 1) touch
// every bank once.
__host__ __device__ constexpr int f4_round(int nt) { return nt == 1 ? 2 : 1; }
__host__ __device__ constexpr int f4_seg_tiles(int nt) { return kF4SegBytes / (128 * nt * 4); }
__device__ __forceinline__ int f4_sum_at(int m, int r) { return ((m ^ ((m >> 2) & 1)) << 4) + (r ^ ((m & 2) << 2)); }
// Byte offset of float x of piece p (both buffers' pieces count up to 64 / nt).
template <int NT>
__device__ __forceinline__ uint32_t f4_hole(int p, int x) {
    return (uint32_t)(p * NT * 4 + (x >> 5)) * 256u + 128u + (uint32_t)(x & 31) * 4u;
}

struct F4Args {
    const __nv_bfloat16 *X;
    const uint8_t *codes;
    const float *absmax;
    void *Y;
    int64_t M, N;
    int K, kbs, nsl;           // inputs, 64-blocks and 256-input slices per row
    int wk;                    // warps along a row in a CTA; the CTA's 16 / wk tiles lie side by side
    int nch, passes;           // CTAs along a row (cluster size); passes over the rows per segment
    int y_f32, vec_scales;
    uint32_t two2, two4, two8, two12;   // 2^2, 2^4, 2^8, 2^12
    float factor;              // (power of two of the decoded weights) / S
};

// Codes of a word as four fp16 pairs; pair_code names the codes of pair p (low half, high half).
// Words 1 of Int4 and E3M0 come from the table, pair by byte: (0,1) (2,3) (4,5) (6,7).
template <int FMT>
__host__ __device__ constexpr bool from_table(int word) { return FMT != QLORA_FMT4_FP4_E2M1 && word == 1; }
template <int FMT>
__host__ __device__ constexpr int pair_code(int word, int p, int half) {
    return from_table<FMT>(word)          ? 2 * p + half
           : FMT == QLORA_FMT4_INT4       ? (p < 2 ? 1 - p : 5 - p) + 4 * half     // (1,5) (0,4) (3,7) (2,6)
           : FMT == QLORA_FMT4_FP4_E2M1   ? 2 * p + 1 - half                        // (1,0) (3,2) (5,4) (7,6)
                                          : (p < 2 ? 1 + 4 * p : 4 * (p - 2)) + 2 * half;   // (1,3) (5,7) (0,2) (4,6)
}
// A code's fp16 operand, for the table.
template <int FMT>
__device__ __forceinline__ uint32_t code_f16(uint32_t n) {
    const uint32_t m = n & 7u, sign = (n & 8u) << 12;
    if (FMT == QLORA_FMT4_INT4) return (m << 8) | sign;
    return (m ? (m + 12u) << 10 : 0u) | sign;
}
__device__ __forceinline__ uint32_t f16x2_of_e3m2(uint16_t v) {
    uint32_t d;
    asm("cvt.rn.f16x2.e3m2x2 %0, %1;" : "=r"(d) : "h"(v));
    return d;
}
template <int FMT>
__device__ __forceinline__ void decode(const F4Args &a, const uint8_t *table, uint32_t lane4, int word, uint32_t w,
                                       uint32_t (&p)[4]) {
    if (from_table<FMT>(word)) {
        // address = byte * 256 + lane * 4, by one permute
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = *reinterpret_cast<const uint32_t *>(table + prmt(w, lane4, 0x5504u | ((uint32_t)i << 4)));
    } else if (FMT == QLORA_FMT4_INT4) {
        const uint32_t w4 = w * a.two4, w8 = w * a.two8, w12 = w * a.two12;
        p[0] = (w8 & 0x07000700u) | (w12 & 0x80008000u);
        p[1] = (w4 & 0x07000700u) | (w8 & 0x80008000u);
        p[2] = (w & 0x07000700u) | (w4 & 0x80008000u);
        p[3] = ((w >> 4) & 0x07000700u) | (w & 0x80008000u);
    } else if (FMT == QLORA_FMT4_FP4_E2M1) {
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3]) : "r"(w));
    } else {
        const uint32_t lo = (w * a.two2) & 0x3c3c3c3cu, hi = (w >> 2) & 0x3c3c3c3cu;
        p[0] = f16x2_of_e3m2((uint16_t)lo);
        p[1] = f16x2_of_e3m2((uint16_t)(lo >> 16));
        p[2] = f16x2_of_e3m2((uint16_t)hi);
        p[3] = f16x2_of_e3m2((uint16_t)(hi >> 16));
    }
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Token operands of one slice (256 inputs from k0) for up to eight tokens from X: lane (g, t)
// holds token g, inputs 64 b + 16 t + 8 j + 0..7 in xb[8 b + 4 j + p], in the order of the
// decoded pairs. Lane u converts inputs 8 u .. 8 u + 7 of every token, which are one such
// group, and hands them over in shared memory (stage(m, u)).
// up0, up1: 2^e of the tokens of accumulator columns 2 t and 2 t + 1.
template <int FMT, typename Stage>
__device__ __forceinline__ void f4_tokens(const __nv_bfloat16 *X, int mn, int K, int k0, int lane, Stage stage,
                                          uint32_t (&xb)[32], float &up0, float &up1) {
    const int g = lane >> 2, t = lane & 3;
    const bool in = k0 + 8 * lane < K;
    uint4 v[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        v[m] = make_uint4(0u, 0u, 0u, 0u);
        if (m < mn && in) v[m] = __ldg(reinterpret_cast<const uint4 *>(X + (int64_t)m * K + k0) + lane);
    }
    up0 = up1 = 0.0f;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        if (m < mn) {
            const uint32_t w[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
            // |x| of the largest, as bf16 bits
            uint32_t big = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                    __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
            big = __reduce_max_sync(0xffffffffu, max(big & 0xffffu, big >> 16));
            // 2^e from the exponent field of the largest; both powers kept normal
            const int ex = min(max((int)(big >> 7), 24), 254);          // 254 also for NaN and infinity
            const float down = __uint_as_float((uint32_t)(268 - ex) << 23), up = __uint_as_float((uint32_t)(ex - 14) << 23);
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = bf16_lo(w[i]) * down;
                f[2 * i + 1] = bf16_hi(w[i]) * down;
            }
            uint32_t o[4];                                 // this lane's inputs are word lane % 2 of a block
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                constexpr bool same = !from_table<FMT>(1);
                const float l0 = f[pair_code<FMT>(0, p, 0)], h0 = f[pair_code<FMT>(0, p, 1)];
                const float l1 = f[pair_code<FMT>(1, p, 0)], h1 = f[pair_code<FMT>(1, p, 1)];
                o[p] = same ? f16x2_of(l0, h0) : f16x2_of((lane & 1) ? l1 : l0, (lane & 1) ? h1 : h0);
            }
            *stage(m & 3, lane) = make_uint4(o[0], o[1], o[2], o[3]);
            up0 = 2 * t == m ? up : up0;
            up1 = 2 * t + 1 == m ? up : up1;
        }
        if ((m & 3) == 3) {                            // four tokens are staged: their lanes take them
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint4 o = make_uint4(0u, 0u, 0u, 0u);
                if (g < mn) o = *stage(g & 3, 8 * (i >> 1) + 2 * t + (i & 1));
                if ((g >> 2) == (m >> 2)) {
                    xb[4 * i] = o.x;
                    xb[4 * i + 1] = o.y;
                    xb[4 * i + 2] = o.z;
                    xb[4 * i + 3] = o.w;
                }
            }
            __syncwarp();
        }
    }
}

// Copies of one step: 16 rows from `codes` and `absmax` (the tile's first row, this lane's
// offsets added), of which `rows` are the weight's; a lane past the last input copies zeros.
struct F4Lane {
    uint32_t dst, code_off, scale_off;   // stage offset of the lane's first chunk; global byte offsets
    int row0;                            // first row of the warp's tile in the CTA's group
    int bytes;                           // 16, or 0 for a chunk past the end of the row
};
__device__ __forceinline__ void f4_issue(const F4Args &a, uint32_t stage, const uint8_t *codes, const float *absmax,
                                         int rows, const F4Lane &l, int s, int lane) {
    const uint32_t rb = (uint32_t)a.K / 2;
    const uint8_t *scales = reinterpret_cast<const uint8_t *>(absmax);
    const uint32_t dst = stage + l.dst;                // rows r + 4 i swizzle alike
    const uint32_t sc = stage + s4::kCodeBytes;
    if (rows >= s4::kStepRows && a.vec_scales) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s4::cp16n(dst + 512 * i, codes + (l.code_off + 4 * i * rb), l.bytes);
        if (lane < 16) s4::cp16n(sc + lane * 16, scales + l.scale_off, 16);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool ok = (lane >> 3) + 4 * i < rows;
        s4::cp16n(dst + 512 * i, ok ? codes + (l.code_off + 4 * i * rb) : a.codes, ok ? l.bytes : 0);
    }
    if (a.vec_scales) {
        const bool ok = lane < rows;
        if (lane < 16) s4::cp16n(sc + lane * 16, ok ? scales + l.scale_off : (const uint8_t *)a.absmax, ok ? 16 : 0);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int q = 8 * i + (lane >> 2), b = 4 * s + (lane & 3);
            const bool ok = q < rows && b < a.kbs;
            s4::cp4n(sc + q * 16 + (lane & 3) * 4, ok ? absmax + (int64_t)(l.row0 + q) * a.kbs + b : a.absmax, ok ? 4 : 0);
        }
    }
}

__device__ __forceinline__ void f4_store(const F4Args &a, int64_t m, int64_t row, float y) {
    y *= a.factor;
    if (a.y_f32) static_cast<float *>(a.Y)[m * a.N + row] = y;
    else static_cast<__nv_bfloat16 *>(a.Y)[m * a.N + row] = __float2bfloat16_rn(y);
}

template <int FMT, int NT, bool CLUSTER>
__global__ void __launch_bounds__(kF4Threads, 1) k_fmt4_linear(const __grid_constant__ F4Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int R = f4_round(NT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_addr(smem) + kF4TableBytes + warp * (kF4Stages * kF4StageBytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kF4TableBytes + kF4RingBytes);   // a round's sums are written; flag
    volatile int *abort = reinterpret_cast<int *>(bars + 1);
    float *seg = reinterpret_cast<float *>(smem + kF4TableBytes + kF4RingBytes + kF4BarBytes);
    const uint32_t bar = smem_addr(bars);
    if (threadIdx.x == 0) {
        mbar_init(bar, kF4Warps);
        *abort = 0;
        fence_barrier_init();
    }
    const int wk = CLUSTER ? kF4Warps : a.wk, tg = kF4Warps / wk;
    const int kw = CLUSTER ? warp : warp % wk, tw = CLUSTER ? 0 : warp / wk;
    const int nch = CLUSTER ? a.nch : 1, passes = CLUSTER ? a.passes : 1;
    const int rank = CLUSTER ? (int)cluster_ctarank() : 0;
    const int ncl = gridDim.x / nch, cl = blockIdx.x / nch;
    const int groups = (int)((a.N + s4::kStepRows * tg - 1) / (s4::kStepRows * tg));
    const int mine = (groups - cl + ncl - 1) / ncl;        // tile groups cl, cl + ncl, ...
    const int64_t m0 = (int64_t)blockIdx.y * kF4Tokens;
    const int mn = (int)min((int64_t)kF4Tokens, a.M - m0);
    // the row's slices, spread evenly over passes x CTAs: this CTA has slices lo .. lo + n - 1 of a pass
    const int parts = passes * nch, sq = a.nsl / parts, srem = a.nsl % parts;
    auto slice_of = [&](int pass) {                         // this warp's slice in a pass, -1 for none
        const int p = pass * nch + rank, n = sq + (p < srem ? 1 : 0);
        return kw < n ? p * sq + min(p, srem) + kw : -1;
    };
    const int seg_len = CLUSTER ? f4_seg_tiles(NT) : mine;

    // the copies run ahead of the products over round, pass and segment borders
    const uint32_t rb = (uint32_t)a.K / 2, sb = (uint32_t)a.kbs * 4;
    const int row_step = ncl * tg * s4::kStepRows;
    F4Lane ln;
    ln.dst = s4::code_off(lane >> 3, lane & 7);
    ln.row0 = tw * s4::kStepRows;
    int is0 = 0, ii = 0, ip = 0, ps = 0, isl = slice_of(0); // issue position: segment, tile in it, pass
    int64_t irow = (int64_t)cl * tg * s4::kStepRows;        // first row of the CTA's tile group
    auto set_lane = [&]() {
        const bool in = isl >= 0 && isl * s4::kStepK + 32 * (lane & 7) < a.K;
        ln.code_off = (ln.row0 + (lane >> 3)) * rb + (in ? (uint32_t)(isl * 128 + (lane & 7) * 16) : 0u);
        ln.scale_off = (ln.row0 + lane) * sb + (uint32_t)max(isl, 0) * 16;
        ln.bytes = in ? 16 : 0;
    };
    set_lane();
    auto issue = [&]() {
        if (isl >= 0 && ii < min(seg_len, mine - is0)) {
            f4_issue(a, ring + ps * kF4StageBytes, a.codes + irow * rb, a.absmax + irow * a.kbs,
                     (int)min(a.N - irow, (int64_t)256) - ln.row0, ln, isl, lane);
            irow += row_step;
            ++ii;
        }
        s4::cp_commit();
        ps = ps + 1 == kF4Stages ? 0 : ps + 1;
        while (CLUSTER && is0 < mine && (isl < 0 || ii == min(seg_len, mine - is0))) {   // next pass or segment
            if (++ip == passes) {
                ip = 0;
                is0 += seg_len;
            }
            ii = 0;
            isl = slice_of(ip);
            irow = ((int64_t)cl + (int64_t)is0 * ncl) * s4::kStepRows;
            set_lane();
        }
    };
#pragma unroll
    for (int i = 0; i < kF4Stages - 1; ++i) issue();

    if (from_table<FMT>(1)) {
        for (int i = threadIdx.x; i < 256 * 8; i += kF4Threads) {
            const uint32_t v = code_f16<FMT>(i >> 7) | (code_f16<FMT>((i >> 3) & 15) << 16);
            *reinterpret_cast<uint4 *>(smem + (i >> 3) * 256 + (i & 7) * 16) = make_uint4(v, v, v, v);
        }
    }
    __syncthreads();
    uint32_t at[4];                                         // this lane's codes of block b in a stage
#pragma unroll
    for (int b = 0; b < 4; ++b) at[b] = ring + g * 128 + t * 8 + ((b ^ (g & 3)) << 5);
    const uint32_t sc_a = ring + s4::kCodeBytes + g * 16;
    // pieces of a round: [tiles side by side][tile of the round][warp along the row]
    const int piece0 = tw * R * wk + kw;                    // this warp's, plus wk per tile of the round
    constexpr int kBufPieces = kF4Warps * R;
    uint8_t *put[4];                                        // this lane's places in piece 0: tokens 2 t, 2 t + 1, rows g, g + 8
#pragma unroll
    for (int i = 0; i < 4; ++i) put[i] = smem + f4_hole<NT>(0, f4_sum_at(2 * t + (i & 1), g + 8 * (i >> 1)));
    // Adds a finished round over the warps, in warp order: tiles i0 .. i0 + rn - 1 of segment s0, written as
    // round number `round`. The warps take turns at the start of the element range.
    auto add_round = [&](int round, int i0, int rn, bool first) {
        if (!mbar_wait(bar, round & 1, abort)) return;
        // element 16 m + r of tile ti; the warps take turns at the start of the range
        for (int e = ((warp + 5 * round) & (kF4Warps - 1)) * 32 + lane; e < tg * R * 128 * NT; e += kF4Threads) {
            const int ti = e / (128 * NT), o = e & (128 * NT - 1), m = o >> 4, r = o & 15;
            const int i = ti & (R - 1);                     // ti = (tile side by side) * R + (tile of the round)
            if (i >= rn || m >= mn) continue;
            const uint8_t *src = smem + f4_hole<NT>((round & 1) * kBufPieces + ti * wk, f4_sum_at(m, r));
            float y = 0.0f;
#pragma unroll 16
            for (int w = 0; w < wk; ++w) y += *reinterpret_cast<const float *>(src + w * (NT * 1024));
            if (CLUSTER) {
                float *dst = seg + (i0 + i) * (128 * NT) + o;
                *dst = first ? y : *dst + y;
            } else {
                const int64_t row = (int64_t)(cl + (i0 + i) * ncl) * (tg * s4::kStepRows) + (ti / R) * s4::kStepRows + r;
                if (row < a.N) f4_store(a, m0 + m, row, y);
            }
        }
    };
    int cs = 0, round = 0;
    for (int s0 = 0; s0 < mine; s0 += seg_len) {
        const int n = min(seg_len, mine - s0);
        for (int pass = 0; pass < passes; ++pass) {
            const int sl = slice_of(pass);
            uint32_t xb[NT][32];
            float up[NT][2];
            if (sl >= 0) {
                // handed over in the places of this warp's own sums: 512 bytes for each of four tokens
                auto stage = [&](int m, int u) {
                    const int p = (m >> 1) * kBufPieces + (NT == 1 ? (m & 1) * wk : 0);
                    return reinterpret_cast<uint4 *>(smem + f4_hole<NT>(p + piece0, 4 * u + (NT == 1 ? 0 : (m & 1) * 128)));
                };
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    f4_tokens<FMT>(a.X + (m0 + 8 * nt) * a.K, mn - 8 * nt, a.K, sl * s4::kStepK, lane, stage, xb[nt],
                                   up[nt][0], up[nt][1]);
            }
            for (int i0 = 0; i0 < n; i0 += R, ++round) {
                const int rn = min(R, n - i0);
                for (int i = 0; i < rn; ++i) {
                    const uint32_t po = ((round & 1) * kBufPieces + piece0 + i * wk) * (NT * 1024);
                    if (sl < 0) {
                        if (i == 0 && i0 > 0) add_round(round - 1, i0 - R, R, pass == 0);
                        for (int e = lane; e < 128 * NT; e += 32) *reinterpret_cast<float *>(smem + po + f4_hole<NT>(0, e)) = 0.0f;
                        continue;
                    }
                    float acc[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
                    s4::cp_wait<kF4Stages - 2>();
                    __syncwarp();
                    issue();
                    const uint32_t so = cs * kF4StageBytes;
                    cs = cs + 1 == kF4Stages ? 0 : cs + 1;
                    const float4 f0 = s4::lds128f(sc_a + so), f1 = s4::lds128f(sc_a + so + 128);
                    const float c0[4] = {f0.x, f0.y, f0.z, f0.w}, c1[4] = {f1.x, f1.y, f1.z, f1.w};
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint2 u = s4::lds64(at[b] + so), v = s4::lds64(at[b] + so + 8 * 128);
                        float c[NT][4];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t p[4], q[4];
                            decode<FMT>(a, smem, lane * 4, j, j ? u.y : u.x, p);
                            decode<FMT>(a, smem, lane * 4, j, j ? v.y : v.x, q);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint32_t *x = xb[nt] + 8 * b + 4 * j;
                                if (j == 0) mma_f16_first(c[nt], p[0], q[0], p[1], q[1], x[0], x[1]);
                                else mma_f16(c[nt], p[0], q[0], p[1], q[1], x[0], x[1]);
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint32_t *x = xb[nt] + 8 * b + 4 * j;
                                mma_f16(c[nt], p[2], q[2], p[3], q[3], x[2], x[3]);
                            }
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            acc[nt][0] = fmaf(c0[b], c[nt][0], acc[nt][0]);
                            acc[nt][1] = fmaf(c0[b], c[nt][1], acc[nt][1]);
                            acc[nt][2] = fmaf(c1[b], c[nt][2], acc[nt][2]);
                            acc[nt][3] = fmaf(c1[b], c[nt][3], acc[nt][3]);
                        }
                    }
                    // the round before, whose buffer the next round needs: a step after it ended
                    if (i == 0 && i0 > 0) add_round(round - 1, i0 - R, R, pass == 0);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (8 * nt + 2 * t + (e & 1) < mn)
                                *reinterpret_cast<float *>(put[e] + po + nt * 1024) = acc[nt][e] * up[nt][e & 1];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
            }
            if (n > 0) {
                const int last = (n - 1) / R * R;
                add_round(round - 1, last, n - last, pass == 0);
            }
            if (CLUSTER) __syncthreads();              // the buffers are free for the next pass's hand-over
        }
        if (CLUSTER) {
            // the CTAs' sums in rank order; the CTAs take turns over the segment's elements
            cluster_sync();
            const uint32_t base = smem_addr(seg);
            for (int e = rank * kF4Threads + threadIdx.x; e < n * 16 * mn; e += nch * kF4Threads) {
                const int i = e / (16 * mn), o = e - i * 16 * mn;
                float y = 0.0f;
                for (int c = 0; c < nch; ++c) y += ld_cluster_f32(map_to_rank(base + 4 * (i * (128 * NT) + o), c));
                const int64_t row = (int64_t)(cl + (s0 + i) * ncl) * s4::kStepRows + (o & 15);
                if (row < a.N) f4_store(a, m0 + (o >> 4), row, y);
            }
            cluster_sync();                            // before the next segment's sums, or the exit
        }
    }
    s4::cp_wait<0>();
}

template <int FMT, int NT>
cudaError_t f4_launch(const F4Args &a, int64_t groups, cudaStream_t st) {
    const bool cluster = a.nch > 1 || a.passes > 1;
    auto kernel = cluster ? k_fmt4_linear<FMT, NT, true> : k_fmt4_linear<FMT, NT, false>;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)a.nch;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.blockDim = dim3(kF4Threads);
    cfg.dynamicSmemBytes = f4_smem(cluster);
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = cluster ? 1 : 0;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return e;
    // clusters that run at once: fewer than SMs / size where the chip's SM groups do not divide
    int most = num_sms();
    if (cluster) {
        static std::atomic<int> active[kF4MaxCluster + 1];
        most = active[a.nch].load(std::memory_order_relaxed);
        if (most == 0) {
            cfg.gridDim = dim3((unsigned)a.nch);
            if ((e = cudaOccupancyMaxActiveClusters(&most, kernel, &cfg)) != cudaSuccess) return e;
            if (most < 1) most = 1;
            active[a.nch].store(most, std::memory_order_relaxed);
        }
    }
    cfg.gridDim = dim3((unsigned)(std::min<int64_t>(groups, most) * a.nch), (unsigned)ceil_div(a.M, (int64_t)kF4Tokens));
    QNF4_LAUNCH("k_fmt4_linear", st, e = cudaLaunchKernelEx(&cfg, kernel, a));
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int FMT>
cudaError_t f4_launch_tiles(const F4Args &a, int64_t groups, cudaStream_t st) {
    const int64_t m = a.M < kF4Tokens ? a.M : kF4Tokens;
    return m <= 8 ? f4_launch<FMT, 1>(a, groups, st) : f4_launch<FMT, 2>(a, groups, st);
}

}  // namespace

cudaError_t launch_fmt4_linear(const __nv_bfloat16 *X, int64_t M, const uint8_t *codes, const float *absmax, int64_t rows,
                               int64_t cols, qlora_fmt4 f, void *Y, bool y_f32, cudaStream_t st) {
    F4Args a;
    a.X = X;
    a.codes = codes;
    a.absmax = absmax;
    a.Y = Y;
    a.M = M;
    a.N = rows;
    a.K = (int)cols;
    a.kbs = (int)(cols / kBlock1);
    a.nsl = (int)ceil_div(cols, s4::kStepK);
    a.y_f32 = y_f32;
    a.two2 = 4;
    a.two4 = 16;
    a.two8 = 256;
    a.two12 = 4096;
    a.vec_scales = a.kbs % 4 == 0 && aligned16(absmax);
    // Int4 operands are m 2^-16; an E3M0 code e is read as 2^(e - 3), its value is 2^(e - 7)
    a.factor = f == QLORA_FMT4_INT4 ? 65536.0f / 7.0f : f == QLORA_FMT4_FP4_E2M1 ? 1.0f / 6.0f : 0.0625f;
    const int sms = num_sms();
    // CTAs along a row: enough for a slice per warp, more while there are fewer tiles than SMs
    const int64_t tiles = ceil_div(rows, (int64_t)s4::kStepRows);
    int64_t nch = ceil_div(a.nsl, kF4Warps);
    while (nch < kF4MaxCluster && tiles * (nch + 1) <= sms && a.nsl >= 4 * (nch + 1)) ++nch;
    if (nch > kF4MaxCluster) nch = kF4MaxCluster;
    a.nch = (int)nch;
    a.passes = (int)ceil_div(a.nsl, nch * kF4Warps);
    a.wk = kF4Warps;
    if (nch == 1)
        while (a.wk > 1 && a.wk / 2 >= a.nsl) a.wk /= 2;
    const int64_t groups = ceil_div(rows, (int64_t)s4::kStepRows * (kF4Warps / a.wk));
    switch (f) {
        case QLORA_FMT4_INT4: return f4_launch_tiles<QLORA_FMT4_INT4>(a, groups, st);
        case QLORA_FMT4_FP4_E2M1: return f4_launch_tiles<QLORA_FMT4_FP4_E2M1>(a, groups, st);
        default: return f4_launch_tiles<QLORA_FMT4_FP4_E3M0>(a, groups, st);
    }
}

}  // namespace qnf4
