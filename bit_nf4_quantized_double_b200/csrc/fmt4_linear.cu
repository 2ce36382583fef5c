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
// (measured 2e-6 instead of 1e-7 of the result). For up to eight tokens Int4 takes a byte from a
// table instead, a word per lane: one permute, which is the address, and one load per two codes
// (32.1 us for [28672, 8192], without a table 35.8; with rows of 128 bytes, whose addresses take
// a multiplication more, 33.7, and half of the codes by those 33.9).
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
// Layout. A warp keeps the token operands of one slice of 256 inputs in registers, converted
// once, and runs down the rows in steps of 16 through its own ring, which its lane 0 fills by
// TMA, two neighbouring steps by a copy (one by one it took 2 us more of the figures below). The
// 16 warps of a CTA hold 16 slices, a cluster of CTAs the whole row; tiles of 16 rows are summed
// over the warps every second step, over the CTAs at the end, in a fixed order. (Tokens in shared
// memory and a whole row per warp need no sums, but a warp per tile is 12 warps per SM at
// [28672, 8192], too few to hide the latencies of the products.)
//
// Measured, one token, [28672, 8192], 132 MB: 26.8 / 31.9 / 32.1 us for E2M1 / E3M0 / Int4 (75 /
// 63 / 63 % of the measured copy rate; [114688, 8192], E2M1: 89 %); 4.4 us for the smallest
// weight, which is launch, first latencies and one sum. E2M1 with 8 tokens 28.4 us, with 9 to 16
// tokens 43 to 44: two operand sets of 32 registers at a limit of 128 (all but one of these forms
// spill 12 to 112 bytes), twice the matrix instructions. Every 16 tokens read the codes again, one
// group after the other: more tokens than a decode step has are not what this plan is for.
#include <algorithm>

#include "launch.h"
#include "tc.cuh"
#include "tmap.h"

namespace qnf4 {

using namespace tc;

namespace {

constexpr int kF4Warps = 16;
constexpr int kF4Threads = 32 * kF4Warps;
constexpr int kF4Stages = 4;
constexpr int kF4StepK = 256;                                          // a step: 16 rows x 256 inputs,
constexpr int kF4StepRows = 16;                                        // 128 bytes of codes per row
constexpr int kF4StageBytes = kF4StepRows * 128;
constexpr int kF4ScaleBytes = kF4StepRows * 16;                        // four block constants per row
constexpr int kF4Tokens = 16;                                          // tokens per pass over the codes
constexpr int kF4MaxCluster = 8;
constexpr int kF4Round = 2;                                            // steps between sums over the warps
static_assert(kF4Stages == 2 * kF4Round, "a round's stages are refilled while the other two are used");

// Shared memory: the warps' rings of codes and of constants, two buffers of the warps' sums of a
// round, the rings' barriers, the round's barrier and the abort flag, a cluster's tile sums.
constexpr int kF4ScaleAt = kF4Warps * kF4Stages * kF4StageBytes;
constexpr int kF4SumAt = kF4ScaleAt + kF4Warps * kF4Stages * kF4ScaleBytes;
__host__ __device__ constexpr int f4_piece(int nt) { return 16 * 8 * nt * 4; }          // a warp's sums of a tile
__host__ __device__ constexpr int f4_buf_bytes(int nt) { return kF4Round * kF4Warps * f4_piece(nt); }
// With a lookup table (a word per byte of codes and lane) its 256 rows are 256 bytes apart, so that a permute of a byte
// and the lane makes an address; the other halves of the rows hold the sums.
__host__ __device__ constexpr int f4_bar_at(int nt, bool table) { return kF4SumAt + (table ? 65536 : 2 * f4_buf_bytes(nt)); }
__host__ __device__ constexpr int f4_seg_at(int nt, bool table) { return f4_bar_at(nt, table) + kF4Warps * 16 + 32; }
__host__ __device__ constexpr int f4_seg_tiles(int nt) { return 32 / nt; }
constexpr int f4_smem(int nt, bool cluster, bool table) {
    return 1024 + f4_seg_at(nt, table) + (cluster ? f4_seg_tiles(nt) * f4_piece(nt) : 0);
}
static_assert(2 * f4_buf_bytes(1) <= 256 * 128, "the sums between the table's rows");
constexpr int kF4Reserved = 1024;                                      // the window's first bytes, which the system keeps
static_assert(f4_smem(1, true, true) <= 232448 && f4_smem(2, true, false) <= 232448, "shared memory");

// A warp's sums of a tile are [token][row], permuted so that the 32 lanes of a store (eight even
// or odd rows of tokens 2 t, or of tokens 2 t + 1) touch every bank once.
__device__ __forceinline__ int f4_sum_at(int m, int r) {
    return ((m ^ ((m >> 2) & 1)) << 4) + ((r >> 1) | (((r & 1) << 3) ^ ((m & 2) << 2)));
}

struct F4Args {
    // bytes [rows, K / 2], boxes of a round and of a step, 128-byte swizzle; fp32 [rows, K / 64] likewise (vec_scales)
    CUtensorMap codes, codes_step, scales, scales_step;
    const __nv_bfloat16 *X;
    const float *absmax;
    void *Y;
    int64_t M, N;
    int K, kbs, nsl;           // inputs, 64-blocks and 256-input slices per row
    int wk;                    // warps along a row in a CTA; the CTA's 16 / wk tiles lie side by side
    int nch, passes;           // CTAs along a row (cluster size); passes over a segment's rows
    int y_f32, vec_scales;
    uint32_t two2, two4, two8, two12;   // 2^2, 2^4, 2^8, 2^12
};

// A decoded operand times 2^operand_scale times sum_factor is v(code) / S, the factor in [1, 2): Int4 operands are m 2^-16
// (m / 8 from the table), an E3M0 code e is read as 2^(e - 3), its value is 2^(e - 7). The power of two goes into the
// tokens' 2^e, so that all sums hold Y / factor: neither do they overflow where Y does not, nor do they lose more than a
// bit as subnormals where Y is none. (All of it applied at the end made the sums 16 Y for E3M0.)
__host__ __device__ constexpr int operand_scale(int fmt, bool table) {
    return fmt == QLORA_FMT4_INT4 ? (table ? 0 : 13) : fmt == QLORA_FMT4_FP4_E2M1 ? -3 : -4;
}
__host__ __device__ constexpr float sum_factor(int fmt) {
    return fmt == QLORA_FMT4_INT4 ? 8.0f / 7.0f : fmt == QLORA_FMT4_FP4_E2M1 ? 8.0f / 6.0f : 1.0f;
}

// Codes of a word as four fp16 pairs; pair_code names the codes of pair p (low half, high half).
template <int FMT>
__host__ __device__ constexpr int pair_code(int p, int half) {
    return FMT == QLORA_FMT4_INT4       ? (p < 2 ? 1 - p : 5 - p) + 4 * half     // (1,5) (0,4) (3,7) (2,6)
           : FMT == QLORA_FMT4_FP4_E2M1 ? 2 * p + 1 - half                        // (1,0) (3,2) (5,4) (7,6)
                                        : (p < 2 ? 1 + 4 * p : 4 * (p - 2)) + 2 * half;   // (1,3) (5,7) (0,2) (4,6)
}
__device__ __forceinline__ uint32_t f16x2_of_e3m2(uint16_t v) {
    uint32_t d;
    asm("cvt.rn.f16x2.e3m2x2 %0, %1;" : "=r"(d) : "h"(v));
    return d;
}
template <int FMT>
__device__ __forceinline__ void decode(const F4Args &a, uint32_t w, uint32_t (&p)[4]) {
    if (FMT == QLORA_FMT4_INT4) {
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

// Codes of a word by the table. at: the lane's word of row 0, without the constant kF4Reserved + kF4SumAt; its upper half
// holds the CTA's place in its cluster, its second byte is zero. Pairs as E2M1's: (1, 0) (3, 2) (5, 4) (7, 6). No one writes
// the table after it was filled: the loads may move freely.
__device__ __forceinline__ void decode_table(uint32_t w, uint32_t at, uint32_t (&p)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("ld.shared.u32 %0, [%1 + %2];"
            : "=r"(p[i]) : "r"(prmt(w, at, 0x7604u | ((uint32_t)i << 4))), "n"(kF4Reserved + kF4SumAt));
}
// A code's value as the table holds it (Int4), in eighths.
__device__ __forceinline__ float table_value(int c) { return (c & 8 ? -0.125f : 0.125f) * (float)(c & 7); }

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
// group, and hands them over in shared memory (stage(m, u): 512 bytes for each of four tokens).
// up0, up1: 2^(e + SCALE) of the tokens of accumulator columns 2 t and 2 t + 1.
template <int FMT, int SCALE, typename Stage>
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
    for (int i = 0; i < 32; ++i) xb[i] = 0u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (4 * h >= mn) break;
#pragma unroll
        for (int mm = 0; mm < 4; ++mm) {
            const int m = 4 * h + mm;
            if (m >= mn) break;
            const uint32_t w[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
            // |x| of the largest, as bf16 bits
            uint32_t big = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                    __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
            big = __reduce_max_sync(0xffffffffu, max(big & 0xffffu, big >> 16));
            // 2^e from the exponent field of the largest; all powers kept normal
            const int ex = min(max((int)(big >> 7), 24), 254);          // 254 also for NaN and infinity
            const float down = __uint_as_float((uint32_t)(268 - ex) << 23), up = __uint_as_float((uint32_t)(ex - 14 + SCALE) << 23);
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = bf16_lo(w[i]) * down;
                f[2 * i + 1] = bf16_hi(w[i]) * down;
            }
            uint32_t o[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) o[p] = f16x2_of(f[pair_code<FMT>(p, 0)], f[pair_code<FMT>(p, 1)]);
            *stage(mm, lane) = make_uint4(o[0], o[1], o[2], o[3]);
            up0 = 2 * t == m ? up : up0;
            up1 = 2 * t + 1 == m ? up : up1;
        }
        __syncwarp();
        if ((g >> 2) == h && g < mn) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 o = *stage(g & 3, 8 * (i >> 1) + 2 * t + (i & 1));
                xb[4 * i] = o.x;
                xb[4 * i + 1] = o.y;
                xb[4 * i + 2] = o.z;
                xb[4 * i + 3] = o.w;
            }
        }
        __syncwarp();                                  // before the next tokens' hand-over
    }
}

// Asynchronous copy of 4 bytes, or of none: zeros.
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, bool valid) {
    const int n = valid ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Block constants of one step where a row's do not start on 16 bytes: rows row0 .., blocks 4 s ..
// (zeros past the last row and block), block lane % 4 of rows lane / 4 and + 8.
__device__ __forceinline__ void f4_scales(const F4Args &a, uint32_t dst, int64_t row0, int s, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int q = 8 * i + (lane >> 2), b = 4 * s + (lane & 3);
        const bool ok = row0 + q < a.N && b < a.kbs;
        cp4(dst + q * 16 + (lane & 3) * 4, ok ? a.absmax + (row0 + q) * a.kbs + b : a.absmax, ok);
    }
}

// Before an early exit: waits, within a limit, for the copies of rounds `used` .. `filled` - 1.
__device__ __noinline__ void f4_drain(uint32_t full, uint32_t used, uint32_t filled) {
    cp_wait<0>();
    const uint64_t t0 = global_timer_ns();
    for (; used != filled; ++used)
        while (!mbar_try_wait(full + 8 * (used & 1u), (used >> 1) & 1u))
            if (global_timer_ns() - t0 > kWaitLimitNs) return;
}

template <int FMT>
__device__ __forceinline__ void f4_store(const F4Args &a, int64_t m, int64_t row, float y) {
    y *= sum_factor(FMT);
    if (a.y_f32) static_cast<float *>(a.Y)[m * a.N + row] = y;
    else static_cast<__nv_bfloat16 *>(a.Y)[m * a.N + row] = __float2bfloat16_rn(y);
}

template <int FMT, int NT, bool CLUSTER, bool VEC, bool TABLE>
__global__ void __launch_bounds__(kF4Threads, 1) k_fmt4_linear(const __grid_constant__ F4Args a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    constexpr int R = kF4Round, SPREAD = TABLE ? 2 : 1, PIECE = SPREAD * f4_piece(NT), BUF = SPREAD * f4_buf_bytes(NT);
    // offset of byte o of a warp's sums
    auto spread = [](int o) { return TABLE ? 2 * (o & ~127) + 128 + (o & 127) : o; };
    uint8_t *smem = align1024(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_addr(smem) + warp * (kF4Stages * kF4StageBytes);
    const uint32_t cring = smem_addr(smem) + kF4ScaleAt + warp * (kF4Stages * kF4ScaleBytes);
    const uint32_t full = smem_addr(smem) + f4_bar_at(NT, TABLE) + warp * 16;               // the ring's two rounds
    const uint32_t bar = smem_addr(smem) + f4_bar_at(NT, TABLE) + kF4Warps * 16;   // a round's sums are written
    volatile int *abort = reinterpret_cast<int *>(smem + f4_bar_at(NT, TABLE) + kF4Warps * 16 + 8);
    float *seg = reinterpret_cast<float *>(smem + f4_seg_at(NT, TABLE));
    // the table's address is made of constants: the window's start below the cluster place has to be the expected one
    if (TABLE && (smem_addr(smem) & 0xffffffu) != (uint32_t)kF4Reserved) {
        if (threadIdx.x == 0) raise_status(QLORA_ERR_CUDA);
        griddep_wait();                                // the kernel before ends before this one
        return;
    }
    if (lane < 2) mbar_init(full + 8 * lane, 1);
    if (threadIdx.x == 0) {
        mbar_init(bar, kF4Warps);
        *abort = 0;
    }
    fence_barrier_init();
    if (lane == 0) {
        tma_prefetch_desc(&a.codes);
        if (VEC) tma_prefetch_desc(&a.scales);
    }
    const uint32_t table = smem_addr(smem) - kF4Reserved + lane * 4;
    if (TABLE)
        for (int i = threadIdx.x; i < 256 * 8; i += kF4Threads) {
            const uint32_t v = f16x2_of(table_value((i >> 3) & 15), table_value(i >> 7));
            *reinterpret_cast<uint4 *>(smem + kF4SumAt + (i >> 3) * 256 + (i & 7) * 16) = make_uint4(v, v, v, v);
        }
    __syncthreads();
    // A kernel behind this one may be set up while this one runs; both touch global memory only after
    // the kernel before them has ended.
    griddep_launch_dependents();
    griddep_wait();

    const int wk = CLUSTER ? kF4Warps : a.wk, tg = kF4Warps / wk;
    const int kw = CLUSTER ? warp : warp % wk, tw = CLUSTER ? 0 : warp / wk;
    const int nch = CLUSTER ? a.nch : 1, passes = CLUSTER ? a.passes : 1;
    const int rank = CLUSTER ? (int)cluster_ctarank() : 0;
    const int ncl = gridDim.x / nch, cl = blockIdx.x / nch;
    const int groups = (int)((a.N + kF4StepRows * tg - 1) / (kF4StepRows * tg));
    // this cluster's tile groups, side by side, so that a copy fetches a round of them
    const int mine = groups / ncl + (cl < groups % ncl ? 1 : 0), first = cl * (groups / ncl) + min(cl, groups % ncl);
    const int64_t m0 = (int64_t)blockIdx.y * kF4Tokens;
    const int mn = (int)min((int64_t)kF4Tokens, a.M - m0);
    // the row's slices, spread evenly over passes x CTAs
    const int parts = passes * nch, sq = a.nsl / parts, srem = a.nsl % parts;

    // this lane's codes of block b in a stage: matrix rows g and g + 8 are rows 2 g and 2 g + 1 of the
    // tile, so that a wavefront of 16 lanes reads 32 bytes of four rows of one parity, which the
    // swizzle keeps in different banks (row 2 g + 1: the other 16 bytes, 128 further)
    // (block b: bits 5 and 6 flipped by b)
    const int at = warp * (kF4Stages * kF4StageBytes) + g * 256 + ((g & 3) << 5) + t * 8;
    const int sc = kF4ScaleAt + warp * (kF4Stages * kF4ScaleBytes) + g * 32;
    // pieces of a buffer: [tiles side by side][tile of the round][warp along the row]
    const int mypiece = kF4SumAt + (tw * R * wk + kw) * PIECE;
    // this lane's place of token 2 t, row 2 g; the other token flips bit 6, the other row bit 5
    const int put = spread(4 * f4_sum_at(2 * t, 2 * g));

    // Adds round `round` (tile groups i0 .. of this CTA, `rn` of them, the first at place sg of the segment) over the
    // `act` warps that have a slice, in warp order.
    auto add_round = [&](int round, int i0, int sg, int rn, int act, bool fresh) {
        if (!mbar_wait_warp(bar, round & 1, abort)) return;
        const uint8_t *buf = smem + kF4SumAt + (round & 1) * BUF;
        for (int e = threadIdx.x; e < tg * R * 128 * NT; e += kF4Threads) {
            const int ti = e / (128 * NT), o = e & (128 * NT - 1), m = o >> 4, r = o & 15;
            const int i = ti & (R - 1);                     // ti = (tile side by side) * R + (tile of the round)
            if (i >= rn || m >= mn) continue;
            const uint8_t *src = buf + ti * wk * PIECE + spread(4 * f4_sum_at(m, r));
            float y = 0.0f;
            if (act == kF4Warps) {
                float v[kF4Warps];
#pragma unroll
                for (int w = 0; w < kF4Warps; ++w) v[w] = *reinterpret_cast<const float *>(src + w * PIECE);
#pragma unroll
                for (int w = 0; w < kF4Warps; ++w) y += v[w];
            } else {
#pragma unroll 4
                for (int w = 0; w < act; ++w) y += *reinterpret_cast<const float *>(src + w * PIECE);
            }
            if (CLUSTER) {
                float *dst = seg + (sg + i) * (128 * NT) + o;
                *dst = fresh ? y : *dst + y;
            } else {
                const int row = ((first + i0) * tg + (ti / R) * rn + i) * kF4StepRows + r;
                if (row < (int)a.N) f4_store<FMT>(a, m0 + m, row, y);
            }
        }
    };

    const int seg_len = CLUSTER ? f4_seg_tiles(NT) : mine;
    uint32_t xb[NT][32];
    float up[NT][2];
    uint32_t used = 0, filled = 0;                          // rounds of this warp's ring
    int round = 0, sl = -1, act = 0;
    bool dead = false;                                      // a wait ran out
    // Fills the other half of the ring with the round of group i, of rn groups: the warp's rn neighbouring tiles (lane 0;
    // the constants by every lane where TMA cannot)
    auto fill = [&](int i, int rn) {
        const int h = (int)(filled & 1u), row0 = ((first + i) * tg + tw * rn) * kF4StepRows;
        if (lane == 0) {
            const uint32_t codes = ring + h * (R * kF4StageBytes), scales = cring + h * (R * kF4ScaleBytes);
            mbar_arrive_expect_tx(full + 8 * h, rn * (kF4StageBytes + (VEC ? kF4ScaleBytes : 0)));
            tma_load_2d(codes, rn == R ? &a.codes : &a.codes_step, full + 8 * h, sl * 128, row0);
            if (VEC) tma_load_2d(scales, rn == R ? &a.scales : &a.scales_step, full + 8 * h, sl * 4, row0);
        }
        if (!VEC)
            for (int q = 0; q < rn; ++q)
                f4_scales(a, cring + (h * R + q) * kF4ScaleBytes, row0 + q * kF4StepRows, sl, lane);
        ++filled;
    };

    for (int s0 = 0; s0 < mine; s0 += seg_len) {
        const int s1 = min(mine, s0 + seg_len);
        for (int pass = 0; pass < passes; ++pass) {
            // tiles whose copies may run ahead: with several passes, this segment's only
            const int ahead = passes > 1 ? s1 : mine;
            if (passes > 1 || s0 == 0) {
                const int p = pass * nch + rank;
                act = sq + (p < srem ? 1 : 0);
                sl = kw < act && !dead ? p * sq + min(p, srem) + kw : -1;
                if (sl >= 0) {
#pragma unroll
                    for (int i = 0; i < kF4Stages; i += R) {
                        if (s0 + i < ahead) fill(s0 + i, min(R, ahead - s0 - i));
                        cp_commit();
                    }
                    // handed over in the places of this warp's own sums (a pass before has been added)
                    auto stage = [&](int m, int u) {
                        return reinterpret_cast<uint4 *>(smem + mypiece + (m >> 1) * BUF + (m & 1) * (wk * PIECE) + spread(16 * u));
                    };
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        f4_tokens<TABLE ? QLORA_FMT4_FP4_E2M1 : FMT, operand_scale(FMT, TABLE)>(
                            a.X + (m0 + 8 * nt) * a.K, mn - 8 * nt, a.K, sl * kF4StepK, lane, stage, xb[nt], up[nt][0], up[nt][1]);
                }
            }
            for (int i0 = s0; i0 < s1; i0 += R, ++round) {
                const int piece = mypiece + (round & 1) * BUF + put;
                if (sl < 0 && i0 > s0) add_round(round - 1, i0 - R, i0 - R - s0, R, act, pass == 0);
                if (sl >= 0) {
                    cp_wait<1>();
                    if (!VEC) __syncwarp();
                    const int h = (int)(used & 1u);
                    const bool landed = mbar_wait_warp(full + 8 * h, (used >> 1) & 1u, abort);
                    if (!landed) {
                        f4_drain(full, used, filled);         // the CTA goes on without this warp's slices
                        dead = true;
                        sl = -1;
                    }
                    ++used;
                    const int base = at + h * (R * kF4StageBytes), scale = sc + h * (R * kF4ScaleBytes);
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        if (!landed || i0 + i >= s1) break;
                        const float4 f0 = *reinterpret_cast<const float4 *>(smem + scale + i * kF4ScaleBytes);
                        const float4 f1 = *reinterpret_cast<const float4 *>(smem + scale + i * kF4ScaleBytes + 16);
                        const float c0[4] = {f0.x, f0.y, f0.z, f0.w}, c1[4] = {f1.x, f1.y, f1.z, f1.w};
                        float acc[NT][4];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const uint2 u = *reinterpret_cast<const uint2 *>(smem + (base ^ (b << 5)) + i * kF4StageBytes);
                            const uint2 v = *reinterpret_cast<const uint2 *>(smem + (base ^ (b << 5) ^ 16) + 128 + i * kF4StageBytes);
                            float cc[NT][4];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                uint32_t p[4], q[4];
                                if (TABLE) {
                                    decode_table(j ? u.y : u.x, table, p);
                                    decode_table(j ? v.y : v.x, table, q);
                                } else {
                                    decode<FMT>(a, j ? u.y : u.x, p);
                                    decode<FMT>(a, j ? v.y : v.x, q);
                                }
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    const uint32_t *x = xb[nt] + 8 * b + 4 * j;
                                    if (j == 0) mma_f16_first(cc[nt], p[0], q[0], p[1], q[1], x[0], x[1]);
                                    else mma_f16(cc[nt], p[0], q[0], p[1], q[1], x[0], x[1]);
                                }
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    const uint32_t *x = xb[nt] + 8 * b + 4 * j;
                                    mma_f16(cc[nt], p[2], q[2], p[3], q[3], x[2], x[3]);
                                }
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                acc[nt][0] = fmaf(c0[b], cc[nt][0], acc[nt][0]);
                                acc[nt][1] = fmaf(c0[b], cc[nt][1], acc[nt][1]);
                                acc[nt][2] = fmaf(c1[b], cc[nt][2], acc[nt][2]);
                                acc[nt][3] = fmaf(c1[b], cc[nt][3], acc[nt][3]);
                            }
                        }
                        // the round before, whose buffer the next round needs: a step after it ended
                        if (i == 0 && i0 > s0) add_round(round - 1, i0 - R, i0 - R - s0, R, act, pass == 0);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (8 * nt + 2 * t + (e & 1) < mn)
                                    *reinterpret_cast<float *>(smem + ((piece + i * wk * PIECE + nt * 512) ^ ((e & 1) << 6) ^ ((e >> 1) << 5))) = acc[nt][e] * up[nt][e & 1];
                    }
                }
                __syncwarp();                          // the stages have been read, the sums written
                if (lane == 0) mbar_arrive(bar);
                if (sl >= 0) {
                    if (i0 + kF4Stages < ahead) fill(i0 + kF4Stages, min(R, ahead - i0 - kF4Stages));
                    cp_commit();
                }
            }
            const int last = s0 + (s1 - s0 - 1) / R * R;
            add_round(round - 1, last, last - s0, s1 - last, act, pass == 0);
            if (CLUSTER) __syncthreads();              // the buffers are free for the next pass's hand-over
        }
        if (CLUSTER) {
            // the CTAs' sums in rank order; the CTAs take turns over the segment's elements
            cluster_sync();
            const uint32_t base = smem_addr(seg);
            for (int e = rank * kF4Threads + threadIdx.x; e < (s1 - s0) * 128 * NT; e += nch * kF4Threads) {
                const int i = e / (128 * NT), o = e & (128 * NT - 1), m = o >> 4;
                const int64_t row = (int64_t)(first + s0 + i) * kF4StepRows + (o & 15);
                if (m >= mn || row >= a.N) continue;
                float y = 0.0f;
                for (int c = 0; c < nch; ++c) y += ld_cluster_f32(map_to_rank(base + 4 * e, c));
                f4_store<FMT>(a, m0 + m, row, y);
            }
            cluster_sync();                            // before the next segment's sums, or the exit
        }
    }
}

template <int FMT, int NT, bool CLUSTER, bool VEC, bool TABLE>
cudaError_t f4_launch(const F4Args &a, int64_t groups, cudaStream_t st) {
    auto kernel = k_fmt4_linear<FMT, NT, CLUSTER, VEC, TABLE>;
    constexpr int smem = f4_smem(NT, CLUSTER, TABLE);
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.nch;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(kF4Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = CLUSTER ? at : at + 1;
    cudaError_t e = set_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    // clusters that run at once: fewer than SMs / size where the chip's SM groups do not divide
    int most = num_sms();
    if (CLUSTER) {
        static DeviceCache active[kF4MaxCluster + 1];
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        most = active[a.nch].get(dev, [&] {
            int n = 0;
            cfg.gridDim = dim3((unsigned)a.nch);
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            return e == cudaSuccess ? std::max(n, 1) : 0;
        });
        if (e != cudaSuccess) return e;
    }
    cfg.numAttrs = (CLUSTER ? 1 : 0) + (profiling_launches() ? 0 : 1);
    cfg.gridDim = dim3((unsigned)(std::min<int64_t>(groups, most) * a.nch), (unsigned)ceil_div(a.M, (int64_t)kF4Tokens));
    QNF4_LAUNCH("k_fmt4_linear", st, e = cudaLaunchKernelEx(&cfg, kernel, a));
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int FMT, int NT, bool TABLE>
cudaError_t f4_launch_form(const F4Args &a, int64_t groups, cudaStream_t st) {
    if (a.nch > 1 || a.passes > 1)
        return a.vec_scales ? f4_launch<FMT, NT, true, true, TABLE>(a, groups, st) : f4_launch<FMT, NT, true, false, TABLE>(a, groups, st);
    return a.vec_scales ? f4_launch<FMT, NT, false, true, TABLE>(a, groups, st) : f4_launch<FMT, NT, false, false, TABLE>(a, groups, st);
}

template <int FMT>
cudaError_t f4_launch_tiles(F4Args &a, int64_t groups, cudaStream_t st) {
    if (a.M > 8) return f4_launch_form<FMT, 2, false>(a, groups, st);
    // The table pays for Int4 once every CTA has work: [28672, 8192] 32.1 us instead of 35.8, [4096, 4096] 5.5 instead of 5.8,
    // but [1001, 1984], half the CTAs, 4.54 instead of 4.47 (filling it). E3M0 takes 31.9 without one. Beside the sums of 16
    // tokens there is no room for it.
    if (FMT == QLORA_FMT4_INT4 && groups * a.nch >= num_sms() && shared_window_at(kF4Reserved))
        return f4_launch_form<FMT, 1, FMT == QLORA_FMT4_INT4>(a, groups, st);
    return f4_launch_form<FMT, 1, false>(a, groups, st);
}

}  // namespace

cudaError_t launch_fmt4_linear(const __nv_bfloat16 *X, int64_t M, const uint8_t *codes, const float *absmax, int64_t rows,
                               int64_t cols, qlora_fmt4 f, void *Y, bool y_f32, cudaStream_t st) {
    F4Args a;
    a.X = X;
    for (int one : {0, 1})
        if (!make_map(one ? &a.codes_step : &a.codes, codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)cols / 2, (uint64_t)rows,
                      (uint64_t)cols / 2, 128, (one ? 1 : kF4Round) * kF4StepRows, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    a.absmax = absmax;
    a.Y = Y;
    a.M = M;
    a.N = rows;
    a.K = (int)cols;
    a.kbs = (int)(cols / kBlock1);
    a.nsl = (int)ceil_div(cols, kF4StepK);
    a.y_f32 = y_f32;
    a.two2 = 4;
    a.two4 = 16;
    a.two8 = 256;
    a.two12 = 4096;
    a.vec_scales = a.kbs % 4 == 0 && aligned16(absmax);
    for (int one : {0, 1})
        if (a.vec_scales &&
            !make_map(one ? &a.scales_step : &a.scales, absmax, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, (uint64_t)a.kbs, (uint64_t)rows,
                      (uint64_t)a.kbs * 4, 4, (one ? 1 : kF4Round) * kF4StepRows, CU_TENSOR_MAP_SWIZZLE_NONE))
            return cudaErrorInvalidValue;
    // CTAs along a row: enough for a slice per warp, more while there are fewer tiles than SMs
    const int64_t tiles = ceil_div(rows, (int64_t)kF4StepRows);
    int64_t nch = ceil_div(a.nsl, kF4Warps);
    while (nch < kF4MaxCluster && tiles * (nch + 1) <= num_sms() && a.nsl >= 4 * (nch + 1)) ++nch;
    if (nch > kF4MaxCluster) nch = kF4MaxCluster;
    a.nch = (int)nch;
    a.passes = (int)ceil_div(a.nsl, nch * kF4Warps);
    a.wk = kF4Warps;
    if (nch == 1)
        while (a.wk > 1 && a.wk / 2 >= a.nsl) a.wk /= 2;
    const int64_t groups = ceil_div(rows, (int64_t)kF4StepRows * (kF4Warps / a.wk));
    switch (f) {
        case QLORA_FMT4_INT4: return f4_launch_tiles<QLORA_FMT4_INT4>(a, groups, st);
        case QLORA_FMT4_FP4_E2M1: return f4_launch_tiles<QLORA_FMT4_FP4_E2M1>(a, groups, st);
        default: return f4_launch_tiles<QLORA_FMT4_FP4_E3M0>(a, groups, st);
    }
}

}  // namespace qnf4
