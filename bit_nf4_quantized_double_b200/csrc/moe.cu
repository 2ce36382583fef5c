// A whole mixture-of-experts layer with NF4 experts for a few tokens (the page "QLoRA: put the
// large model in memory, then change it with a small adapter", wq-win.github.io/llm/074-qlora,
// sections 1 to 3, gives the stored weight and its product; the layer around it is the usual one):
//   logits[t, e] = sum_d X[t, d] R[e, d];  the k largest per token, ties to the lower expert;
//   weight = softmax over all experts at the chosen ones, divided by their sum if renorm;
//   Y[t] = sum_j weight[t, j] D_e (silu(G_e x_t) * (U_e x_t)),  e = expert[t, j].
// G, U [E F, D] and D [E D, F] hold the experts' rows one after the other.
//
// Two launches. k_moe_route: logits in fp64 (the products of bf16 values are exact there, and
// logits keep their order down to fp64's rounding of a sum), the tokens as scaled
// fp16, the grid barriers' counters cleared. k_moe_experts (cooperative, one CTA per SM): every
// CTA chooses the experts (the same few hundred comparisons in each), then streams its share of
// the gate and up tiles, a grid barrier, its share of the down tiles, a grid barrier, and its
// share of the weighted sums. The chosen experts' codes, 0.516 bytes per weight, bound it; the
// copies of the first down tiles run while the CTA waits at the first barrier.
//
// Products. Sixteen warps each hold the tokens of a job (an expert's tokens, at most eight) for
// one slice of 256 inputs in registers and take tiles of 16 weight rows: eight gate and the eight
// up rows of the same outputs, or 16 down rows. A code byte becomes an fp16 pair by one permute
// (byte * 256 + lane * 4 + the table's address) and one load from a table replicated per lane;
// mma.sync m16n8k16 sums a 64-block, fp32 arithmetic applies its constant. Eight more warps do
// everything else, in step with the others by two barriers per stage of a ring of four: one
// copies the codes (TMA), three add the sixteen warps' results in a fixed order, four turn int8
// constants into c = scale8 (scale2 / 127) + offset. With all of it in the sixteen warps a tile took
// about 560 instructions of a warp, 200 of them the products. 24 warps leave 80 registers, 32 of
// them tokens: what the roles share (shares of the phases, lists) stays in shared memory, since
// every spill in the products costs (147 instead of 127 us for the second case below); 52 bytes
// are still spilled. The waits' votes (a warp gives up as one) take 0.5 to 1 %.
//
// Measured, (T, E, k, d, f): (1, 8, 2, 4096, 11008) 53 us, (4, ...) 121, (32, ...) 213, floors of
// 21 / 58 / 85 at the measured copy rate; (1, 64, 8, 2048, 1024) 25 us, (16, ...) 70. About 16 us
// are fixed: logits, choice (2.5 to 5.5), two grid barriers (1.2 each), first copies, last sums. A
// group of 16 warps' tiles, 32 KB, takes 1.0 us (0.74 at the copy rate).
//
// Roundings besides fp32: the codebook to fp16 (2^-11 relative; bf16 would be 2^-8, as much as
// the output's own), the tokens to fp16 after scaling by a power of two per token and 256 inputs
// (exact within 2^-31 of the largest), silu(g) u to fp16 likewise (2^-11).
#include <cuda_fp16.h>

#include <algorithm>

#include "launch.h"
#include "tc.cuh"
#include "tmap.h"

namespace qnf4 {

using namespace tc;

namespace {

constexpr int kMoeWarps = 16;                       // that multiply
constexpr int kMoeScalers = 4, kMoeAdders = 3;
constexpr int kMoeHelpers = 1 + kMoeAdders + kMoeScalers;   // the copies, the sums, the block constants
constexpr int kMoeThreads = 32 * (kMoeWarps + kMoeHelpers);
constexpr int kMoeStages = 4;
constexpr int kMoeStepK = 256;
constexpr int kMoeStageBytes = kMoeWarps * 16 * 128;    // per warp 16 rows x 256 inputs
constexpr int kMoeScaleRow = 16 * 16 + 16;          // a row's block constants, four per warp, and 16 bytes against bank conflicts
constexpr int kMoeScaleBytes = 16 * kMoeScaleRow;   // of a stage
constexpr int kMoeJob = 8;                          // tokens of a job
constexpr int kMoeMaxTokens = 64, kMoeMaxExperts = 256, kMoeMaxTopK = 16;
constexpr int kMoeMaxSlots = kMoeMaxTokens * kMoeMaxTopK;
constexpr int kMoeMaxJobs = kMoeMaxExperts + kMoeMaxSlots / 8;

struct MoeJob {
    short expert, first, count, pad;                // slots order[first .. first + count - 1]
};

// Shared memory, by absolute address of the shared window. The table's 256 rows are 256 bytes
// apart, 128 bytes used (a word per lane); it starts at 65536, so that one permute of a code byte
// and a constant of the lane is the address of a lookup. The other halves of its rows hold the
// warps' sums, a buffer per stage. Below it the first stage, the constants and the lists, above
// it the other stages.
constexpr uint32_t kMoeTable = 65536;
constexpr uint32_t kMoeLow = 1024;                  // the system keeps the first 1024 bytes of the window
constexpr uint32_t kMoeHigh = 2 * 65536;
constexpr uint32_t kMoeScaleAt = kMoeLow + kMoeStageBytes;
constexpr uint32_t kMoeWeightAt = kMoeScaleAt + kMoeStages * kMoeScaleBytes;
constexpr uint32_t kMoeChoiceAt = kMoeWeightAt + kMoeMaxSlots * 4;
constexpr uint32_t kMoeOrderAt = kMoeChoiceAt + kMoeMaxSlots * 2;
constexpr uint32_t kMoeJobAt = kMoeOrderAt + kMoeMaxSlots * 2;
constexpr uint32_t kMoeBarAt = kMoeJobAt + kMoeMaxJobs * 8;
constexpr int kMoeSmem = kMoeHigh + (kMoeStages - 1) * kMoeStageBytes - kMoeLow;
constexpr uint32_t kMoePhaseAt = kMoeBarAt + 128;
static_assert(kMoeSmem <= 232448 && kMoePhaseAt + 128 <= kMoeTable, "shared memory");

__device__ __forceinline__ uint32_t stage_at(int st) { return st == 0 ? kMoeLow : kMoeHigh + (st - 1) * kMoeStageBytes; }

struct MoeWeight {
    // 128-byte swizzle. Where a row is a whole number of slices: bytes (128, rows, slices), boxes of a chunk's slices and
    // of one less (chunks differ by at most one); else bytes (cols / 2, rows), box of one slice.
    CUtensorMap codes, codes_less;
    const int8_t *scale8;
    const float *scale2, *offset;
};
struct MoeArgs {
    MoeWeight gate, up, down;
    const double *logits;                           // [T, E]
    const __half *xq;                               // [T, 256 nsl1] tokens / 2^e
    const float *xup;                               // [T, nsl1] 2^e
    float *h;                                       // [T k, F] silu(g) u; with nck1 > 1 [T k, nck1, 2, F] sums of g, u
    float *part;                                    // [T k, nck2, D]
    unsigned *counters;                             // two grid barriers
    __nv_bfloat16 *Y;
    int *experts;                                   // [T, k], or null
    float *weights;                                 // [T, k], or null
    int T, D, F, E, k, renorm;
    int whole1, whole2;                             // D, F are multiples of 256
    int nsl1, nsl2, lwk1, lwk2, nck1, nck2;         // of D and F: slices, log2 of warps along a row, chunks of at most 16 slices
    float q[16];                                    // codebook
};

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

// Eight values as fp16 after scaling by 2^-e, with 2^e such that the largest magnitude of the warp's
// 256 lies in [2^14, 2^15); returns 2^e. NaN and infinity stay what they are.
__device__ __forceinline__ float scale_f16(const float (&f)[8], uint4 &o) {
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) big = max(big, __float_as_uint(f[i]) & 0x7fffffffu);
    big = __reduce_max_sync(0xffffffffu, big);
    const int ex = min(max((int)(big >> 23), 24), 254);              // both powers kept normal
    const float down = __uint_as_float((uint32_t)(268 - ex) << 23);
    o.x = f16x2_of(f[0] * down, f[1] * down);
    o.y = f16x2_of(f[2] * down, f[3] * down);
    o.z = f16x2_of(f[4] * down, f[5] * down);
    o.w = f16x2_of(f[6] * down, f[7] * down);
    return __uint_as_float((uint32_t)(ex - 14) << 23);
}

// ---------------------------------------------------------------- routing
constexpr int kRouteThreads = 256;

__device__ __forceinline__ void bf16x8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

// A CTA per (expert, TOK tokens): its eight warps take 256 inputs each in turn and add their sums in warp order; then a
// CTA per eight (token, slice) conversions. The router is a few hundred KB, so the kernel is a latency, mostly of fp64
// additions that wait for one another: with a warp per logit it took 6 to 12 us. TOK is 1 while that leaves at most four
// CTAs per SM (8 experts, 32 tokens of 4096 inputs: 3.35 us, 5.35 with 4), else 4, which converts the router's values
// once for four tokens (64 experts, 16 tokens of 2048 inputs: 4.3 us, 5.0 with 1).
template <bool F32, int TOK>
__global__ void __launch_bounds__(kRouteThreads) k_moe_route(const __nv_bfloat16 *X, const void *router, double *logits,
                                                             __half *xq, float *xup, unsigned *counters, int T, int D,
                                                             int E, int nsl) {
    __shared__ double sums[TOK][kRouteThreads / 32];
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tq = (T + TOK - 1) / TOK;
    if (blockIdx.x == 0 && threadIdx.x < 2) counters[threadIdx.x] = 0u;
    if ((int)blockIdx.x >= E * tq) {
        const int i = ((int)blockIdx.x - E * tq) * (kRouteThreads / 32) + warp, t = i / nsl, s = i - t * nsl;
        if (t >= T) return;
        const int k = s * kMoeStepK + 8 * lane;
        float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (k < D) bf16x8(__ldg(reinterpret_cast<const uint4 *>(X + (int64_t)t * D + k)), f);
        uint4 o;
        const float up = scale_f16(f, o);
        *reinterpret_cast<uint4 *>(xq + (int64_t)t * nsl * kMoeStepK + k) = o;
        if (lane == 0) xup[t * nsl + s] = up;
        return;
    }
    const int e = (int)blockIdx.x / tq, t0 = ((int)blockIdx.x - e * tq) * TOK;
    double acc[TOK][2];
#pragma unroll
    for (int i = 0; i < TOK; ++i) acc[i][0] = acc[i][1] = 0.0;
#pragma unroll 2
    for (int k = 256 * warp + 8 * lane; k < D; k += 8 * kRouteThreads) {
        float r[8];
        if (F32) {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(router) + (int64_t)e * D + k);
            const float4 a = __ldg(p), b = __ldg(p + 1);
            r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
            r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
        } else {
            bf16x8(__ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(router) + (int64_t)e * D + k)), r);
        }
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
            if (TOK > 1 && t0 + i >= T) break;
            float x[8];
            bf16x8(__ldg(reinterpret_cast<const uint4 *>(X + (int64_t)(t0 + i) * D + k)), x);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j & 1] = fma((double)x[j], (double)r[j], acc[i][j & 1]);
        }
    }
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
        if (t0 + i >= T) break;
        double v = acc[i][0] + acc[i][1];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) sums[i][warp] = v;
    }
    __syncthreads();
    if (threadIdx.x < TOK && t0 + (int)threadIdx.x < T) {
        double v = 0.0;
#pragma unroll
        for (int w = 0; w < kRouteThreads / 32; ++w) v += sums[threadIdx.x][w];
        logits[(int64_t)(t0 + threadIdx.x) * E + e] = v;
    }
}

// Order-preserving key of a logit: NaN above everything, -0 with +0.
__device__ __forceinline__ unsigned long long logit_key(double v) {
    v += 0.0;
    if (v != v) return ~0ull;
    const unsigned long long b = (unsigned long long)__double_as_longlong(v);
    return (b >> 63) ? ~b : b | (1ull << 63);
}
// The logit of a key (NaN for every NaN, +0 for -0).
__device__ __forceinline__ double key_logit(unsigned long long k) {
    return __longlong_as_double((long long)((k >> 63) ? k ^ (1ull << 63) : ~k));
}
// exp(d) for d <= 0: the part of d that fp32 drops enters as its first-order term.
__device__ __forceinline__ float exp_f64(double d) {
    const float hi = (float)d;
    if (!(hi > -1e30f)) return expf(hi);
    return expf(hi) * (1.0f + (float)(d - (double)hi));
}

constexpr int kMoeBatch = 2048;                      // (token, expert) logits that are ranked at a time
struct MoeScratch {                                  // of the choice, before the stages are filled
    unsigned long long key[kMoeBatch];
    unsigned high[kMoeBatch];                        // the keys' upper halves
    float p[kMoeBatch];                              // exp(logit - largest)
    double top[kMoeMaxTokens];                       // largest logit
    unsigned tokens[kMoeMaxExperts][2];              // a bit per token that chose the expert
};

// The chosen experts of every token and their weights, by the whole CTA. A thread per (token, expert) counts the token's
// logits before its own (ties go to the lower expert), which is the expert's rank: no round waits for the one before.
__device__ __forceinline__ void moe_choose(const MoeArgs &a, MoeScratch &sh, float *weight, unsigned short *choice) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.E, batch = max(1, kMoeBatch / E);
#pragma unroll 1
    for (int t0 = 0; t0 < a.T; t0 += batch) {
        const int nt = min(batch, a.T - t0), n = nt * E;
        const double *logits = a.logits + (int64_t)t0 * E;
        for (int i = threadIdx.x; i < n; i += kMoeThreads) {
            const unsigned long long key = logit_key(__ldcg(logits + i));
            sh.key[i] = key;
            sh.high[i] = (unsigned)(key >> 32);
        }
        __syncthreads();
#pragma unroll 1
        for (int i = threadIdx.x; i < n; i += kMoeThreads) {
            const int t = i / E, e = i - t * E;
            const unsigned *row = sh.high + t * E, mine = row[e];
            int rank = 0, same = 0;
            if (E % 4 == 0) {
#pragma unroll 4
                for (int q = 0; q < E; q += 4) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(row + q);
                    rank += (v.x > mine ? 1 : 0) + (v.y > mine ? 1 : 0) + (v.z > mine ? 1 : 0) + (v.w > mine ? 1 : 0);
                    same += (v.x == mine ? 1 : 0) + (v.y == mine ? 1 : 0) + (v.z == mine ? 1 : 0) + (v.w == mine ? 1 : 0);
                }
            } else {
                for (int q = 0; q < E; ++q) {
                    rank += row[q] > mine ? 1 : 0;
                    same += row[q] == mine ? 1 : 0;
                }
            }
            if (same > 1) {                                  // the lower halves and the order of the experts decide
                const unsigned long long *full = sh.key + t * E, own = full[e];
#pragma unroll 1
                for (int q = 0; q < E; ++q) rank += row[q] == mine && (full[q] > own || (full[q] == own && q < e)) ? 1 : 0;
            }
            if (rank < a.k) {
                choice[(t0 + t) * a.k + rank] = (unsigned short)e;
                atomicOr(&sh.tokens[e][(t0 + t) >> 5], 1u << ((t0 + t) & 31));
            }
            if (rank == 0) sh.top[t0 + t] = key_logit(sh.key[i]);
        }
        __syncthreads();
#pragma unroll 1
        for (int i = threadIdx.x; i < n; i += kMoeThreads) sh.p[i] = exp_f64(key_logit(sh.key[i]) - sh.top[t0 + i / E]);
        __syncthreads();
        // weights: a warp per token
#pragma unroll 1
        for (int t = warp; t < nt; t += kMoeWarps + kMoeHelpers) {
            const unsigned short *mine = choice + (t0 + t) * a.k;
            double sum = 0.0;
            if (a.renorm) sum = lane < a.k ? (double)sh.p[t * E + mine[lane]] : 0.0;
            else
                for (int e = lane; e < E; e += 32) sum += (double)sh.p[t * E + e];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane < a.k) weight[(t0 + t) * a.k + lane] = (float)((double)sh.p[t * E + mine[lane]] / sum);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- experts
__device__ __forceinline__ int tile_row(int g) { return 2 * (g & 3) + (g >> 2); }
// Shared address of a warp's sum of (token m, matrix row r) of a stage's tile: the 32 lanes of a store
// (eight rows of tokens 2 t, or of tokens 2 t + 1) touch every bank once.
__device__ __forceinline__ uint32_t sum_at(int stage, int warp, int m, int r) {
    const int x = ((m ^ ((m >> 2) & 1)) << 4) + (r ^ ((m & 2) << 2));
    return kMoeTable + (uint32_t)((stage * kMoeWarps + warp) * 4 + (x >> 5)) * 256u + 128u + (uint32_t)(x & 31) * 4u;
}

// A phase's groups (16 warps' tiles), ordered (job, chunk, group).
struct MoePhase {
    int job, chunk, group;                          // this CTA's first group
    int count;                                      // its groups
    int per, nck, nsl;                              // groups per segment (a job's chunk); chunks; slices
    int lwk, kbs, width;                            // log2 of the warps along a row; blocks per row; outputs per expert
};
// First slice of chunk c: the slices are spread evenly.
__device__ __forceinline__ int chunk_first(const MoePhase &p, int c) {
    if (p.nck == 1) return c ? p.nsl : 0;
    const int q = p.nsl / p.nck, r = p.nsl - q * p.nck;
    return c * q + min(c, r);
}

// Position in the CTA's groups, those of phase 0 and then those of phase 1, with what its segment (job and chunk) fixes.
struct MoeCursor {
    int phase, jobno, chunk, group, left, run;      // run: groups left in the segment
    int first, slices, row, step;                   // the chunk's slices; the group's first weight row; rows of a group
    MoeJob job;
    __device__ __forceinline__ void segment(const MoePhase &p, const MoeJob *jobs) {
        run = min(left, p.per - group);
        if (run <= 0) return;
        first = chunk_first(p, chunk);
        slices = chunk_first(p, chunk + 1) - first;
        job = jobs[jobno];
        step = (phase ? 16 : 8) << (4 - p.lwk);
        row = job.expert * p.width + group * step;
    }
    __device__ __forceinline__ void enter(int ph, const MoePhase &p, const MoeJob *jobs) {
        phase = ph;
        jobno = p.job;
        chunk = p.chunk;
        group = p.group;
        left = p.count;
        segment(p, jobs);
    }
    __device__ __forceinline__ void start(const MoePhase &p0, const MoePhase &p1, const MoeJob *jobs) {
        enter(0, p0, jobs);
        if (left == 0) enter(1, p1, jobs);
    }
    __device__ __forceinline__ void next(const MoePhase &p0, const MoePhase &p1, const MoeJob *jobs) {
        --left;
        ++group;
        row += step;
        if (--run > 0) return;
        if (left == 0) {
            if (phase == 0) enter(1, p1, jobs);
            return;
        }
        const MoePhase &p = phase ? p1 : p0;
        group = 0;
        if (++chunk == p.nck) {
            chunk = 0;
            ++jobno;
        }
        segment(p, jobs);
    }
};

// This CTA's groups of a phase: an even share of groups and of the time that a segment's tokens take, `start` groups'
// worth, which a CTA that begins inside of a segment pays too.
__device__ __forceinline__ MoePhase moe_share(int njobs, int nck, int nsl, int lwk, int width, int rows, int cols, int start) {
    MoePhase p;
    const int tg = kMoeWarps >> lwk;
    p.per = (width / rows + tg - 1) >> (4 - lwk);
    const unsigned all = (unsigned)(p.per + start), n = (unsigned)njobs * nck * all, nc = gridDim.x, c = blockIdx.x;
    const unsigned q = n / nc, r = n - q * nc, x0 = c * q + min(c, r), x1 = x0 + q + (c < r ? 1 : 0);
    const unsigned seg = x0 / all, last = x1 / all;
    p.group = max((int)(x0 - seg * all) - start, 0);
    p.count = (int)(last - seg) * p.per + max((int)(x1 - last * all) - start, 0) - p.group;
    p.job = nck == 1 ? (int)seg : (int)(seg / nck);
    p.chunk = (int)seg - p.job * nck;
    p.nck = nck;
    p.nsl = nsl;
    p.lwk = lwk;
    p.kbs = cols / 64;
    p.width = width;
    return p;
}

struct MoeCta {
    uint8_t *window;                                // the shared window's address 0
    const MoeJob *jobs;
    const unsigned short *order;                    // slots by job
    uint32_t full, done, go;                        // barriers: per stage; per stage; the first grid barrier is passed
    volatile int *abort;
};

// Bounded grid barrier for one thread of the CTA, after the CTA's writes are ordered before it.
__device__ __forceinline__ void grid_arrive_wait(unsigned *counter, volatile int *abort) {
    __threadfence();
    atomicAdd(counter, 1u);
    const uint64_t t0 = global_timer_ns();
    while (true) {
        unsigned v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
        if (v >= gridDim.x) break;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            raise_status(QLORA_ERR_TIMEOUT);
            break;
        }
    }
    __threadfence();
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// Eight hidden values of a slot from input k on, from the sums of g and u over the chunks of D, in order.
__device__ __forceinline__ void moe_hidden(const MoeArgs &a, int slot, int k, float (&f)[8]) {
    auto add = [](float (&v)[8], const float *src) {
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(src)), y = __ldcg(reinterpret_cast<const float4 *>(src) + 1);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    };
    float u[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = 0; c < a.nck1; ++c) {
        const float *src = a.h + ((int64_t)slot * a.nck1 + c) * 2 * a.F + k;
        add(f, src);
        add(u, src + a.F);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = silu(f[i]) * u[i];
}

// A word of the lookup table, which no one writes after it was filled: the load may move freely.
__device__ __forceinline__ uint32_t table_word(uint32_t at) {
    uint32_t v;
    asm("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}

// ---------------- the sixteen warps that multiply
// Token operands of a slice: lane (g, t) holds token g of the job, inputs 64 b + 16 t + 8 j + 0..7 in
// xb[8 b + 4 j ..]; up: 2^e of tokens 2 t and 2 t + 1.
__device__ __forceinline__ void moe_tokens(const MoeArgs &a, const MoeCta &c, int phase, const MoeJob &job, int sl,
                                           uint32_t (&xb)[32], float (&up)[2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    up[0] = up[1] = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) xb[i] = 0u;
    if (phase == 0) {
        const int s0 = c.order[job.first + min(2 * t, job.count - 1)], s1 = c.order[job.first + min(2 * t + 1, job.count - 1)];
        if (g < job.count) {
            const int tok = c.order[job.first + g] / a.k;
            const uint4 *src = reinterpret_cast<const uint4 *>(a.xq + ((int64_t)tok * a.nsl1 + sl) * kMoeStepK) + 2 * t;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 v = __ldcg(src + 8 * (i >> 1) + (i & 1));
                xb[4 * i] = v.x;
                xb[4 * i + 1] = v.y;
                xb[4 * i + 2] = v.z;
                xb[4 * i + 3] = v.w;
            }
        }
        up[0] = __ldcg(a.xup + (s0 / a.k) * a.nsl1 + sl);
        up[1] = __ldcg(a.xup + (s1 / a.k) * a.nsl1 + sl);
    } else {
        // lane u converts inputs 8 u .. 8 u + 7 of a token's hidden values; the token's four lanes collect theirs. Two
        // tokens' values are on their way at a time (four of them: spills in the products)
        const int k = sl * kMoeStepK + 8 * lane;
        auto convert = [&](int m, const float (&f)[8]) {
            uint4 o;
            const float s = scale_f16(f, o);
            up[0] = 2 * t == m ? s : up[0];
            up[1] = 2 * t + 1 == m ? s : up[1];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int src = 8 * (i >> 1) + 2 * t + (i & 1);
                const uint32_t v0 = __shfl_sync(0xffffffffu, o.x, src), v1 = __shfl_sync(0xffffffffu, o.y, src);
                const uint32_t v2 = __shfl_sync(0xffffffffu, o.z, src), v3 = __shfl_sync(0xffffffffu, o.w, src);
                xb[4 * i] = g == m ? v0 : xb[4 * i];
                xb[4 * i + 1] = g == m ? v1 : xb[4 * i + 1];
                xb[4 * i + 2] = g == m ? v2 : xb[4 * i + 2];
                xb[4 * i + 3] = g == m ? v3 : xb[4 * i + 3];
            }
        };
        const bool in = k < a.F;
        if (a.nck1 == 1) {
#pragma unroll 1
            for (int m = 0; m < job.count; m += 2) {
                float4 v[4];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int slot = c.order[job.first + min(m + q, job.count - 1)];
                    const float4 *src = reinterpret_cast<const float4 *>(a.h + (int64_t)slot * a.F + k);
                    v[2 * q] = v[2 * q + 1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (in && (q == 0 || m + q < job.count)) {
                        v[2 * q] = __ldcg(src);
                        v[2 * q + 1] = __ldcg(src + 1);
                    }
                }
#pragma unroll 1
                for (int q = m; q < min(m + 2, job.count); ++q) {
                    const float f[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
                    convert(q, f);
                    v[0] = v[2];
                    v[1] = v[3];
                }
            }
        } else {
#pragma unroll 1
            for (int m = 0; m < job.count; ++m) {
                float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                if (in) moe_hidden(a, c.order[job.first + m], k, f);
                convert(m, f);
            }
        }
    }
}

__device__ __forceinline__ void moe_multiply(const MoeArgs &a, const MoeCta &c, const MoePhase &p0, const MoePhase &p1) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // this lane's codes (matrix rows g, g + 8: rows tile_row(g), + 8 of the warp's 16; block b: bits 5 and 6 flipped
    // by b), constants, sums (the other token: bit 6 flipped; the other row: bit 5)
    const uint32_t at = tile_row(g) * 128 + (((t >> 1) ^ tile_row(g)) << 4) + (t & 1) * 8;
    const uint32_t sc = kMoeScaleAt + tile_row(g) * kMoeScaleRow + warp * 16, put = sum_at(0, warp, 2 * t, g);
    const uint32_t table = kMoeTable | (uint32_t)(lane * 4);

    uint32_t xb[32];
    float up[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 32; ++i) xb[i] = 0u;
    int n = 0;                                               // group of the CTA
#pragma unroll 1
    for (int phase = 0; phase < 2; ++phase) {
        const MoePhase &p = phase ? p1 : p0;
        if (phase == 1 && p.count > 0 && !mbar_wait_warp(c.go, 0, c.abort)) return;   // every CTA's hidden values
        int jobno = p.job, chunk = p.chunk, run = min(p.count, p.per - p.group);
#pragma unroll 1
        for (int left = p.count; left > 0; left -= run, run = min(left, p.per)) {
            const int first = chunk_first(p, chunk), kw = warp & ((1 << p.lwk) - 1);
            const MoeJob job = c.jobs[jobno];
            const bool mine = kw < chunk_first(p, chunk + 1) - first;     // the warp has a slice in this segment
            const int mn = job.count;
            if (mine) moe_tokens(a, c, phase, job, first + kw, xb, up);
            // phase 0: all warps' eight gate rows, then all warps' up rows; phase 1: 16 rows per warp
            const int lo_at = warp * (phase ? 2048 : 1024), hi_at = phase ? 1024 : kMoeWarps * 1024;
#pragma unroll 1
            for (const int end = n + run; n < end; ++n) {
                const int st = n & (kMoeStages - 1);
                if (!mbar_wait_warp(c.full + 8 * st, (n / kMoeStages) & 1, c.abort)) return;
                if (mine) {
                    const uint32_t lo = stage_at(st) + lo_at + at;
                    const uint8_t *scale = c.window + (sc + st * kMoeScaleBytes);
                    const float4 f0 = *reinterpret_cast<const float4 *>(scale);
                    const float4 f1 = *reinterpret_cast<const float4 *>(scale + 8 * kMoeScaleRow);
                    const float c0[4] = {f0.x, f0.y, f0.z, f0.w}, c1[4] = {f1.x, f1.y, f1.z, f1.w};
                    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint8_t *code = c.window + (lo ^ (uint32_t)(b << 5));
                        const uint2 u = *reinterpret_cast<const uint2 *>(code), v = *reinterpret_cast<const uint2 *>(code + hi_at);
                        float cc[4];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t wu = j ? u.y : u.x, wv = j ? v.y : v.x;
                            uint32_t d[4], e[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                d[i] = table_word(prmt(wu, table, 0x7604u | ((uint32_t)i << 4)));
                                e[i] = table_word(prmt(wv, table, 0x7604u | ((uint32_t)i << 4)));
                            }
                            const uint32_t *x = xb + 8 * b + 4 * j;
                            if (j == 0) mma_f16_first(cc, d[0], e[0], d[1], e[1], x[0], x[1]);
                            else mma_f16(cc, d[0], e[0], d[1], e[1], x[0], x[1]);
                            mma_f16(cc, d[2], e[2], d[3], e[3], x[2], x[3]);
                        }
                        acc[0] = fmaf(c0[b], cc[0], acc[0]);
                        acc[1] = fmaf(c0[b], cc[1], acc[1]);
                        acc[2] = fmaf(c1[b], cc[2], acc[2]);
                        acc[3] = fmaf(c1[b], cc[3], acc[3]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (2 * t + (e & 1) < mn)
                            *reinterpret_cast<float *>(c.window + ((put + st * (kMoeWarps * 1024)) ^ (uint32_t)((e & 1) << 6) ^ (uint32_t)((e >> 1) << 5))) = acc[e] * up[e & 1];
                }
                __syncwarp();                                // the stage has been read, the sums written
                if (lane == 0) mbar_arrive(c.done + 8 * st);
            }
            if (++chunk == p.nck) {
                chunk = 0;
                ++jobno;
            }
        }
    }
}

// ---------------- the eight warps around them
// Copies of one group's codes. Rows past an expert's last tile are the next expert's or zeros (a group's tiles need not
// divide the expert): their sums are not used.
__device__ __forceinline__ void moe_copy(const MoeArgs &a, const MoeCta &c, const MoePhase &p, const MoeCursor &cur, int st) {
    const int lane = threadIdx.x & 31, n = cur.slices, rows = cur.phase ? 16 : 8, tg = kMoeWarps >> p.lwk;
    const uint32_t bar = c.full + 8 * st, base = stage_at(st);
    if (lane == 0) mbar_arrive_expect_tx(bar, n * tg * 2048);
    __syncwarp();
    if (cur.phase ? a.whole2 : a.whole1) {
        // one copy per tile and weight
        if (lane < tg) {
            const bool less = n * p.nck < p.nsl;             // a chunk one slice shorter than the longest
            const uint32_t dst = base + (lane << p.lwk) * rows * 128;
            const int row = cur.row + lane * rows;
            if (cur.phase) {
                tma_load_3d(dst, less ? &a.down.codes_less : &a.down.codes, bar, 0, row, cur.first);
            } else {
                tma_load_3d(dst, less ? &a.gate.codes_less : &a.gate.codes, bar, 0, row, cur.first);
                tma_load_3d(dst + kMoeWarps * 1024, less ? &a.up.codes_less : &a.up.codes, bar, 0, row, cur.first);
            }
        }
    } else {
        const int side = lane >> p.lwk, s = lane & ((1 << p.lwk) - 1);
        if (lane < kMoeWarps && s < n) {
            const uint32_t dst = base + lane * rows * 128;
            const int row = cur.row + side * rows, x = (cur.first + s) * 128;
            if (cur.phase) {
                tma_load_2d(dst, &a.down.codes, bar, x, row);
            } else {
                tma_load_2d(dst, &a.gate.codes, bar, x, row);
                tma_load_2d(dst + kMoeWarps * 1024, &a.up.codes, bar, x, row);
            }
        }
    }
    __syncwarp();
}

// Constants of a group, sixteen rows of a tile in two halves: gate and up rows, or the first and the last eight. A lane
// of the four warps has a unit, four blocks of a row, in each: (tile of the group, row, slice), slices fastest, so that
// the lanes read runs of a row. Its place relative to the half's first row is the same in every group of a chunk.
static_assert(32 * kMoeScalers >= 8 * kMoeWarps, "a unit per lane and half");
struct MoeUnit {
    int off;                                                 // first block, relative to the half's first row; INT_MAX: none
    int dst;                                                 // shared offset in a stage; 8 rows further for the second half
    int valid;                                               // blocks of the unit that the row has (up to 4)
    int key;                                                 // phase and chunk
};
struct MoeRaw {
    uint32_t w[2][2];                                        // the aligned words of int8 that hold a unit's blocks
    float s[2][2];                                           // second-level scales of the unit's first and last block
    int low[2];                                              // the half's first block, low bits
};

__device__ __forceinline__ void moe_unit(const MoePhase &p, const MoeCursor &cur, MoeUnit &u) {
    const int n = cur.slices, rows = cur.phase ? 16 : 8;
    const int hl = threadIdx.x - 32 * (kMoeWarps + 1 + kMoeAdders), rs = hl / n, q = hl - rs * n, r = rs & 7, side = rs >> 3;
    u.off = side < kMoeWarps >> p.lwk ? (side * rows + r) * p.kbs + 4 * (cur.first + q) : 0x7fffffff;
    u.dst = r * kMoeScaleRow + ((side << p.lwk) + q) * 16;
    u.valid = min(4, p.kbs - 4 * (cur.first + q));
    u.key = cur.phase * 65536 + cur.chunk;
}

// Loads the units of a group (rows past the expert's outputs stay zero: their sums are not used). ALIGNED: rows of a
// multiple of four blocks, so that a unit is one word, of one second-level group.
template <bool ALIGNED>
__device__ __forceinline__ void moe_raw(const MoeArgs &a, const MoePhase &p, const MoeCursor &cur, const MoeUnit &u, MoeRaw &raw) {
    const int room = (p.width - cur.group * cur.step) * p.kbs;   // blocks to the expert's end
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const MoeWeight &w = cur.phase ? a.down : i ? a.up : a.gate;
        const int past = cur.phase && i ? 8 : 0;             // rows
        const int64_t base = (int64_t)(cur.row + past) * p.kbs;
        raw.low[i] = (int)(base & 255);
        raw.w[i][0] = raw.w[i][1] = 0u;
        raw.s[i][0] = raw.s[i][1] = 0.0f;
        if (u.off < room - past * p.kbs) {
            const int8_t *p8 = w.scale8 + base;
            const float *p2 = w.scale2 + (base >> 8);
            const int b = raw.low[i] + u.off;                // the unit's first block, from p2's first on
            if (ALIGNED) {
                raw.w[i][0] = __ldg(reinterpret_cast<const unsigned int *>(p8 + u.off));
            } else {
                const int lo = (raw.low[i] & 3) + u.off;
                p8 -= raw.low[i] & 3;
                raw.w[i][0] = __ldg(reinterpret_cast<const unsigned int *>(p8 + (lo & ~3)));
                raw.w[i][1] = __ldg(reinterpret_cast<const unsigned int *>(p8 + ((lo + u.valid - 1) & ~3)));
                raw.s[i][1] = __ldg(p2 + ((b + u.valid - 1) >> 8));
            }
            raw.s[i][0] = __ldg(p2 + (b >> 8));
        }
    }
}

template <bool ALIGNED>
__device__ __forceinline__ void moe_constants(const MoeCta &c, int st, const MoeUnit &u, const MoeRaw &raw, float mu0, float mu1) {
    if (u.off == 0x7fffffff) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int b0 = raw.low[i] + u.off;                   // first block, modulo 256 and modulo 4
        const uint32_t w = ALIGNED ? raw.w[i][0] : __funnelshift_r(raw.w[i][0], raw.w[i][1], 8 * (b0 & 3));
        const float mu = i ? mu1 : mu0, s0 = raw.s[i][0] * (1.0f / 127.0f);
        float v[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            float s = s0;
            if (!ALIGNED && b >= 256 - (b0 & 255)) s = raw.s[i][1] * (1.0f / 127.0f);   // the next second-level group
            v[b] = fmaf((float)(int8_t)(w >> (8 * b)), s, mu);
            if (!ALIGNED && b >= u.valid) v[b] = 0.0f;
        }
        *reinterpret_cast<float4 *>(c.window + (kMoeScaleAt + st * kMoeScaleBytes + u.dst + i * 8 * kMoeScaleRow)) =
            make_float4(v[0], v[1], v[2], v[3]);
    }
}

// Adds four neighbouring values of a tile of N warps, in warp order; only the first n of them.
template <int N>
__device__ __forceinline__ void moe_add(const uint8_t *src, float4 &y, int n = N) {
    float4 v[N];
#pragma unroll
    for (int q = 0; q < N; ++q)
        v[q] = q < n ? *reinterpret_cast<const float4 *>(src + q * 1024) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int q = 0; q < N; ++q) y = make_float4(y.x + v[q].x, y.y + v[q].y, y.z + v[q].z, y.w + v[q].w);
}

// The sums of one group: hidden values, or partial sums of outputs. A lane has four neighbouring matrix rows r of a token
// and a tile; tile_row leaves them two outputs apart.
__device__ __forceinline__ void moe_sums(const MoeArgs &a, const MoeCta &c, const MoePhase &p, const MoeCursor &cur, int st) {
    const int lane = threadIdx.x & 31, act = cur.slices, ltg = 4 - p.lwk, q = lane & 3;
    const int total = ((cur.job.count + 1) >> 1) << (3 + ltg), out0 = cur.group * cur.step;
    const bool few = total == 8;                             // eight lanes have all values: a quarter of the warps for each eight
#pragma unroll 1
    for (int e0 = 0; e0 < total; e0 += 32) {
        const int e = few ? lane & 7 : e0 + lane, side = (e >> 3) & ((1 << ltg) - 1), m = ((e >> 2) & 1) + 2 * (e >> (3 + ltg));
        bool in = e < total && m < cur.job.count;
        const uint8_t *src = c.window + sum_at(st, side << p.lwk, in ? m : 0, 4 * q);
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (few) {
            const int run = (act + 3) >> 2, w = (lane >> 3) * run;
            moe_add<4>(src + w * 1024, y, min(run, act - w));
#pragma unroll
            for (int o = 8; o < 32; o *= 2) {
                y.x += __shfl_xor_sync(0xffffffffu, y.x, o);
                y.y += __shfl_xor_sync(0xffffffffu, y.y, o);
                y.z += __shfl_xor_sync(0xffffffffu, y.z, o);
                y.w += __shfl_xor_sync(0xffffffffu, y.w, o);
            }
            in = in && lane < 8;
        } else {
            int w = 0;
#pragma unroll 1
            for (; w + 8 <= act; w += 8) moe_add<8>(src + w * 1024, y);
            if (act & 4) {
                moe_add<4>(src + w * 1024, y);
                w += 4;
            }
            if (act & 2) {
                moe_add<2>(src + w * 1024, y);
                w += 2;
            }
            if (act & 1) moe_add<1>(src + w * 1024, y);
        }
        const int slot = c.order[cur.job.first + (in ? m : 0)];
        if (cur.phase) {
            // rows 8 (q / 2) + 2 i + (q & 1): the even lane takes the first four of eight, the odd one the others
            const bool odd = q & 1;
            const float s0 = __shfl_xor_sync(0xffffffffu, odd ? y.x : y.z, 1), s1 = __shfl_xor_sync(0xffffffffu, odd ? y.y : y.w, 1);
            const int out = out0 + side * 16 + 4 * q;
            if (in && out < p.width)
                __stcg(reinterpret_cast<float4 *>(a.part + ((int64_t)slot * a.nck2 + cur.chunk) * a.D + out),
                       odd ? make_float4(s0, y.z, s1, y.w) : make_float4(y.x, s0, y.y, s1));
        } else {
            // lanes 0 and 1 of four have gate, 2 and 3 up products of the same outputs: half of them each
            const bool up = q & 2;
            const float s0 = __shfl_xor_sync(0xffffffffu, up ? y.x : y.z, 2), s1 = __shfl_xor_sync(0xffffffffu, up ? y.y : y.w, 2);
            const float g0 = up ? s0 : y.x, g1 = up ? s1 : y.y, u0 = up ? y.z : s0, u1 = up ? y.w : s1;
            const int out = out0 + side * 8 + (up ? 4 : 0) + (q & 1);
            if (!in || out >= p.width) continue;
            if (a.nck1 == 1) {
                float *dst = a.h + (int64_t)slot * a.F + out;
                __stcg(dst, silu(g0) * u0);
                __stcg(dst + 2, silu(g1) * u1);
            } else {
                float *dst = a.h + ((int64_t)slot * a.nck1 + cur.chunk) * 2 * a.F + out;
                __stcg(dst, g0);
                __stcg(dst + 2, g1);
                __stcg(dst + a.F, u0);
                __stcg(dst + a.F + 2, u1);
            }
        }
    }
}

// Group n + 4 follows in the stage of group n once that is done: copied by one warp, its constants made by four; the
// sums of group n, whose places group n + 4 takes, by one of three warps in turn.
__device__ __forceinline__ void moe_copier(const MoeArgs &a, const MoeCta &c, const MoePhase &p0, const MoePhase &p1) {
    const int total = p0.count + p1.count;
    MoeCursor cur;
    cur.start(p0, p1, c.jobs);
#pragma unroll 1
    for (int n = 0; n < total; ++n) {
        const int st = n & (kMoeStages - 1);
        if (n >= kMoeStages && !mbar_wait_warp(c.done + 8 * st, (n / kMoeStages - 1) & 1, c.abort)) return;
        moe_copy(a, c, cur.phase ? p1 : p0, cur, st);
        cur.next(p0, p1, c.jobs);
    }
}

__device__ __forceinline__ void moe_adder(const MoeArgs &a, const MoeCta &c, const MoePhase &p0, const MoePhase &p1) {
    const int lane = threadIdx.x & 31, h = (threadIdx.x >> 5) - kMoeWarps - 1, total = p0.count + p1.count;
    // every CTA's hidden values: this CTA's are written once these warps are past its last group of phase 0, or have
    // given up (all three come here, so that none waits for another without a limit)
    auto meet = [&]() {
        named_bar_sync(1, 32 * kMoeAdders);
        if (h == 0 && lane == 0) {
            grid_arrive_wait(a.counters, c.abort);
            mbar_arrive(c.go);
        }
        __syncwarp();
    };
    if (h == 0 && lane < kMoeStages) mbar_arrive(c.full + 8 * lane);     // no sums before the first use of a stage
    __syncwarp();
    if (p0.count == 0) meet();
    MoeCursor cur;
    cur.start(p0, p1, c.jobs);
    int turn = 0;
#pragma unroll 1
    for (int n = 0; n < total; ++n) {
        const int st = n & (kMoeStages - 1);
        if (turn == h) {
            if (!mbar_wait_warp(c.done + 8 * st, (n / kMoeStages) & 1, c.abort)) {
                if (n < p0.count) meet();
                return;
            }
            moe_sums(a, c, cur.phase ? p1 : p0, cur, st);
            __syncwarp();
            if (lane == 0) mbar_arrive(c.full + 8 * st);
        }
        turn = turn + 1 == kMoeAdders ? 0 : turn + 1;
        cur.next(p0, p1, c.jobs);
        if (n == p0.count - 1) meet();
    }
}

__device__ __forceinline__ void moe_scaler(const MoeArgs &a, const MoeCta &c, const MoePhase &p0, const MoePhase &p1) {
    const int lane = threadIdx.x & 31, total = p0.count + p1.count;
    const float mu[3] = {__ldg(a.gate.offset), __ldg(a.up.offset), __ldg(a.down.offset)};
    // two groups' constants are loaded ahead, in registers
    MoeUnit ua, ub;
    MoeRaw ra, rb;
    MoeCursor ahead;
    ahead.start(p0, p1, c.jobs);
    ua.key = ub.key = -1;
    auto load = [&](MoeUnit &u, MoeRaw &r) {
        const MoePhase &p = ahead.phase ? p1 : p0;
        if (u.key != ahead.phase * 65536 + ahead.chunk) moe_unit(p, ahead, u);
        if (p.kbs & 3) moe_raw<false>(a, p, ahead, u, r);
        else moe_raw<true>(a, p, ahead, u, r);
        ahead.next(p0, p1, c.jobs);
    };
    auto step = [&](int n, MoeUnit &u, MoeRaw &r) {
        const int st = n & (kMoeStages - 1), phase = n >= p0.count;
        if (n >= kMoeStages && !mbar_wait_warp(c.done + 8 * st, (n / kMoeStages - 1) & 1, c.abort)) return false;
        const float mu0 = phase ? mu[2] : mu[0], mu1 = phase ? mu[2] : mu[1];
        if ((phase ? p1 : p0).kbs & 3) moe_constants<false>(c, st, u, r, mu0, mu1);
        else moe_constants<true>(c, st, u, r, mu0, mu1);
        __syncwarp();
        if (lane == 0) mbar_arrive(c.full + 8 * st);
        if (n + 2 < total) load(u, r);
        return true;
    };
    if (total > 0) load(ua, ra);
    if (total > 1) load(ub, rb);
#pragma unroll 1
    for (int n = 0; n < total; n += 2) {
        if (!step(n, ua, ra)) return;
        if (n + 1 < total && !step(n + 1, ub, rb)) return;
    }
}

// Shared memory starts elsewhere than the addresses say: reported, nothing touched.
__device__ __noinline__ void moe_misplaced() {
    if (threadIdx.x == 0) raise_status(QLORA_ERR_CUDA);
    griddep_wait();                                          // the routing kernel ends before this one
}

__global__ void __launch_bounds__(kMoeThreads, 1) k_moe_experts(const __grid_constant__ MoeArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // every shared address below is absolute (the compiler is not to know that they are equal from here on: with it, the
    // code became slower, 25.5 instead of 24.7 us for the smallest layer)
    uint32_t base = smem_addr(smem_raw);
    asm volatile("" : "+r"(base));
    if (base != kMoeLow) {
        moe_misplaced();
        return;
    }
    MoeCta c;
    c.window = smem_raw - smem_addr(smem_raw);
    float *weight = reinterpret_cast<float *>(c.window + kMoeWeightAt);
    unsigned short *choice = reinterpret_cast<unsigned short *>(c.window + kMoeChoiceAt);
    unsigned short *order = reinterpret_cast<unsigned short *>(c.window + kMoeOrderAt);
    MoeJob *jobs = reinterpret_cast<MoeJob *>(c.window + kMoeJobAt);
    MoeScratch &scratch = *reinterpret_cast<MoeScratch *>(c.window + kMoeHigh);
    c.jobs = jobs;
    c.order = order;
    c.full = kMoeBarAt;
    c.done = kMoeBarAt + 8 * kMoeStages;
    c.go = kMoeBarAt + 16 * kMoeStages;
    int *flags = reinterpret_cast<int *>(c.window + kMoeBarAt + 16 * kMoeStages + 8);   // abort, jobs
    c.abort = flags;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMoeStages; ++s) {
            mbar_init(c.full + 8 * s, 2 + kMoeScalers);      // the copies, the sums before, the constants
            mbar_init(c.done + 8 * s, kMoeWarps);
        }
        mbar_init(c.go, 1);
        flags[0] = 0;
    }
    fence_barrier_init();
    // table word (byte, lane) = fp16 pair (Q[byte >> 4] low half, Q[byte & 15] high half)
    for (int i = threadIdx.x; i < 256 * 8; i += kMoeThreads) {
        const uint32_t v = f16x2_of(a.q[i >> 7], a.q[(i >> 3) & 15]);
        *reinterpret_cast<uint4 *>(c.window + kMoeTable + (i >> 3) * 256 + (i & 7) * 16) = make_uint4(v, v, v, v);
    }
    for (int e = threadIdx.x; e < 2 * a.E; e += kMoeThreads) scratch.tokens[e >> 1][e & 1] = 0u;
    if (threadIdx.x < 3) tma_prefetch_desc(threadIdx.x == 0 ? &a.gate.codes : threadIdx.x == 1 ? &a.up.codes : &a.down.codes);
    griddep_wait();

    // ---------------- the chosen experts, the same in every CTA
    __syncthreads();
    moe_choose(a, scratch, weight, choice);
    const int slots = a.T * a.k;
    if (warp == 0) {
        // jobs in expert order: exclusive sums of the slots and jobs before an expert, 32 experts at a time
        int s0 = 0, j0 = 0;
#pragma unroll 1
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane, n = e < a.E ? __popc(scratch.tokens[e][0]) + __popc(scratch.tokens[e][1]) : 0;
            const int nj = (n + kMoeJob - 1) / kMoeJob;
            int s = n, j = nj;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int ps = __shfl_up_sync(0xffffffffu, s, o), pj = __shfl_up_sync(0xffffffffu, j, o);
                if (lane >= o) {
                    s += ps;
                    j += pj;
                }
            }
            const int first = s0 + s - n;
            for (int q = 0; q < nj; ++q)
                jobs[j0 + j - nj + q] = {(short)e, (short)(first + q * kMoeJob), (short)min(kMoeJob, n - q * kMoeJob), 0};
            if (e < a.E) scratch.p[e] = __int_as_float(first);
            s0 += __shfl_sync(0xffffffffu, s, 31);
            j0 += __shfl_sync(0xffffffffu, j, 31);
        }
        if (lane == 0) flags[1] = j0;
    }
    __syncthreads();
    // slots by expert, in token order
    for (int s = threadIdx.x; s < slots; s += kMoeThreads) {
        const int e = choice[s], t = s / a.k;
        const unsigned lo = scratch.tokens[e][0], hi = scratch.tokens[e][1];
        const int before = t < 32 ? __popc(lo & ((1u << t) - 1u)) : __popc(lo) + __popc(hi & ((1u << (t - 32)) - 1u));
        order[__float_as_int(scratch.p[e]) + before] = (unsigned short)s;
        if (blockIdx.x == 0) {
            if (a.experts) a.experts[s] = e;
            if (a.weights) a.weights[s] = weight[s];
        }
    }
    // ---------------- this CTA's share of the two phases
    MoePhase *phases = reinterpret_cast<MoePhase *>(c.window + kMoePhaseAt);
    // (a segment's tokens take 1.0 to 2.4 us in the first phase, 1.3 to 4 us in the second, a group 1 us)
    if (threadIdx.x == 0) phases[0] = moe_share(flags[1], a.nck1, a.nsl1, a.lwk1, a.F, 8, a.D, 2);
    if (threadIdx.x == 32) phases[1] = moe_share(flags[1], a.nck2, a.nsl2, a.lwk2, a.D, 16, a.F, slots >= 6 * flags[1] ? 4 : 2);
    fence_proxy_async_smem();                                // the copies overwrite the scratch
    __syncthreads();
    const MoePhase &p0 = phases[0], &p1 = phases[1];
    if (warp < kMoeWarps) moe_multiply(a, c, p0, p1);
    else if (warp == kMoeWarps) moe_copier(a, c, p0, p1);
    else if (warp <= kMoeWarps + kMoeAdders) moe_adder(a, c, p0, p1);
    else moe_scaler(a, c, p0, p1);
    __syncthreads();
    if (threadIdx.x == 0) {
        if (*c.abort) {                                      // a wait ran out: within a limit, let copies under way land
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000ull) {
            }
        }
        grid_arrive_wait(a.counters + 1, c.abort);
    }
    __syncthreads();

    // ---------------- Y[t] = sum over choices in order, each the sum of its chunks in order
    const int d4 = a.D / 4, parts = a.k * a.nck2;
    // (eight lanes read a line of 128 bytes; the lines are dealt out over the CTAs)
    for (int i = (int)((threadIdx.x >> 3) * gridDim.x + blockIdx.x) * 8 + (threadIdx.x & 7); i < a.T * d4;
         i += (int)gridDim.x * kMoeThreads) {
        const int t = i / d4, d = i - t * d4;
        const float4 *src = reinterpret_cast<const float4 *>(a.part + (int64_t)t * parts * a.D) + d;
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f}, s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        int j = 0, q = 0;
#pragma unroll 1
        for (int p = 0; p < parts; p += 8) {
            float4 v[8];
#pragma unroll
            for (int o = 0; o < 8; ++o)
                if (p + o < parts) v[o] = __ldcg(src + (int64_t)(p + o) * d4);
#pragma unroll
            for (int o = 0; o < 8; ++o) {
                if (p + o >= parts) break;
                s[0] += v[o].x;
                s[1] += v[o].y;
                s[2] += v[o].z;
                s[3] += v[o].w;
                if (++q == a.nck2) {
                    const float wt = weight[t * a.k + j++];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[e] = fmaf(wt, s[e], y[e]);
                        s[e] = 0.0f;
                    }
                    q = 0;
                }
            }
        }
        reinterpret_cast<uint2 *>(a.Y)[i] = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    }
}

// log2 of the warps along a row of nsl slices
int moe_along(int nsl) {
    int l = 4;
    while (l > 0 && (1 << (l - 1)) >= nsl) --l;
    return l;
}

struct MoeLayout {
    size_t logits, xq, xup, h, part, counters, total;
};
MoeLayout moe_layout(int64_t T, int64_t D, int64_t F, int64_t E, int64_t k) {
    const int64_t nsl1 = ceil_div(D, kMoeStepK), nck1 = ceil_div(nsl1, kMoeWarps), nck2 = ceil_div(ceil_div(F, kMoeStepK), kMoeWarps);
    MoeLayout l;
    size_t n = 0;
    auto take = [&](size_t b) {
        const size_t at = n;
        n += align256(b);
        return at;
    };
    l.logits = take((size_t)T * E * 8);
    l.xq = take((size_t)T * nsl1 * kMoeStepK * 2);
    l.xup = take((size_t)T * nsl1 * 4);
    l.h = take((size_t)T * k * F * (nck1 > 1 ? 2 * nck1 : 1) * 4);
    l.part = take((size_t)T * k * nck2 * D * 4);
    l.counters = take(8);
    l.total = n;
    return l;
}

bool moe_weight(MoeWeight *w, const NF4View &v, int rows, int nsl, int nck) {
    w->scale8 = v.scale8;
    w->scale2 = v.scale2;
    w->offset = v.offset;
    if (v.cols % kMoeStepK != 0)
        return make_map(&w->codes, v.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)v.cols / 2, (uint64_t)v.rows,
                        (uint64_t)v.cols / 2, 128, (uint32_t)rows, CU_TENSOR_MAP_SWIZZLE_128B);
    const uint64_t dims[3] = {128, (uint64_t)v.rows, (uint64_t)nsl}, strides[2] = {(uint64_t)v.cols / 2, 128};
    const uint32_t most = (uint32_t)ceil_div(nsl, nck), least = (uint32_t)std::max(nsl / nck, 1);
    const uint32_t box[3] = {128, (uint32_t)rows, most}, box_less[3] = {128, (uint32_t)rows, least};
    if (!make_map_3d(&w->codes, v.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return false;
    if (most == least) {                                     // every chunk the same: not used
        w->codes_less = w->codes;
        return true;
    }
    return make_map_3d(&w->codes_less, v.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, strides, box_less, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

// Shapes that the kernels take; T tokens, D, F, E experts, k of them per token.
bool moe_shape_ok(int64_t T, int64_t D, int64_t F, int64_t E, int64_t k) {
    return T >= 1 && T <= kMoeMaxTokens && E >= 1 && E <= kMoeMaxExperts && k >= 1 && k <= E && k <= kMoeMaxTopK && D >= 64 &&
           F >= 64 && D % 64 == 0 && F % 64 == 0 && D <= (1 << 16) && F <= (1 << 16);
}

size_t moe_workspace_bytes(int64_t T, int64_t D, int64_t F, int64_t E, int64_t k) { return moe_layout(T, D, F, E, k).total; }

cudaError_t launch_moe(const __nv_bfloat16 *X, int64_t T, const void *router, bool router_f32, const NF4View &gate,
                       const NF4View &up, const NF4View &down, int64_t D, int64_t F, int64_t E, int k, bool renorm,
                       __nv_bfloat16 *Y, int *experts, float *weights, void *ws, cudaStream_t st) {
    const MoeLayout l = moe_layout(T, D, F, E, k);
    char *p = static_cast<char *>(ws);
    MoeArgs a;
    double *logits = reinterpret_cast<double *>(p + l.logits);
    __half *xq = reinterpret_cast<__half *>(p + l.xq);
    float *xup = reinterpret_cast<float *>(p + l.xup);
    a.logits = logits;
    a.xq = xq;
    a.xup = xup;
    a.h = reinterpret_cast<float *>(p + l.h);
    a.part = reinterpret_cast<float *>(p + l.part);
    a.counters = reinterpret_cast<unsigned *>(p + l.counters);
    a.Y = Y;
    a.experts = experts;
    a.weights = weights;
    a.T = (int)T;
    a.D = (int)D;
    a.F = (int)F;
    a.E = (int)E;
    a.k = k;
    a.renorm = renorm;
    a.nsl1 = (int)ceil_div(D, kMoeStepK);
    a.nsl2 = (int)ceil_div(F, kMoeStepK);
    a.nck1 = (int)ceil_div(a.nsl1, kMoeWarps);
    a.nck2 = (int)ceil_div(a.nsl2, kMoeWarps);
    a.lwk1 = moe_along(a.nsl1);
    a.lwk2 = moe_along(a.nsl2);
    a.whole1 = D % kMoeStepK == 0;
    a.whole2 = F % kMoeStepK == 0;
    if (!moe_weight(&a.gate, gate, 8, a.nsl1, a.nck1) || !moe_weight(&a.up, up, 8, a.nsl1, a.nck1) ||
        !moe_weight(&a.down, down, 16, a.nsl2, a.nck2))
        return cudaErrorInvalidValue;
    const Codebook &cb = host_codebook();
    for (int i = 0; i < 16; ++i) a.q[i] = cb.q[i];
    const int sms = num_sms();
    cudaError_t e = set_smem(k_moe_experts, kMoeSmem);
    if (e != cudaSuccess) return e;
    if (!shared_window_at((int)kMoeLow)) return cudaErrorInvalidValue;   // the kernel's shared addresses are absolute

    const int tok = E * T <= 4 * sms ? 1 : 4;
    const int rgrid = (int)(E * ceil_div(T, (int64_t)tok) + ceil_div(T * a.nsl1, (int64_t)(kRouteThreads / 32)));
    const auto route = router_f32 ? (tok == 1 ? k_moe_route<true, 1> : k_moe_route<true, 4>)
                                  : (tok == 1 ? k_moe_route<false, 1> : k_moe_route<false, 4>);
    QNF4_LAUNCH("k_moe_route", st,
                route<<<rgrid, kRouteThreads, 0, st>>>(X, router, logits, xq, xup, a.counters, a.T, a.D, a.E, a.nsl1));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;

    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)sms);
    cfg.blockDim = dim3(kMoeThreads);
    cfg.dynamicSmemBytes = kMoeSmem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = profiling_launches() ? 1 : 2;
    QNF4_LAUNCH("k_moe_experts", st, e = cudaLaunchKernelEx(&cfg, k_moe_experts, a));
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qnf4
