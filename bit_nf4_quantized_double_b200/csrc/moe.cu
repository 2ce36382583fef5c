// A whole mixture-of-experts layer with NF4 experts for a few tokens (the page "QLoRA: put the
// large model in memory, then change it with a small adapter", wq-win.github.io/llm/074-qlora,
// sections 1 to 3, gives the stored weight and its product; the layer around it is the usual one):
//   logits[t, e] = sum_d X[t, d] R[e, d];  the k largest per token, ties to the lower expert;
//   weight = softmax over all experts at the chosen ones, divided by their sum if renorm;
//   Y[t] = sum_j weight[t, j] D_e (silu(G_e x_t) * (U_e x_t)),  e = expert[t, j].
// G, U [E F, D] and D [E D, F] hold the experts' rows one after the other.
//
// Two launches. k_moe_route: logits in fp64 (the products of bf16 values are exact there, and
// neighbouring logits keep their order whatever the order of the sum), the tokens as scaled
// fp16, the grid barriers' counters cleared. k_moe_experts (cooperative, one CTA per SM): every
// CTA chooses the experts (the same few hundred comparisons in each), then streams its share of
// the gate and up tiles, a grid barrier, its share of the down tiles, a grid barrier, and its
// share of the weighted sums. The chosen experts' codes, 0.516 bytes per weight, bound it; the
// copies of the first down tiles run while the CTA waits at the first barrier.
//
// Products. A warp holds the tokens of a job (an expert's tokens, at most 16) for one slice of
// 256 inputs in registers and takes tiles of 16 weight rows through its own ring of stages: eight
// gate and the eight up rows of the same outputs, or 16 down rows. A code byte becomes an fp16
// pair by one permute (address = byte * 256 + lane * 4) and one load from a table replicated per
// lane; mma.sync m16n8k16 sums a 64-block, fp32 arithmetic applies its constant
// c = scale8 (scale2 / 127) + offset. The warps' sums of a tile are added in warp order.
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

constexpr int kMoeWarps = 16;
constexpr int kMoeThreads = 32 * kMoeWarps;
constexpr int kMoeStages = 4;
constexpr int kMoeStepK = 256;
constexpr int kMoeStageBytes = 16 * 128;            // 16 rows x 256 inputs
constexpr int kMoeScaleBytes = 16 * 16;             // per row: two words of int8 constants, two scales
constexpr int kMoeJobTokens = 16;
constexpr int kMoeMaxTokens = 64, kMoeMaxExperts = 256, kMoeMaxTopK = 16;
constexpr int kMoeMaxSlots = kMoeMaxTokens * kMoeMaxTopK;
constexpr int kMoeMaxJobs = kMoeMaxExperts + kMoeMaxSlots / kMoeJobTokens;

struct MoeJob {
    short expert, first, count, pad;                // slots order[first .. first + count - 1]
};

// Shared memory. The table's 256 rows are 256 bytes apart, 128 bytes used (a word per lane); the
// other halves ("holes", 32 floats each) hold two buffers of the warps' sums.
constexpr int kMoeRingAt = 65536;
constexpr int kMoeScaleAt = kMoeRingAt + kMoeWarps * kMoeStages * kMoeStageBytes;
constexpr int kMoeWeightAt = kMoeScaleAt + kMoeWarps * kMoeStages * kMoeScaleBytes;
constexpr int kMoeChoiceAt = kMoeWeightAt + kMoeMaxSlots * 4;
constexpr int kMoeOrderAt = kMoeChoiceAt + kMoeMaxSlots * 2;
constexpr int kMoeJobAt = kMoeOrderAt + kMoeMaxSlots * 2;
constexpr int kMoeCountAt = kMoeJobAt + kMoeMaxJobs * 8;
constexpr int kMoeBarAt = kMoeCountAt + kMoeMaxExperts * 4;
constexpr int kMoeSmem = 1024 + kMoeBarAt + kMoeWarps * kMoeStages * 8 + 32;
static_assert(kMoeSmem <= 232448, "shared memory");

struct MoeWeight {
    CUtensorMap codes;                              // bytes [rows, cols / 2], 128-byte swizzle
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
    int nsl1, nsl2, wk1, wk2, nck1, nck2;           // of D and F: slices, warps along a row, chunks of at most 16 slices
    float q[16];                                    // codebook
};

__device__ __forceinline__ void cp4n(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
__device__ __noinline__ bool moe_wait_slow(uint32_t bar, uint32_t parity, volatile int *abort) {
    return mbar_wait(bar, parity, abort);
}
__device__ __forceinline__ bool moe_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    return mbar_try_wait(bar, parity) || moe_wait_slow(bar, parity, abort);
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
constexpr int kRouteTokens = 4;                     // tokens per logits item

__device__ __forceinline__ void bf16x8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

// One warp per item: (expert, four tokens) logits, then (token, slice) conversions. The router is
// E D values, a few hundred KB, so the kernel is a latency: a warp has all loads of 1024 inputs
// under way at once.
template <bool F32>
__global__ void __launch_bounds__(kRouteThreads) k_moe_route(const __nv_bfloat16 *X, const void *router, double *logits,
                                                             __half *xq, float *xup, unsigned *counters, int T, int D,
                                                             int E, int nsl) {
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, tq = (T + kRouteTokens - 1) / kRouteTokens;
    if (blockIdx.x == 0 && threadIdx.x < 2) counters[threadIdx.x] = 0u;
    const int items = E * tq + T * nsl;
    for (int it = blockIdx.x * (kRouteThreads / 32) + (threadIdx.x >> 5); it < items; it += gridDim.x * (kRouteThreads / 32)) {
        if (it < E * tq) {
            const int e = it / tq, t0 = (it - e * tq) * kRouteTokens;
            double acc[kRouteTokens];
#pragma unroll
            for (int i = 0; i < kRouteTokens; ++i) acc[i] = 0.0;
#pragma unroll 4
            for (int k = 8 * lane; k < D; k += 256) {
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
                for (int i = 0; i < kRouteTokens; ++i) {
                    if (t0 + i >= T) break;
                    float x[8];
                    bf16x8(__ldg(reinterpret_cast<const uint4 *>(X + (int64_t)(t0 + i) * D + k)), x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[i] = fma((double)x[j], (double)r[j], acc[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < kRouteTokens; ++i) {
                if (t0 + i >= T) break;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
                if (lane == 0) logits[(int64_t)(t0 + i) * E + e] = acc[i];
            }
        } else {
            const int c = it - E * tq, t = c / nsl, s = c - t * nsl, k = s * kMoeStepK + 8 * lane;
            float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (k < D) bf16x8(__ldg(reinterpret_cast<const uint4 *>(X + (int64_t)t * D + k)), f);
            uint4 o;
            const float up = scale_f16(f, o);
            *reinterpret_cast<uint4 *>(xq + (int64_t)t * nsl * kMoeStepK + k) = o;
            if (lane == 0) xup[t * nsl + s] = up;
        }
    }
}

// Order-preserving key of a logit: NaN above everything, -0 with +0.
__device__ __forceinline__ unsigned long long logit_key(double v) {
    v += 0.0;
    if (v != v) return ~0ull;
    const unsigned long long b = (unsigned long long)__double_as_longlong(v);
    return (b >> 63) ? ~b : b | (1ull << 63);
}
// exp(d) for d <= 0: the part of d that fp32 drops enters as its first-order term.
__device__ __forceinline__ float exp_f64(double d) {
    const float hi = (float)d;
    if (!(hi > -1e30f)) return expf(hi);
    return expf(hi) * (1.0f + (float)(d - (double)hi));
}

// One warp: the k largest logits of a token (ties to the lower expert) and their weights.
__device__ __forceinline__ void moe_choose(const MoeArgs &a, int t, int lane, float *weight, unsigned short *choice) {
    constexpr int PER = kMoeMaxExperts / 32;
    unsigned long long key[PER];
    double val[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        key[i] = 0ull;                                       // below every logit's key
        val[i] = 0.0;
        if (e < a.E) {
            val[i] = __ldcg(a.logits + (int64_t)t * a.E + e);
            key[i] = logit_key(val[i]);
        }
    }
    double top = 0.0, sum = 0.0;
    float mine = 0.0f;                                       // lane j: numerator of choice j
    for (int j = 0; j < a.k; ++j) {
        unsigned long long best = 0ull;
        double bv = 0.0;
        int be = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) {
                best = key[i];
                bv = val[i];
                be = lane + 32 * i;
            }
        const unsigned hi = __reduce_max_sync(0xffffffffu, (unsigned)(best >> 32));
        const unsigned lo = __reduce_max_sync(0xffffffffu, (unsigned)(best >> 32) == hi ? (unsigned)best : 0u);
        const bool match = (unsigned)(best >> 32) == hi && (unsigned)best == lo && be != 0x7fffffff;
        const int e = (int)__reduce_min_sync(0xffffffffu, match ? (unsigned)be : 0x7fffffffu);
        const double v = __shfl_sync(0xffffffffu, bv, e & 31);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 32 * i == e) key[i] = 0ull;
        if (j == 0) {
            top = v;
            // the softmax's denominator
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 32 * i < a.E) sum += (double)exp_f64(val[i] - top);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        const float p = exp_f64(v - top);
        if (lane == j) mine = p;
        if (lane == 0) choice[t * a.k + j] = (unsigned short)e;
    }
    if (a.renorm) {
        sum = lane < a.k ? (double)mine : 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane < a.k) weight[t * a.k + lane] = (float)((double)mine / sum);
}

// ---------------------------------------------------------------- experts
__device__ __forceinline__ int tile_row(int g) { return 2 * (g & 3) + (g >> 2); }
// Place of (token m, matrix row r) in a warp's sums of a tile: the 32 lanes of a store (eight rows of
// tokens 2 t, or of tokens 2 t + 1) touch every bank once.
__device__ __forceinline__ int sum_at(int m, int r) { return ((m ^ ((m >> 2) & 1)) << 4) + (r ^ ((m & 2) << 2)); }
// Byte offset of float x of piece p (pieces of 128 nt floats).
__device__ __forceinline__ uint32_t hole(int nt, int p, int x) {
    return (uint32_t)(p * nt * 4 + (x >> 5)) * 256u + 128u + (uint32_t)(x & 31) * 4u;
}

// Bounded grid barrier: every CTA of the cooperative launch arrives once.
__device__ __forceinline__ void grid_barrier(unsigned *counter, volatile int *abort) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(counter, 1u);
        const uint64_t t0 = global_timer_ns();
        unsigned v;
        do {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
            if (v < gridDim.x && global_timer_ns() - t0 > kWaitLimitNs) {
                *abort = 1;
                raise_status(QLORA_ERR_TIMEOUT);
                break;
            }
        } while (v < gridDim.x);
        __threadfence();
    }
    __syncthreads();
}

// Everything a warp of k_moe_experts carries along.
struct MoeWarp {
    uint8_t *smem;
    const MoeJob *jobs;
    const unsigned short *order;                    // slots by job
    int warp, lane, njobs;
    uint32_t ring, cring, full, bar;
    volatile int *abort;
    // the copies' position: phase (0 gate and up, 1 down, 2 none), the group's place and how many are left
    int iphase, igroup, iseg, ileft;                // segment iseg: job * nck + chunk
    int issued, done, round;
    bool dead;
};

struct MoePhase {
    int begin, end;                                 // this CTA's groups
    int per;                                        // groups per segment (a job's chunk)
};

// First slice of chunk c of nck: the slices are spread evenly.
__device__ __forceinline__ int chunk_first(int nsl, int nck, int c) {
    const int q = nsl / nck, r = nsl % nck;
    return c * q + min(c, r);
}
// This warp's slice in a segment of a phase, or -1.
__device__ __forceinline__ int moe_slice(const MoeArgs &a, const MoeWarp &w, int phase, int seg) {
    if (w.dead) return -1;
    const int nsl = phase ? a.nsl2 : a.nsl1, nck = phase ? a.nck2 : a.nck1, wk = phase ? a.wk2 : a.wk1;
    const int c = seg % nck, first = chunk_first(nsl, nck, c), n = chunk_first(nsl, nck, c + 1) - first, kw = w.warp & (wk - 1);
    return kw < n ? first + kw : -1;
}

// int8 constants and second-level scales of 16 rows (row(i), i = lane % 16), blocks 4 s ..: two aligned words of
// int8 from the byte of block 4 s on, the scales of the first and the last block's groups.
__device__ __forceinline__ void moe_scales(const int8_t *scale8, const float *scale2, uint32_t dst, int64_t row, int kbs, int s,
                                           int lane) {
    const int left = min(4, kbs - 4 * s);           // blocks of the step (>= 1)
    const int64_t b = row * kbs + 4 * s;            // first block
    const int64_t b4 = (b & ~3ll) + ((lane & 16) ? 4 : 0);
    const int64_t n = b + left - b4;                // bytes from b4 to the end of the step's blocks
    const uint32_t at = dst + (lane & 15) * 16 + ((lane & 16) ? 4 : 0);
    cp4n(at, n > 0 ? scale8 + b4 : scale8, n > 4 ? 4 : n > 0 ? (int)n : 0);
    cp4n(at + 8, scale2 + (((lane & 16) ? b + left - 1 : b) >> 8), 4);
}

// Fills the warp's next stage, if any group is left for it.
__device__ __forceinline__ void moe_fill(const MoeArgs &a, MoeWarp &w, const MoePhase &p0, const MoePhase &p1) {
    int sl = -1;
    while (w.iphase < 2) {
        if (w.ileft == 0) {                                  // the other phase
            if (++w.iphase == 2) break;
            w.ileft = p1.end - p1.begin;
            w.iseg = p1.begin / p1.per;
            w.igroup = p1.begin - w.iseg * p1.per;
            continue;
        }
        sl = moe_slice(a, w, w.iphase, w.iseg);
        if (sl >= 0) break;
        const int skip = min(w.ileft, (w.iphase ? p1.per : p0.per) - w.igroup);   // a segment without a slice for this warp
        w.ileft -= skip;
        w.igroup = 0;
        ++w.iseg;
    }
    if (w.iphase < 2) {
        const int st = w.issued & (kMoeStages - 1), lane = w.lane;
        const uint32_t dst = w.ring + st * kMoeStageBytes, cdst = w.cring + st * kMoeScaleBytes, bar = w.full + 8 * st;
        if (w.iphase == 0) {
            const int tile = (w.igroup * kMoeWarps + w.warp) / a.wk1, f0 = min(tile * 8, a.F - 8);
            const int row = w.jobs[w.iseg / a.nck1].expert * a.F + f0;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, kMoeStageBytes);
                tma_load_2d(dst, &a.gate.codes, bar, sl * 128, row);
                tma_load_2d(dst + 1024, &a.up.codes, bar, sl * 128, row);
            }
            moe_scales((lane & 8) ? a.up.scale8 : a.gate.scale8, (lane & 8) ? a.up.scale2 : a.gate.scale2, cdst, row + (lane & 7),
                       a.D / 64, sl, lane);
        } else {
            const int tile = (w.igroup * kMoeWarps + w.warp) / a.wk2, d0 = min(tile * 16, a.D - 16);
            const int row = w.jobs[w.iseg / a.nck2].expert * a.D + d0;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, kMoeStageBytes);
                tma_load_2d(dst, &a.down.codes, bar, sl * 128, row);
            }
            moe_scales(a.down.scale8, a.down.scale2, cdst, row + (lane & 15), a.F / 64, sl, lane);
        }
        ++w.issued;
        --w.ileft;
        if (++w.igroup == (w.iphase ? p1.per : p0.per)) {
            w.igroup = 0;
            ++w.iseg;
        }
    }
    cp_commit();
}

__device__ __noinline__ void moe_drain(uint32_t full, int done, int issued) {
    cp_wait<0>();
    const uint64_t t0 = global_timer_ns();
    for (; done < issued; ++done)
        while (!mbar_try_wait(full + 8 * (done & (kMoeStages - 1)), (done / kMoeStages) & 1))
            if (global_timer_ns() - t0 > kWaitLimitNs) return;
}

__device__ __forceinline__ float i8_f32(uint32_t word, int i) {     // byte i of word ^ 0x80808080, as int8
    return __uint_as_float(prmt(word, 0x4b000000u, 0x7440u + i)) - 8388736.0f;
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// Eight hidden values of a slot from input k on.
__device__ __forceinline__ void moe_hidden(const MoeArgs &a, int slot, int k, float (&f)[8]) {
    auto add = [](float (&v)[8], const float *src) {
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(src)), y = __ldcg(reinterpret_cast<const float4 *>(src) + 1);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    };
    if (a.nck1 == 1) {
        add(f, a.h + (int64_t)slot * a.F + k);
        return;
    }
    float u[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = 0; c < a.nck1; ++c) {                       // the chunks of D in order
        const float *src = a.h + ((int64_t)slot * a.nck1 + c) * 2 * a.F + k;
        add(f, src);
        add(u, src + a.F);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = silu(f[i]) * u[i];
}

// Runs groups g0 .. g1 - 1 of segment `seg` of a phase: tokens of the job (up to 8 NT) into registers, then rounds of
// R tiles per warp, summed over the warps: h, or the partial sums of the outputs.
template <int NT, int PHASE>
__device__ __forceinline__ void moe_run(const MoeArgs &a, MoeWarp &w, const MoePhase &p0, const MoePhase &p1, int seg, int g0, int g1) {
    constexpr int R = NT == 1 ? 2 : 1;
    const int lane = w.lane, g = lane >> 2, t = lane & 3;
    const int wk = PHASE ? a.wk2 : a.wk1, tg = kMoeWarps / wk, kw = w.warp % wk, tw = w.warp / wk;
    const int kbs = (PHASE ? a.F : a.D) / 64;
    const int nck = PHASE ? a.nck2 : a.nck1, nsl = PHASE ? a.nsl2 : a.nsl1, chunk = seg % nck;
    const MoeJob job = w.jobs[seg / nck];
    const int mn = job.count, sl = moe_slice(a, w, PHASE, seg);
    const int act = chunk_first(nsl, nck, chunk + 1) - chunk_first(nsl, nck, chunk);   // warps with a slice
    const int piece0 = tw * R * wk + kw;
    constexpr int kBufPieces = kMoeWarps * R;

    uint32_t xb[NT][32];
    float up[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        up[nt][0] = up[nt][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) xb[nt][i] = 0u;
    }
    if (sl >= 0) {
        if (PHASE == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int m = 8 * nt + g;
                if (m < mn) {
                    const int tok = w.order[job.first + m] / a.k;
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.xq + ((int64_t)tok * a.nsl1 + sl) * kMoeStepK) + 2 * t;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 v = __ldcg(src + 8 * (i >> 1) + (i & 1));
                        xb[nt][4 * i] = v.x;
                        xb[nt][4 * i + 1] = v.y;
                        xb[nt][4 * i + 2] = v.z;
                        xb[nt][4 * i + 3] = v.w;
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (8 * nt + 2 * t + i < mn)
                        up[nt][i] = __ldcg(a.xup + (w.order[job.first + 8 * nt + 2 * t + i] / a.k) * a.nsl1 + sl);
            }
        } else {
            // h is converted here, four tokens at a time through the places of this warp's own sums
            auto stage = [&](int m, int u) {
                const int p = (m >> 1) * kBufPieces + (NT == 1 ? (m & 1) * wk : 0);
                return reinterpret_cast<uint4 *>(w.smem + hole(NT, p + piece0, 4 * u + (NT == 1 ? 0 : (m & 1) * 128)));
            };
            const int k = sl * kMoeStepK + 8 * lane;
#pragma unroll
            for (int q = 0; q < 2 * NT; ++q) {
                if (4 * q >= mn) break;
                float f[4][8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[i][j] = 0.0f;
                    if (4 * q + i < mn && k < a.F) moe_hidden(a, w.order[job.first + 4 * q + i], k, f[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (4 * q + i >= mn) break;
                    uint4 o;
                    const float s = scale_f16(f[i], o);
                    *stage(i, lane) = o;
                    const int m = (4 * q + i) & 7;
                    up[q / 2][0] = 2 * t == m ? s : up[q / 2][0];
                    up[q / 2][1] = 2 * t + 1 == m ? s : up[q / 2][1];
                }
                __syncwarp();
                if ((g >> 2) == (q & 1) && 8 * (q / 2) + g < mn) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 v = *stage(g & 3, 8 * (i >> 1) + 2 * t + (i & 1));
                        xb[q / 2][4 * i] = v.x;
                        xb[q / 2][4 * i + 1] = v.y;
                        xb[q / 2][4 * i + 2] = v.z;
                        xb[q / 2][4 * i + 3] = v.w;
                    }
                }
                __syncwarp();
            }
        }
    }

    // this lane's codes in a stage (matrix rows g, g + 8: stage rows tile_row(g), + 8), constants, places of its sums
    const uint8_t *at[4];
#pragma unroll
    for (int b = 0; b < 4; ++b)
        at[b] = w.smem + kMoeRingAt + w.warp * (kMoeStages * kMoeStageBytes) + tile_row(g) * 128 +
                (((2 * b + (t >> 1)) ^ tile_row(g)) << 4) + (t & 1) * 8;
    const uint8_t *sc = w.smem + kMoeScaleAt + w.warp * (kMoeStages * kMoeScaleBytes) + tile_row(g) * 16;
    int put[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) put[e] = (int)hole(NT, 0, sum_at(2 * t + (e & 1), g + 8 * (e >> 1)));
    const float mu0 = __ldg(PHASE ? a.down.offset : a.gate.offset), mu1 = __ldg(PHASE ? a.down.offset : a.up.offset);
    // a tile's rows start at a multiple of 8, so the byte of the first block in its word depends on the row alone
    const int shift = 8 * ((tile_row(g) * kbs) & 3);
    const uint32_t lane4 = lane * 4;

    auto add_round = [&](int round, int i0, int rn) {
        if (!moe_wait(w.bar, round & 1, w.abort)) return;
        constexpr int ROWS = PHASE ? 16 : 8;                 // outputs of a tile
        for (int e = w.warp * 32 + lane; e < tg * R * ROWS * 8 * NT; e += kMoeThreads) {
            const int r = e & (ROWS - 1), m = (e / ROWS) & (8 * NT - 1), ti = e / (ROWS * 8 * NT), i = ti & (R - 1);
            const int tile = (i0 + i) * tg + ti / R;
            if (i >= rn || m >= mn || tile * ROWS >= (PHASE ? a.D : a.F)) continue;
            const uint8_t *src = w.smem + hole(NT, (round & 1) * kBufPieces + ti * wk, sum_at(m, r));
            float y = 0.0f;
#pragma unroll 8
            for (int q = 0; q < act; ++q) y += *reinterpret_cast<const float *>(src + q * (NT * 1024));
            const int slot = w.order[job.first + m], out = tile * ROWS + (r & 8) + tile_row(r & 7);
            if (PHASE == 0) {
                const uint8_t *src1 = w.smem + hole(NT, (round & 1) * kBufPieces + ti * wk, sum_at(m, r + 8));
                float u = 0.0f;
#pragma unroll 8
                for (int q = 0; q < act; ++q) u += *reinterpret_cast<const float *>(src1 + q * (NT * 1024));
                if (a.nck1 == 1) {
                    __stcg(a.h + (int64_t)slot * a.F + out, silu(y) * u);
                } else {
                    float *dst = a.h + ((int64_t)slot * a.nck1 + chunk) * 2 * a.F + out;
                    __stcg(dst, y);
                    __stcg(dst + a.F, u);
                }
            } else {
                __stcg(a.part + ((int64_t)slot * a.nck2 + chunk) * a.D + out, y);
            }
        }
    };

    for (int i0 = g0; i0 < g1; i0 += R, ++w.round) {
        const int rn = min(R, g1 - i0);
        if (sl < 0 && i0 > g0) add_round(w.round - 1, i0 - R, R);
        int used = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (sl < 0 || w.dead || i >= rn) break;
            const int st = w.done & (kMoeStages - 1), so = st * kMoeStageBytes;
            if (i == 0) cp_wait<kMoeStages - 1>();
            else cp_wait<kMoeStages - 2>();
            if (!moe_wait(w.full + 8 * st, (w.done / kMoeStages) & 1, w.abort)) {
                moe_drain(w.full, w.done, w.issued);         // the CTA goes on without this warp's slices
                w.dead = true;
                break;
            }
            __syncwarp();                                    // every lane's copies of the constants have landed
            ++w.done;
            ++used;
            // c = scale8 (scale2 / 127) + offset of the four blocks of both rows
            float c0[4], c1[4];
            {
                const uint4 q0 = *reinterpret_cast<const uint4 *>(sc + st * kMoeScaleBytes);
                const uint4 q1 = *reinterpret_cast<const uint4 *>(sc + st * kMoeScaleBytes + 128);
                const uint32_t w0 = __funnelshift_r(q0.x, q0.y, shift) ^ 0x80808080u;
                const uint32_t w1 = __funnelshift_r(q1.x, q1.y, shift) ^ 0x80808080u;
                const float s0 = __uint_as_float(q0.z) * (1.0f / 127.0f), s1 = __uint_as_float(q1.z) * (1.0f / 127.0f);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    c0[b] = fmaf(i8_f32(w0, b), s0, mu0);
                    c1[b] = fmaf(i8_f32(w1, b), s1, mu1);
                }
                if (kbs & 3) {                               // a second-level group may end inside the step
                    const int tile = (i0 + i) * tg + tw;
                    const int row = PHASE ? job.expert * a.D + min(tile * 16, a.D - 16) : job.expert * a.F + min(tile * 8, a.F - 8);
                    const int64_t b0 = (int64_t)(row + tile_row(g)) * kbs + 4 * sl, b1 = PHASE ? b0 + 8 * kbs : b0;
                    const float z0 = __uint_as_float(q0.w) * (1.0f / 127.0f), z1 = __uint_as_float(q1.w) * (1.0f / 127.0f);
#pragma unroll
                    for (int b = 1; b < 4; ++b) {
                        if (((b0 + b) >> 8) != (b0 >> 8)) c0[b] = fmaf(i8_f32(w0, b), z0, mu0);
                        if (((b1 + b) >> 8) != (b1 >> 8)) c1[b] = fmaf(i8_f32(w1, b), z1, mu1);
                    }
                }
            }
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint2 u = *reinterpret_cast<const uint2 *>(at[b] + so), v = *reinterpret_cast<const uint2 *>(at[b] + so + 1024);
                float cc[NT][4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t wu = j ? u.y : u.x, wv = j ? v.y : v.x;
                    uint32_t p[4], q[4];
#pragma unroll
                    for (int i2 = 0; i2 < 4; ++i2) {
                        p[i2] = *reinterpret_cast<const uint32_t *>(w.smem + prmt(wu, lane4, 0x5504u | ((uint32_t)i2 << 4)));
                        q[i2] = *reinterpret_cast<const uint32_t *>(w.smem + prmt(wv, lane4, 0x5504u | ((uint32_t)i2 << 4)));
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
            if (i == 0 && i0 > g0) add_round(w.round - 1, i0 - R, R);
            uint8_t *piece = w.smem + ((w.round & 1) * kBufPieces + piece0 + i * wk) * (NT * 1024);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (8 * nt + 2 * t + (e & 1) < mn)
                        *reinterpret_cast<float *>(piece + nt * 1024 + put[e]) = acc[nt][e] * up[nt][e & 1];
        }
        __syncwarp();                                        // the stages have been read, the sums written
        if (lane == 0) mbar_arrive(w.bar);
        for (int i = 0; i < used; ++i) moe_fill(a, w, p0, p1);
    }
    const int last = g0 + (g1 - g0 - 1) / R * R;
    add_round(w.round - 1, last, g1 - last);
    __syncthreads();                                         // the sums' places are free for the next run
}

template <int PHASE>
__device__ __forceinline__ void moe_phase(const MoeArgs &a, MoeWarp &w, const MoePhase &p0, const MoePhase &p1) {
    const MoePhase &p = PHASE ? p1 : p0;
    for (int i = p.begin; i < p.end;) {
        const int seg = i / p.per, first = seg * p.per, n = min(p.end, first + p.per);
        if (w.jobs[seg / (PHASE ? a.nck2 : a.nck1)].count <= 8) moe_run<1, PHASE>(a, w, p0, p1, seg, i - first, n - first);
        else moe_run<2, PHASE>(a, w, p0, p1, seg, i - first, n - first);
        i = n;
    }
}

__global__ void __launch_bounds__(kMoeThreads, 1) k_moe_experts(const __grid_constant__ MoeArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    MoeWarp w;
    w.smem = align1024(smem_raw);
    w.warp = threadIdx.x >> 5;
    w.lane = threadIdx.x & 31;
    const int warp = w.warp, lane = w.lane;
    float *weight = reinterpret_cast<float *>(w.smem + kMoeWeightAt);
    unsigned short *choice = reinterpret_cast<unsigned short *>(w.smem + kMoeChoiceAt);
    unsigned short *order = reinterpret_cast<unsigned short *>(w.smem + kMoeOrderAt);
    MoeJob *jobs = reinterpret_cast<MoeJob *>(w.smem + kMoeJobAt);
    int *count = reinterpret_cast<int *>(w.smem + kMoeCountAt);
    w.jobs = jobs;
    w.order = order;
    w.ring = smem_addr(w.smem) + kMoeRingAt + warp * (kMoeStages * kMoeStageBytes);
    w.cring = smem_addr(w.smem) + kMoeScaleAt + warp * (kMoeStages * kMoeScaleBytes);
    w.full = smem_addr(w.smem) + kMoeBarAt + warp * (kMoeStages * 8);
    w.bar = smem_addr(w.smem) + kMoeBarAt + kMoeWarps * kMoeStages * 8;
    int *flags = reinterpret_cast<int *>(w.smem + kMoeBarAt + kMoeWarps * kMoeStages * 8 + 8);   // abort, jobs
    w.abort = flags;
    if (lane < kMoeStages) mbar_init(w.full + 8 * lane, 1);
    if (threadIdx.x == 0) {
        mbar_init(w.bar, kMoeWarps);
        flags[0] = 0;
    }
    fence_barrier_init();
    // table word (byte, lane) = fp16 pair (Q[byte >> 4] low half, Q[byte & 15] high half)
    for (int i = threadIdx.x; i < 256 * 8; i += kMoeThreads) {
        const uint32_t v = f16x2_of(a.q[i >> 7], a.q[(i >> 3) & 15]);
        *reinterpret_cast<uint4 *>(w.smem + (i >> 3) * 256 + (i & 7) * 16) = make_uint4(v, v, v, v);
    }
    for (int e = threadIdx.x; e < a.E; e += kMoeThreads) count[e] = 0;
    if (threadIdx.x < 3) tma_prefetch_desc(threadIdx.x == 0 ? &a.gate.codes : threadIdx.x == 1 ? &a.up.codes : &a.down.codes);
    griddep_wait();

    // ---------------- the chosen experts, the same in every CTA
    for (int t = warp; t < a.T; t += kMoeWarps) moe_choose(a, t, lane, weight, choice);
    __syncthreads();
    const int slots = a.T * a.k;
    for (int s = threadIdx.x; s < slots; s += kMoeThreads) {
        atomicAdd(&count[choice[s]], 1);                     // a count: the order does not matter
        if (blockIdx.x == 0) {
            if (a.experts) a.experts[s] = choice[s];
            if (a.weights) a.weights[s] = weight[s];
        }
    }
    __syncthreads();
    if (warp == 0) {
        // jobs in expert order: exclusive sums of the slots and jobs before an expert, 32 experts at a time
        int s0 = 0, j0 = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane, n = e < a.E ? count[e] : 0, nj = (n + kMoeJobTokens - 1) / kMoeJobTokens;
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
                jobs[j0 + j - nj + q] = {(short)e, (short)(first + q * kMoeJobTokens),
                                         (short)min(kMoeJobTokens, n - q * kMoeJobTokens), 0};
            if (e < a.E) count[e] = first;
            s0 += __shfl_sync(0xffffffffu, s, 31);
            j0 += __shfl_sync(0xffffffffu, j, 31);
        }
        if (lane == 0) flags[1] = j0;
    }
    __syncthreads();
    // slots by expert, in slot order: a slot's place is the number of earlier slots of its expert
    for (int s = threadIdx.x; s < slots; s += kMoeThreads) {
        const int e = choice[s];
        int before = 0;
        for (int q = 0; q < s; ++q) before += choice[q] == e ? 1 : 0;
        order[count[e] + before] = (unsigned short)s;
    }
    __syncthreads();
    w.njobs = flags[1];

    // ---------------- this CTA's share of the two phases
    const int tg1 = kMoeWarps / a.wk1, tg2 = kMoeWarps / a.wk2;
    MoePhase p0, p1;
    p0.per = (a.F / 8 + tg1 - 1) / tg1;
    p1.per = (a.D / 16 + tg2 - 1) / tg2;
    const int64_t n0 = (int64_t)w.njobs * a.nck1 * p0.per, n1 = (int64_t)w.njobs * a.nck2 * p1.per, c = blockIdx.x, nc = gridDim.x;
    p0.begin = (int)(n0 * c / nc);
    p0.end = (int)(n0 * (c + 1) / nc);
    p1.begin = (int)(n1 * c / nc);
    p1.end = (int)(n1 * (c + 1) / nc);
    w.iphase = 0;
    w.ileft = p0.end - p0.begin;
    w.iseg = p0.begin / p0.per;
    w.igroup = p0.begin - w.iseg * p0.per;
    w.issued = w.done = w.round = 0;
    w.dead = false;
    for (int i = 0; i < kMoeStages; ++i) moe_fill(a, w, p0, p1);

    moe_phase<0>(a, w, p0, p1);
    grid_barrier(a.counters, w.abort);
    moe_phase<1>(a, w, p0, p1);
    grid_barrier(a.counters + 1, w.abort);

    // ---------------- Y[t] = sum over choices in order, each the sum of its chunks in order
    const int d4 = a.D / 4;
    for (int64_t i = (int64_t)blockIdx.x * kMoeThreads + threadIdx.x; i < (int64_t)a.T * d4; i += (int64_t)gridDim.x * kMoeThreads) {
        const int t = (int)(i / d4), d = (int)(i - (int64_t)t * d4);
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int j = 0; j < a.k; ++j) {
            const int slot = t * a.k + j;
            const float4 *src = reinterpret_cast<const float4 *>(a.part + (int64_t)slot * a.nck2 * a.D) + d;
            float4 s = __ldcg(src);
            for (int q = 1; q < a.nck2; ++q) {
                const float4 v = __ldcg(src + (int64_t)q * d4);
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            const float wt = weight[slot];
            y[0] = fmaf(wt, s.x, y[0]);
            y[1] = fmaf(wt, s.y, y[1]);
            y[2] = fmaf(wt, s.z, y[2]);
            y[3] = fmaf(wt, s.w, y[3]);
        }
        reinterpret_cast<uint2 *>(a.Y)[i] = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    }
}

int moe_along(int nsl) {
    int wk = kMoeWarps;
    while (wk > 1 && wk / 2 >= nsl) wk /= 2;
    return wk;
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

bool moe_weight(MoeWeight *w, const NF4View &v, int box_rows) {
    w->scale8 = v.scale8;
    w->scale2 = v.scale2;
    w->offset = v.offset;
    return make_map(&w->codes, v.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)v.cols / 2, (uint64_t)v.rows,
                    (uint64_t)v.cols / 2, 128, (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
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
    if (!moe_weight(&a.gate, gate, 8) || !moe_weight(&a.up, up, 8) || !moe_weight(&a.down, down, 16)) return cudaErrorInvalidValue;
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
    a.wk1 = a.nck1 > 1 ? kMoeWarps : moe_along(a.nsl1);
    a.wk2 = a.nck2 > 1 ? kMoeWarps : moe_along(a.nsl2);
    const Codebook &cb = host_codebook();
    for (int i = 0; i < 16; ++i) a.q[i] = cb.q[i];
    const int sms = num_sms();
    cudaError_t e = set_smem(k_moe_experts, kMoeSmem);
    if (e != cudaSuccess) return e;

    const int64_t items = E * ceil_div(T, (int64_t)kRouteTokens) + T * a.nsl1;
    const int rgrid = (int)std::min<int64_t>(ceil_div(items, (int64_t)(kRouteThreads / 32)), 4 * (int64_t)sms);
    if (router_f32)
        QNF4_LAUNCH("k_moe_route", st,
                    k_moe_route<true><<<rgrid, kRouteThreads, 0, st>>>(X, router, logits, xq, xup, a.counters, a.T, a.D, a.E, a.nsl1));
    else
        QNF4_LAUNCH("k_moe_route", st,
                    k_moe_route<false><<<rgrid, kRouteThreads, 0, st>>>(X, router, logits, xq, xup, a.counters, a.T, a.D, a.E, a.nsl1));
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
