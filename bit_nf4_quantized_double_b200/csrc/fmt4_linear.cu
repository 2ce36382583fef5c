// Product of a few tokens with a weight kept in one of the group-scaled 4-bit formats of
// fmt4.cu (page "QLoRA: put the large model in memory, then change it with a small adapter",
// wq-win.github.io/llm/074-qlora, section 4, evidence 1 names the formats):
//   Y[m, n] = (1 / S) sum_b absmax[n, b] sum_{k in block b} v(code[n, k]) X[m, k].
//
// The 4-bit codes are read once from HBM; 0.5625 bytes per weight bound the kernel for few
// tokens. A weight becomes a bf16 value by bit placement, without a table: two codes of a
// word, 16 bits apart, go to the two halves of a register with their sign in bit 15 and
// their three magnitude bits where bf16 reads them as the format's own value times a power
// of two (a subnormal for Int4), and one bf16x2 multiplication by a power of two makes the
// value normal. The three formats' values have at most three significant bits and X is bf16,
// so every product is exact; sums, block constants and the row sum are fp32, rounded once at
// the end.
#include "launch.h"
#include "stream4.cuh"

namespace qnf4 {

using namespace tc;

namespace {

constexpr int kF4Warps = 8;
constexpr int kF4Threads = 32 * kF4Warps;
constexpr int kF4Stages = 4;
constexpr int kF4StageBytes = s4::kCodeBytes + s4::kStepRows * 16;   // codes, four fp32 constants per row
constexpr int kF4Tokens = 16;                                          // tokens per pass over the codes

__host__ __device__ constexpr int f4_red_floats(int nt) { return kF4Warps * 64 * nt; }
__host__ __device__ constexpr int f4_smem(int nt) { return kF4Warps * kF4Stages * kF4StageBytes + 2 * f4_red_floats(nt) * 4; }

struct F4Args {
    const __nv_bfloat16 *X;
    const uint8_t *codes;
    const float *absmax;
    void *Y;
    int64_t M, N;
    int K, kbs, nsteps, wk;    // inputs, blocks and steps per row; warps along a row (1, 2, 4, 8)
    int y_f32, vec_scales;
    float factor;              // (power of two of the decoded values) / S
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__host__ __device__ constexpr uint32_t pow2_bf16x2(int e) { return (uint32_t)(e + 127) * 0x00800080u; }

// Codes I and I + 4 (nibbles, from the low end) of a word as a bf16x2 pair. Int4: magnitude
// bits as a subnormal, m 2^-133 (odd I: 16 times that), times 2^126 or 2^122: m 2^-7. E2M1:
// exponent and mantissa bits at the end of bf16's exponent and the top of its mantissa: the
// value times 2^-126, subnormals included. E3M0: the exponent field alone, value times 2^-120.
template <int FMT, int I>
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, uint32_t w8) {
    constexpr int J = I & 1;                          // nibble J of the halves of w or w >> 8
    const uint32_t s = I < 2 ? w : w8;
    const uint32_t sign = s << (12 - 4 * J);
    if (FMT == QLORA_FMT4_INT4) {
        const uint32_t m = s & (J ? 0x00700070u : 0x00070007u);
        return mul_bf16x2(m | (sign & 0x80008000u), pow2_bf16x2(J ? 122 : 126));
    }
    if (FMT == QLORA_FMT4_FP4_E2M1) {
        const uint32_t m = (s << (6 - 4 * J)) & 0x01c001c0u;
        return mul_bf16x2(m | (sign & 0x80008000u), pow2_bf16x2(126));
    }
    const uint32_t m = (s << (7 - 4 * J)) & 0x03800380u;
    return mul_bf16x2(m | (sign & 0x80008000u), pow2_bf16x2(120));
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Copies of one step: rows row0 .. row0 + 15, inputs 256 s .. (zero past the last row or input).
__device__ __forceinline__ void f4_issue(const F4Args &a, uint32_t stage, int64_t row0, int s, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + (lane >> 3), c = lane & 7;
        const bool ok = row0 + r < a.N && s * s4::kStepK + 32 * c < a.K;
        const uint8_t *src = a.codes + (ok ? (row0 + r) * (int64_t)(a.K / 2) + s * 128 + c * 16 : 0);
        s4::cp16(stage + s4::code_off(r, c), src, ok);
    }
    const uint32_t sc = stage + s4::kCodeBytes;
    if (a.vec_scales) {
        if (lane < 16) {
            const bool ok = row0 + lane < a.N;
            s4::cp16(sc + lane * 16, a.absmax + (ok ? (row0 + lane) * (int64_t)a.kbs + 4 * s : 0), ok);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 8 * i + (lane >> 2), b = 4 * s + (lane & 3);
            const bool ok = row0 + r < a.N && b < a.kbs;
            s4::cp4(sc + r * 16 + (lane & 3) * 4, a.absmax + (ok ? (row0 + r) * (int64_t)a.kbs + b : 0), ok);
        }
    }
}

template <int FMT, int NT>
__global__ void __launch_bounds__(kF4Threads, 3) k_fmt4_linear(const __grid_constant__ F4Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_addr(smem) + warp * (kF4Stages * kF4StageBytes);
    float *red = reinterpret_cast<float *>(smem + kF4Warps * kF4Stages * kF4StageBytes);
    const int wk = a.wk, tg = kF4Warps / wk;               // warps per tile, tiles side by side in the CTA
    const int kw = warp % wk, tw = warp / wk;
    const int64_t groups = (a.N + s4::kStepRows * tg - 1) / (s4::kStepRows * tg);
    const int nq = (a.nsteps - kw + wk - 1) / wk;          // this warp's steps per tile
    const int64_t m0 = (int64_t)blockIdx.y * kF4Tokens;
    const int mn = (int)min((int64_t)kF4Tokens, a.M - m0);

    // the copies run ahead of the products by up to kF4Stages - 1 steps, over tile borders
    int64_t pg = blockIdx.x;
    int pq = 0, ps = 0;
    auto issue = [&]() {
        if (pg < groups && nq > 0) {
            f4_issue(a, ring + ps * kF4StageBytes, (pg * tg + tw) * s4::kStepRows, kw + pq * wk, lane);
            if (++pq == nq) {
                pq = 0;
                pg += gridDim.x;
            }
        }
        s4::cp_commit();
        ps = ps + 1 == kF4Stages ? 0 : ps + 1;
    };
#pragma unroll
    for (int i = 0; i < kF4Stages - 1; ++i) issue();

    const bool active = (t >> 1) == (g & 1);               // this lane's column holds this half's inputs
    int cs = 0, buf = 0;
    for (int64_t gi = blockIdx.x; gi < groups; gi += gridDim.x, buf ^= 1) {
        float acc[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = 0.0f;
        for (int q = 0; q < nq; ++q) {
            const int k0 = (kw + q * wk) * s4::kStepK;
            s4::cp_wait<kF4Stages - 2>();
            __syncwarp();
            issue();
            const uint32_t st = ring + cs * kF4StageBytes;
            cs = cs + 1 == kF4Stages ? 0 : cs + 1;
            const float4 s0 = s4::lds128f(st + s4::kCodeBytes + g * 16), s1 = s4::lds128f(st + s4::kCodeBytes + (g + 8) * 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int kl = k0 + 128 * h + 32 * t;
                uint32_t xb[NT][16];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int m = 4 * nt + (g >> 1);
                    const bool ld = active && m < mn && kl < a.K;
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.X + (m0 + m) * a.K + kl);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 v = ld ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
                        // inputs in the order of the decoded pairs: (1,5) (0,4) (3,7) (2,6)
                        xb[nt][4 * j] = prmt(v.x, v.z, 0x7632u);
                        xb[nt][4 * j + 1] = prmt(v.x, v.z, 0x5410u);
                        xb[nt][4 * j + 2] = prmt(v.y, v.w, 0x7632u);
                        xb[nt][4 * j + 3] = prmt(v.y, v.w, 0x5410u);
                    }
                }
                const uint4 w0 = s4::lds128(st + s4::code_off(g, 4 * h + t)), w1 = s4::lds128(st + s4::code_off(g + 8, 4 * h + t));
                float c[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t u = j == 0 ? w0.x : j == 1 ? w0.y : j == 2 ? w0.z : w0.w, u8 = u >> 8;
                    const uint32_t v = j == 0 ? w1.x : j == 1 ? w1.y : j == 2 ? w1.z : w1.w, v8 = v >> 8;
                    const uint32_t a0 = decode_pair<FMT, 0>(u, u8), a2 = decode_pair<FMT, 1>(u, u8);
                    const uint32_t a1 = decode_pair<FMT, 0>(v, v8), a3 = decode_pair<FMT, 1>(v, v8);
                    const uint32_t e0 = decode_pair<FMT, 2>(u, u8), e2 = decode_pair<FMT, 3>(u, u8);
                    const uint32_t e1 = decode_pair<FMT, 2>(v, v8), e3 = decode_pair<FMT, 3>(v, v8);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816(c[nt], a0, a1, a2, a3, xb[nt][4 * j], xb[nt][4 * j + 1]);
                        mma16816(c[nt], e0, e1, e2, e3, xb[nt][4 * j + 2], xb[nt][4 * j + 3]);
                    }
                }
                const float p0 = h ? s0.z : s0.x, p1 = h ? s0.w : s0.y, r0 = h ? s1.z : s1.x, r1 = h ? s1.w : s1.y;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    acc[nt][0] = fmaf(p1, c[nt][1], fmaf(p0, c[nt][0], acc[nt][0]));
                    acc[nt][1] = fmaf(r1, c[nt][3], fmaf(r0, c[nt][2], acc[nt][1]));
                }
            }
        }
        // the warps' sums along the row, added in warp order
        float *rb = red + buf * f4_red_floats(NT);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            rb[(warp * NT + nt) * 64 + t * 16 + g] = acc[nt][0];
            rb[(warp * NT + nt) * 64 + t * 16 + g + 8] = acc[nt][1];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < tg * NT * 64; i += kF4Threads) {
            const int r = i & 15, m = (i >> 4) % (4 * NT), ti = i / (64 * NT);
            const int64_t row = (gi * tg + ti) * s4::kStepRows + r;
            if (m >= mn || row >= a.N) continue;
            float y = 0.0f;
            for (int w = 0; w < wk; ++w) y += rb[((ti * wk + w) * NT + (m >> 2)) * 64 + (m & 3) * 16 + r];
            y *= a.factor;
            if (a.y_f32) static_cast<float *>(a.Y)[(m0 + m) * a.N + row] = y;
            else static_cast<__nv_bfloat16 *>(a.Y)[(m0 + m) * a.N + row] = __float2bfloat16_rn(y);
        }
    }
    s4::cp_wait<0>();
}

template <int FMT>
cudaError_t f4_launch(const F4Args &a, dim3 grid, int nt, cudaStream_t st) {
    auto go = [&](auto kernel, int smem) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        QNF4_LAUNCH("k_fmt4_linear", st, kernel<<<grid, kF4Threads, smem, st>>>(a));
        return cudaGetLastError();
    };
    switch (nt) {
        case 1: return go(k_fmt4_linear<FMT, 1>, f4_smem(1));
        case 2: return go(k_fmt4_linear<FMT, 2>, f4_smem(2));
        case 3: return go(k_fmt4_linear<FMT, 3>, f4_smem(3));
        default: return go(k_fmt4_linear<FMT, 4>, f4_smem(4));
    }
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
    a.nsteps = (int)ceil_div(cols, s4::kStepK);
    a.wk = a.nsteps >= 8 ? 8 : a.nsteps >= 4 ? 4 : a.nsteps >= 2 ? 2 : 1;
    a.y_f32 = y_f32;
    a.vec_scales = a.kbs % 4 == 0 && aligned16(absmax);
    a.factor = f == QLORA_FMT4_INT4 ? 128.0f / 7.0f : f == QLORA_FMT4_FP4_E2M1 ? 1.0f / 6.0f : 1.0f;
    const int64_t groups = ceil_div(rows, (int64_t)s4::kStepRows * (kF4Warps / a.wk));
    // equal shares: the fewest CTAs that give no CTA more than the share of a full grid
    const int64_t full = (int64_t)num_sms() * 3;
    const int64_t share = ceil_div(groups, full);
    const int nt = (int)ceil_div(M < kF4Tokens ? M : kF4Tokens, (int64_t)4);
    const dim3 grid((unsigned)ceil_div(groups, share), (unsigned)ceil_div(M, (int64_t)kF4Tokens));
    switch (f) {
        case QLORA_FMT4_INT4: return f4_launch<QLORA_FMT4_INT4>(a, grid, nt, st);
        case QLORA_FMT4_FP4_E2M1: return f4_launch<QLORA_FMT4_FP4_E2M1>(a, grid, nt, st);
        default: return f4_launch<QLORA_FMT4_FP4_E3M0>(a, grid, nt, st);
    }
}

}  // namespace qnf4
