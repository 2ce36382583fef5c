// Device helpers shared by the decode-time products that stream 4-bit codes through a
// warp's own ring of shared-memory stages (fmt4_linear.cu, moe.cu).
//
// A step is 16 weight rows x 256 inputs: 128 bytes of codes per row. A warp fills a stage
// with asynchronous 16-byte copies, four rows (whole 128-byte lines) per instruction, and
// waits only for its own copies (cp.async groups), so the ring needs no barrier.
//
// The products run on mma.sync m16n8k16 with the weight rows as A. Lane (g = lane / 4,
// t = lane % 4) takes 16 bytes of codes per row and 128 inputs, k = 32 t .. 32 t + 31: its
// lanes t = 0, 1 hold the first 64-block of the 128 inputs and t = 2, 3 the second. One sum
// over all four lanes would mix two blocks that have different constants. The eight columns
// of B keep them apart: column 2 m holds token m's inputs in lanes t < 2 and zeros in the
// others, column 2 m + 1 the reverse, so one mma gives both blocks' sums of four tokens.
#pragma once

#include "tc.cuh"

namespace qnf4 {
namespace s4 {

constexpr int kStepK = 256;                         // inputs per step
constexpr int kStepRows = 16;
constexpr int kCodeBytes = kStepRows * 128;

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool valid) {
    const int n = valid ? 16 : 0;                   // bytes read; the rest of the 16 is zero-filled
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, bool valid) {
    const int n = valid ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte offset in a stage of 16-byte chunk `c` (0..7) of row `r`: odd rows swap the halves of
// the 128 bytes, so that the eight lanes of a shared-memory wavefront (two rows, four
// chunks of one half) touch every bank once.
__device__ __forceinline__ uint32_t code_off(int r, int c) { return (uint32_t)(r * 128 + ((c ^ ((r & 1) << 2)) << 4)); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float4 lds128f(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}

}  // namespace s4
}  // namespace qnf4
