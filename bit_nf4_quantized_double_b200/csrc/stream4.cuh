// Device helpers shared by the decode-time products that stream 4-bit codes through a
// warp's own ring of shared-memory stages (fmt4_linear.cu, moe.cu).
//
// A step is 16 weight rows x 256 inputs: 128 bytes of codes per row. A warp fills a stage
// with asynchronous 16-byte copies, four rows (whole 128-byte lines) per instruction, and
// waits only for its own copies (cp.async groups), so the ring needs no barrier.
#pragma once

#include "tc.cuh"

namespace qnf4 {
namespace s4 {

constexpr int kStepK = 256;                         // inputs per step
constexpr int kStepRows = 16;
constexpr int kCodeBytes = kStepRows * 128;

// Asynchronous copies of n bytes (16 or 4, or 0 for zeros).
__device__ __forceinline__ void cp16n(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp4n(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte offset in a stage of 16-byte chunk `c` (0..7) of row `r`: the 32-byte blocks of a row are
// XOR-permuted by the row, so that four rows' reads of one block (eight bytes per lane, a
// wavefront of 16 lanes) touch every bank once.
__device__ __forceinline__ uint32_t code_off(int r, int c) { return (uint32_t)(r * 128 + ((c ^ ((r & 3) << 1)) << 4)); }

__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ float4 lds128f(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}

}  // namespace s4
}  // namespace qnf4
