// streaming.cuh -- what the bandwidth-bound kernels (linear recurrence, layer
// normalisation) share: asynchronous copies into shared memory and arithmetic
// on pairs of fp32 values.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

namespace gdr {
namespace streaming {

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&p);
}

// Asynchronous copy of `bytes` <= N bytes (N = 4, 8 or 16) into N bytes of
// shared memory; the rest is zero and not read.
template <int N>
__device__ __forceinline__ void copy_async(void *dst, const void *src,
                                           int bytes) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d),
                 "l"(src), "r"(bytes)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d),
                 "l"(src), "n"(N), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copies_landed() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
// Copies in groups: ends a group; waits until all but the last N have landed.
__device__ __forceinline__ void copies_sent() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_landed_but() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two fp32 values in a register pair, for the instructions that work on both
// at once.
struct Pair {
  unsigned long long u;
};
__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p.u) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ void split(Pair p, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p.u));
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d.u) : "l"(a.u), "l"(b.u), "l"(c.u));
  return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.u) : "l"(a.u), "l"(b.u));
  return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.u) : "l"(a.u), "l"(b.u));
  return d;
}

}  // namespace streaming
}  // namespace gdr
