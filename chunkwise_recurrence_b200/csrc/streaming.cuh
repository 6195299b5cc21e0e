// streaming.cuh -- what the bandwidth-bound kernels (linear recurrence, layer
// normalisation) share: asynchronous copies into shared memory and arithmetic
// on pairs of fp32 values, and their launches.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace gdr {
namespace streaming {

// Launches overlap: the blocks of the next launch, if it is `early`, may take
// their places on the SMs as this one's last blocks leave (next_may_start,
// once all of this one's have begun) and wait there until it has ended and its
// results are visible (prior_done, before anything is read or written).  Layer
// norm one call after another, bf16: backward 8192 x 16 heads of 128 25.1 us a
// call without, 22.0 with; 32768 x 2048 72.4 and 69.4; forward 15.0 and 13.8,
// 45.8 and 45.0.
__device__ __forceinline__ void prior_done() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void next_may_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Reads what the launch before may have written, after prior_done().  An
// ordinary load: the read-only path (__ldg) is for what nothing writes from
// this kernel's first block on, and the wait does not order it.
template <typename T>
__device__ __forceinline__ T load(const T *p) {
  return *p;
}
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, int smem,
                   int cluster, bool early, cudaStream_t stream, A... args) {
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = early;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

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
