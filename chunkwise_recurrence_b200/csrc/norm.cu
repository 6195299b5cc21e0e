// Layer normalisation of libgdr, in front of a token mixer (per token, over
// the model's width) and behind it (per token and head): forward and
// backward.
//
// Per (token, head) row of d channels:
//   y = (x - mean) rstd w + b,   rstd = 1 / sqrt(var + eps)
// and backwards, with xh = (x - mean) rstd and g = dy w:
//   dx = rstd (g - mean(g) - xh mean(g xh)),
//   dw = sum over tokens of dy xh,   db = sum over tokens of dy.
// Both are bound by HBM: x (and dy) are read once, y (dx) is written once.  A
// row lives in the registers of G threads, so the mean, then the squared
// distances from it, are summed without a second read; the backward pass
// needs no saved statistics for the same reason.  Two rounds of reductions a
// row: sum x with sum g, then sum (x - mean)^2 with sum g (x - mean).
//
// dw and db: a group of threads stays with the same channels of the same
// head and walks over tokens, so its sums stay in registers; each block
// writes one partial row and a second kernel adds those, always in the same
// order.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "gdr_internal.h"

namespace gdr {
namespace {

constexpr int kMaxDim = 16384;

// V consecutive elements as one load
template <typename T, int V>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 8> { using type = uint4; };
template <>
struct Vec<__nv_bfloat16, 1> { using type = unsigned short; };
template <>
struct Vec<float, 4> { using type = float4; };
template <>
struct Vec<float, 1> { using type = float; };

__device__ __forceinline__ float lo16(uint32_t u) {
  return __uint_as_float(u << 16);
}
__device__ __forceinline__ float hi16(uint32_t u) {
  return __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ void unpack(const uint4 &r, float *f) {
  f[0] = lo16(r.x), f[1] = hi16(r.x), f[2] = lo16(r.y), f[3] = hi16(r.y);
  f[4] = lo16(r.z), f[5] = hi16(r.z), f[6] = lo16(r.w), f[7] = hi16(r.w);
}
__device__ __forceinline__ void unpack(const unsigned short &r, float *f) {
  f[0] = __uint_as_float((unsigned)r << 16);
}
__device__ __forceinline__ void unpack(const float4 &r, float *f) {
  f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w;
}
__device__ __forceinline__ void unpack(const float &r, float *f) { f[0] = r; }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&p);
}
template <int V>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float *f) {
  if constexpr (V == 8)
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]),
                   pack2(f[6], f[7]));
  else
    *p = __float2bfloat16_rn(f[0]);
}
template <int V>
__device__ __forceinline__ void store(float *p, const float *f) {
  if constexpr (V == 4)
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
  else
    *p = f[0];
}
// V parameters (fp32; V = 8 as two loads)
template <int V>
__device__ __forceinline__ void load_param(const float *p, float *f) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      unpack(__ldg(reinterpret_cast<const float4 *>(p + i)), f + i);
  } else {
    f[0] = __ldg(p);
  }
}

// Sums of two values over the G threads of a group.  G <= 32: within the
// warp; else over the group's warps through shared memory (every thread of
// the block calls; `sm` is not in use by an earlier call that some thread
// may still be reading).
template <int G>
__device__ __forceinline__ float2 group_sum(float2 s, float2 *sm) {
#pragma unroll
  for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1) {
    s.x += __shfl_xor_sync(~0u, s.x, o);
    s.y += __shfl_xor_sync(~0u, s.y, o);
  }
  if constexpr (G > 32) {
    constexpr int NW = G / 32;
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) sm[w] = s;
    __syncthreads();
    const float2 *g = sm + (w / NW) * NW;
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      s.x += g[i].x;
      s.y += g[i].y;
    }
  }
  return s;
}

constexpr int block_of(int G) { return G > 256 ? G : 256; }

// ----------------------------------------------------------------- forward

template <typename T, int V, int G, int NV>
__global__ void __launch_bounds__(block_of(G))
    gdr_norm_fwd_kernel(const T *x, long long ldx, const float *w,
                        const float *b, T *out, long long rows, int H, int d,
                        float eps) {
  using raw_t = typename Vec<T, V>::type;
  __shared__ float2 sm[2][block_of(G) / 32];
  constexpr int GPB = block_of(G) / G;
  const int l = threadIdx.x % G;
  const long long row = (long long)blockIdx.x * GPB + threadIdx.x / G;
  const bool has = row < rows;
  const long long tok = row / H;
  const int h = (int)(row - tok * H);
  const int nv = has ? d / V : 0;
  const T *xp = x + tok * ldx + (long long)h * d;
  raw_t raw[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    raw[j] = raw_t{};
    if (l + j * G < nv)
      raw[j] = __ldg(reinterpret_cast<const raw_t *>(xp) + l + j * G);
  }
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float f[V];
    unpack(raw[j], f);
#pragma unroll
    for (int v = 0; v < V; ++v) s += f[v];
  }
  const float inv = 1.f / (float)d;
  const float mean = group_sum<G>(make_float2(s, 0.f), sm[0]).x * inv;
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float f[V];
    unpack(raw[j], f);
    if (l + j * G < nv)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float c = f[v] - mean;
        q = fmaf(c, c, q);
      }
  }
  const float var = group_sum<G>(make_float2(q, 0.f), sm[1]).x * inv;
  const float rstd = 1.f / sqrtf(var + eps);
  T *op = out + row * d;
  const long long pc = (long long)h * d;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = l + j * G;
    if (i < nv) {
      float f[V], wf[V], bf[V];
      unpack(raw[j], f);
#pragma unroll
      for (int v = 0; v < V; ++v) wf[v] = 1.f, bf[v] = 0.f;
      if (w) load_param<V>(w + pc + i * V, wf);
      if (b) load_param<V>(b + pc + i * V, bf);
#pragma unroll
      for (int v = 0; v < V; ++v)
        f[v] = fmaf((f[v] - mean) * rstd, wf[v], bf[v]);
      store<V>(op + i * V, f);
    }
  }
}

// ---------------------------------------------------------------- backward

// Block (slice, head block): GPB groups; HB = min(H, GPB) heads, each by
// K = GPB / HB groups that take every (slices K)-th token.
template <typename T, int V, int G, int NV>
__global__ void __launch_bounds__(block_of(G))
    gdr_norm_bwd_kernel(const T *x, long long ldx, const float *w,
                        const T *dy, T *dx, float *part_w, float *part_b,
                        int ntok, int H, int d, float eps) {
  using raw_t = typename Vec<T, V>::type;
  constexpr int GPB = block_of(G) / G;
  constexpr int E = NV * V;
  __shared__ float2 sm[2][block_of(G) / 32];
  const int l = threadIdx.x % G, g = threadIdx.x / G;
  const int HB = H < GPB ? H : GPB, K = GPB / HB;
  const int hb = g % HB, kk = g / HB;
  const int head = blockIdx.y * HB + hb;
  const bool active = kk < K && head < H;
  const int nv = active ? d / V : 0;
  const int stride = gridDim.x * K;
  const int first = blockIdx.x * K;
  const int iters = (ntok - first + stride - 1) / stride;
  const long long pc = (long long)head * d;
  const float inv = 1.f / (float)d;
  float wf[E], aw[E], ab[E];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      wf[j * V + v] = 1.f;
      aw[j * V + v] = ab[j * V + v] = 0.f;
    }
    if (w && l + j * G < nv)
      load_param<V>(w + pc + (l + j * G) * V, wf + j * V);
  }
  for (int it = 0; it < iters; ++it) {
    const long long tok = first + (long long)it * stride + kk;
    const int n = tok < ntok ? nv : 0;
    const T *xp = x + tok * ldx + pc;
    const T *yp = dy + (tok * H + head) * d;
    raw_t xr[NV], yr[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xr[j] = yr[j] = raw_t{};
      if (l + j * G < n) {
        xr[j] = __ldg(reinterpret_cast<const raw_t *>(xp) + l + j * G);
        yr[j] = __ldg(reinterpret_cast<const raw_t *>(yp) + l + j * G);
      }
    }
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V], y[V];
      unpack(xr[j], f);
      unpack(yr[j], y);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s.x += f[v];
        s.y = fmaf(y[v], wf[j * V + v], s.y);
      }
    }
    s = group_sum<G>(s, sm[0]);
    const float mean = s.x * inv, m1 = s.y * inv;
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V], y[V];
      unpack(xr[j], f);
      unpack(yr[j], y);
      if (l + j * G < n)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float c = f[v] - mean;
          s.x = fmaf(c, c, s.x);
          s.y = fmaf(y[v] * wf[j * V + v], c, s.y);
        }
    }
    s = group_sum<G>(s, sm[1]);
    const float rstd = 1.f / sqrtf(s.x * inv + eps);
    const float m2 = s.y * inv * rstd;
    T *op = dx + (tok * H + head) * d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (l + j * G < n) {
        float f[V], y[V];
        unpack(xr[j], f);
        unpack(yr[j], y);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float xh = (f[v] - mean) * rstd;
          aw[j * V + v] = fmaf(y[v], xh, aw[j * V + v]);
          ab[j * V + v] += y[v];
          f[v] = rstd * (fmaf(y[v], wf[j * V + v], -m1) - xh * m2);
        }
        store<V>(op + (l + j * G) * V, f);
      }
    }
  }
  // the block's sums: its groups of one head are added in order
  if (!part_w && !part_b) return;
  const long long prow = (long long)blockIdx.x * H * d + pc;
  if (K == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (l + j * G < nv) {
        const long long o = prow + (l + j * G) * V;
        if (part_w) store<V % 4 ? 1 : 4>(part_w + o, aw + j * V);
        if (part_b) store<V % 4 ? 1 : 4>(part_b + o, ab + j * V);
        if constexpr (V == 8) {
          if (part_w) store<4>(part_w + o + 4, aw + j * V + 4);
          if (part_b) store<4>(part_b + o + 4, ab + j * V + 4);
        }
      }
    return;
  }
  if constexpr (GPB > 1) {
    __shared__ float acc[256 * E];
    for (int pass = 0; pass < 2; ++pass) {
      float *part = pass ? part_b : part_w;
      if (!part) continue;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e)
        acc[e * 256 + threadIdx.x] = pass ? ab[e] : aw[e];
      __syncthreads();
      if (kk == 0)
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (l + j * G < nv)
#pragma unroll
            for (int v = 0; v < V; ++v) {
              float s = 0.f;
              for (int k = 0; k < K; ++k)
                s += acc[(j * V + v) * 256 + (k * HB + hb) * G + l];
              part[prow + (l + j * G) * V + v] = s;
            }
    }
  }
}

// dst[c] = the sum over `slices` rows of part[.][c], c < n: 32 columns a
// block, 8 threads a column, always in the same order.  blockIdx.y chooses
// between the weight's and the bias's sums.
__global__ void __launch_bounds__(256)
    gdr_norm_sum_kernel(const float *part_w, const float *part_b, float *dw,
                        float *db, int n, int slices) {
  __shared__ float sm[8][32];
  const bool bias = blockIdx.y == 1 || !dw;
  const float *part = bias ? part_b : part_w;
  float *dst = bias ? db : dw;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  float s = 0.f;
  if (c < n)
    for (int i = k; i < slices; i += 8) s += part[(long long)i * n + c];
  sm[k][threadIdx.x & 31] = s;
  __syncthreads();
  if (k == 0 && c < n) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sm[i][threadIdx.x];
    dst[c] = s;
  }
}

// ---------------------------------------------------------------- launches

struct NormParams {
  const void *x;
  long long ldx;
  const float *w, *b;
  void *out;               // forward: y; backward: dx
  const void *dy;
  float *dw, *db;
  float *part_w, *part_b;  // [slices][H * d] each
  int slices;
  int ntok, H, d;
  float eps;
};

template <typename T, int V, int G, int NV>
cudaError_t launch_fwd(const NormParams &p, cudaStream_t s) {
  constexpr int GPB = block_of(G) / G;
  const long long rows = (long long)p.ntok * p.H;
  gdr_norm_fwd_kernel<T, V, G, NV>
      <<<(unsigned)((rows + GPB - 1) / GPB), block_of(G), 0, s>>>(
          static_cast<const T *>(p.x), p.ldx, p.w, p.b,
          static_cast<T *>(p.out), rows, p.H, p.d, p.eps);
  return cudaGetLastError();
}

// Rows of up to 64 values a lane stay within a warp; wider ones take a block.
template <typename T, int V>
cudaError_t run_fwd(const NormParams &p, cudaStream_t s) {
  constexpr int N = 64 / V;   // vectors per thread at 64 values
  const int nv = p.d / V;
  if (nv <= 1) return launch_fwd<T, V, 1, 1>(p, s);
  if (nv <= 2) return launch_fwd<T, V, 2, 1>(p, s);
  if (nv <= 4) return launch_fwd<T, V, 4, 1>(p, s);
  if (nv <= 8) return launch_fwd<T, V, 8, 1>(p, s);
  if (nv <= 16) return launch_fwd<T, V, 16, 1>(p, s);
  if (nv <= 32) return launch_fwd<T, V, 32, 1>(p, s);
  if (nv <= 32 * N / 4) return launch_fwd<T, V, 32, N / 4>(p, s);
  if (nv <= 32 * N / 2) return launch_fwd<T, V, 32, N / 2>(p, s);
  if (nv <= 32 * N) return launch_fwd<T, V, 32, N>(p, s);
  if (nv <= 256 * N / 4) return launch_fwd<T, V, 256, N / 4>(p, s);
  if (nv <= 256 * N / 2) return launch_fwd<T, V, 256, N / 2>(p, s);
  return launch_fwd<T, V, 256, N>(p, s);
}

// Threads per row of the backward pass: 16 values each.
int bwd_group(int d) {
  int g = 1;
  while (g * 16 < d) g *= 2;
  return g;
}
struct Cut {
  int slices, hblocks;
};
Cut bwd_cut(int ntok, int H, int d) {
  const int G = bwd_group(d);
  const int gpb = block_of(G) / G;
  const int hb = H < gpb ? H : gpb, k = gpb / hb;
  Cut c;
  c.hblocks = (H + hb - 1) / hb;
  const int want = (148 * (G > 512 ? 1 : G > 256 ? 2 : 3) + c.hblocks - 1) / c.hblocks;
  const int most = (ntok + k - 1) / k;
  c.slices = want < most ? want : most;
  return c;
}

template <typename T, int V, int G>
cudaError_t launch_bwd(const NormParams &p, cudaStream_t s) {
  const Cut c = bwd_cut(p.ntok, p.H, p.d);
  gdr_norm_bwd_kernel<T, V, G, 16 / V>
      <<<dim3(c.slices, c.hblocks), block_of(G), 0, s>>>(
          static_cast<const T *>(p.x), p.ldx, p.w,
          static_cast<const T *>(p.dy), static_cast<T *>(p.out), p.part_w,
          p.part_b, p.ntok, p.H, p.d, p.eps);
  return cudaGetLastError();
}
template <typename T, int V>
cudaError_t run_bwd(const NormParams &p, cudaStream_t s) {
  switch (bwd_group(p.d)) {
    case 1: return launch_bwd<T, V, 1>(p, s);
    case 2: return launch_bwd<T, V, 2>(p, s);
    case 4: return launch_bwd<T, V, 4>(p, s);
    case 8: return launch_bwd<T, V, 8>(p, s);
    case 16: return launch_bwd<T, V, 16>(p, s);
    case 32: return launch_bwd<T, V, 32>(p, s);
    case 64: return launch_bwd<T, V, 64>(p, s);
    case 128: return launch_bwd<T, V, 128>(p, s);
    case 256: return launch_bwd<T, V, 256>(p, s);
    case 512: return launch_bwd<T, V, 512>(p, s);
    default: return launch_bwd<T, V, 1024>(p, s);
  }
}

// 16-byte loads where every row starts on a 16-byte boundary, else one
// element at a time.
bool wide(const NormParams &p, int es) {
  return (long long)p.d * es % 16 == 0 && p.ldx * es % 16 == 0;
}

gdr_status check_norm(const void *x, long long ldx, int ntok, int H, int d,
                      float eps, gdr_dtype dtype) {
  if (ntok < 0 || H < 0 || d < 1) return GDR_ERR_INVALID_ARGUMENT;
  if (dtype != GDR_BF16 && dtype != GDR_FP32) return GDR_ERR_INVALID_ARGUMENT;
  if (!(eps >= 0.f)) return GDR_ERR_INVALID_ARGUMENT;
  if (d > kMaxDim || H > 65535) return GDR_ERR_UNSUPPORTED;
  if (ntok > INT_MAX / 2 || (long long)ntok * H > INT_MAX)
    return GDR_ERR_UNSUPPORTED;   // grid bounds
  if (ldx < (long long)H * d) return GDR_ERR_INVALID_ARGUMENT;
  return GDR_OK;
}
bool misaligned(const void *p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) != 0;
}
bool meet(const void *a, long long na, const void *b, long long nb) {
  if (!a || !b || na <= 0 || nb <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a);
  const uintptr_t y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

}  // namespace
}  // namespace gdr

extern "C" gdr_status gdr_layer_norm(const void *x, long long ldx,
                                     const float *weight, const float *bias,
                                     void *out, int ntok, int H, int d,
                                     float eps, gdr_dtype dtype,
                                     cudaStream_t stream) {
  using namespace gdr;
  gdr_status st = check_norm(x, ldx, ntok, H, d, eps, dtype);
  if (st != GDR_OK) return st;
  const long long n = (long long)ntok * H * d;
  if (n == 0) return GDR_OK;
  if (!x || !out) return GDR_ERR_INVALID_ARGUMENT;
  const void *ptrs[] = {x, weight, bias, out};
  for (const void *q : ptrs)
    if (misaligned(q)) return GDR_ERR_INVALID_ARGUMENT;
  const int es = dtype == GDR_BF16 ? 2 : 4;
  const long long pb = 4ll * H * d;
  if (meet(out, n * es, x, ((ntok - 1) * ldx + (long long)H * d) * es) ||
      meet(out, n * es, weight, pb) || meet(out, n * es, bias, pb))
    return GDR_ERR_INVALID_ARGUMENT;
  NormParams p{};
  p.x = x;
  p.ldx = ldx;
  p.w = weight;
  p.b = bias;
  p.out = out;
  p.ntok = ntok;
  p.H = H;
  p.d = d;
  p.eps = eps;
  cudaError_t e;
  if (dtype == GDR_BF16)
    e = wide(p, 2) ? run_fwd<__nv_bfloat16, 8>(p, stream)
                   : run_fwd<__nv_bfloat16, 1>(p, stream);
  else
    e = wide(p, 4) ? run_fwd<float, 4>(p, stream)
                   : run_fwd<float, 1>(p, stream);
  return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
}

extern "C" gdr_status gdr_layer_norm_backward(
    const void *x, long long ldx, const float *weight, const void *d_out,
    void *dx, float *d_weight, float *d_bias, int ntok, int H, int d,
    float eps, gdr_dtype dtype, cudaStream_t stream) {
  using namespace gdr;
  gdr_status st = check_norm(x, ldx, ntok, H, d, eps, dtype);
  if (st != GDR_OK) return st;
  const long long n = (long long)ntok * H * d, hd = (long long)H * d;
  if (hd == 0) return GDR_OK;
  if (n > 0 && (!x || !d_out || !dx)) return GDR_ERR_INVALID_ARGUMENT;
  const void *ptrs[] = {x, weight, d_out, dx, d_weight, d_bias};
  for (const void *q : ptrs)
    if (misaligned(q)) return GDR_ERR_INVALID_ARGUMENT;
  const int es = dtype == GDR_BF16 ? 2 : 4;
  const struct {
    const void *p;
    long long bytes;
  } b[] = {{dx, n * es},
           {d_weight, 4 * hd},
           {d_bias, 4 * hd},
           {x, ntok ? ((ntok - 1) * ldx + hd) * es : 0},
           {weight, 4 * hd},
           {d_out, n * es}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 6; ++j)
      if (meet(b[i].p, b[i].bytes, b[j].p, b[j].bytes))
        return GDR_ERR_INVALID_ARGUMENT;
  if (ntok == 0) {   // no token: the parameters' gradients are zero
    for (float *g : {d_weight, d_bias})
      if (g && cudaMemsetAsync(g, 0, 4 * hd, stream) != cudaSuccess)
        return GDR_ERR_CUDA;
    return GDR_OK;
  }
  NormParams p{};
  p.x = x;
  p.ldx = ldx;
  p.w = weight;
  p.out = dx;
  p.dy = d_out;
  p.dw = d_weight;
  p.db = d_bias;
  p.ntok = ntok;
  p.H = H;
  p.d = d;
  p.eps = eps;
  const int slices = bwd_cut(ntok, H, d).slices;
  const size_t one = (size_t)(4 * hd * slices + 255) & ~(size_t)255;
  const int narr = (d_weight ? 1 : 0) + (d_bias ? 1 : 0);
  void *ws = nullptr;
  if (narr) {
    st = scratch_get(&ws, one * narr, stream);
    if (st != GDR_OK) return st;
    char *at = static_cast<char *>(ws);
    if (d_weight) {
      p.part_w = reinterpret_cast<float *>(at);
      at += one;
    }
    if (d_bias) p.part_b = reinterpret_cast<float *>(at);
  }
  cudaError_t e;
  if (dtype == GDR_BF16)
    e = wide(p, 2) ? run_bwd<__nv_bfloat16, 8>(p, stream)
                   : run_bwd<__nv_bfloat16, 1>(p, stream);
  else
    e = wide(p, 4) ? run_bwd<float, 4>(p, stream)
                   : run_bwd<float, 1>(p, stream);
  if (e == cudaSuccess && narr) {
    gdr_norm_sum_kernel<<<dim3((unsigned)((hd + 31) / 32), narr), 256, 0,
                          stream>>>(p.part_w, p.part_b, d_weight, d_bias,
                                    (int)hd, slices);
    e = cudaGetLastError();
  }
  const cudaError_t f = ws ? scratch_put(ws, stream) : cudaSuccess;
  return (e == cudaSuccess && f == cudaSuccess) ? GDR_OK : GDR_ERR_CUDA;
}
