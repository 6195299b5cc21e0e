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
// row lives in the registers of G threads, 16 values each, so the mean, then
// the squared distances from it, are summed without a second read; the
// backward pass needs no saved statistics for the same reason.  Two rounds of
// reductions a row: sum x with sum g, then sum (x - mean)^2 with
// sum g (x - mean).
//
// The grid is as many blocks as the GPU holds; a group of threads stays with
// the same channels of the same head and walks over tokens.  So w and b are
// read once, the next two rows are on their way while one is computed
// (asynchronous copies into shared memory), and the sums dw and db stay in
// registers; each block (or each group, where there are few) writes one partial
// row of them and a second kernel adds those, always in the same order.
//
// Measured in short runs (us, and the share of the 6.53 TB/s a copy reaches;
// bf16 unless said): forward 32768 x 2048 44 (0.93), 8192 x 16 heads of 128 12
// (0.85), 16384 x 4096 44 (0.94), 8192 x 8192 57 (0.72), fp32 16384 x 2048 47
// (0.87); backward 32768 x 2048 69 (0.89), 8192 x 16 x 128 21 (0.73), 16384 x
// 4096 79 (0.78), 8192 x 8192 92 (0.67), fp32 16384 x 2048 74 (0.83).  In runs
// of seconds 32768 x 16 heads of 128 take 48 us forward, 32768 x 2048 78
// backward.  Rows that are not aligned take about three times as long: 32768 x
// 2047 contiguous 121 and 206, with tokens apart 101 and 242.  What is left of
// the backward pass: about 5 us for its ends and the second kernel, and the
// two meetings a row, which two blocks an SM (128 registers a thread) do not
// hide in full.  Rows of more than 8192 channels take 1024 threads of 64
// registers, whose sums spill: 201 us for 4096 x 16384 (0.31).

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "gdr_internal.h"
#include "norm_rows.h"
#include "sm100.cuh"
#include "streaming.cuh"

namespace gdr {
namespace {

namespace cg = cooperative_groups;
using namespace streaming;

constexpr int kMaxDim = 16384;
constexpr int kE = 16;          // values of a row that a thread holds
// Blocks of up to 256 threads that an SM is meant to hold, and the registers
// that go with them (larger blocks: one).
constexpr int kFwdBlocks = 3, kBwdBlocks = 2;
constexpr int kSms = 148;

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
// Sums one or two values over the G threads of each group.  G <= 32: within
// the warp; else over the group's warps through shared memory, the group
// meeting at its own barrier (`sm` is not in use by an earlier call that some
// thread may still be reading).
template <int G, bool TWO>
__device__ __forceinline__ void group_sum(float &a, float &b, float2 *sm) {
  constexpr int W = G < 32 ? G : 32;
  if constexpr (W > 1 && TWO) {
    // the lower half of the threads goes on with a, the upper half with b
    const bool up = threadIdx.x & (W / 2);
    const float give = up ? a : b;
    float keep = up ? b : a;
    keep += __shfl_xor_sync(~0u, give, W / 2);
#pragma unroll
    for (int o = W / 4; o > 0; o >>= 1) keep += __shfl_xor_sync(~0u, keep, o);
    if constexpr (G <= 32) {
      const float other = __shfl_xor_sync(~0u, keep, W / 2);
      a = up ? other : keep;
      b = up ? keep : other;
    } else {
      if (threadIdx.x % 16 == 0)
        reinterpret_cast<float *>(sm)[threadIdx.x / 16] = keep;
    }
  } else {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) a += __shfl_xor_sync(~0u, a, o);
    if (G > 32 && threadIdx.x % 32 == 0) sm[threadIdx.x / 32].x = a;
  }
  if constexpr (G > 32) {
    constexpr int NW = G / 32;
    sm100::named_bar_sync(1 + threadIdx.x / G, G);
    const float2 *g = sm + threadIdx.x / G * NW;
    if constexpr (NW <= 8) {
      a = b = 0.f;
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        a += g[j].x;
        if constexpr (TWO) b += g[j].y;
      }
    } else {
      const float2 t = g[threadIdx.x % NW];
      a = t.x;
      if constexpr (TWO) b = t.y;
#pragma unroll
      for (int o = NW / 2; o > 0; o >>= 1) {
        a += __shfl_xor_sync(~0u, a, o);
        if constexpr (TWO) b += __shfl_xor_sync(~0u, b, o);
      }
    }
  }
}

constexpr int block_of(int G) { return G > 256 ? G : 256; }

// How a block's groups of G threads share heads and tokens: HB heads, each by
// K groups.
struct Share {
  int head, kk, K;
  bool active;
};
template <int G>
__device__ __forceinline__ Share share(int H) {
  constexpr int GPB = block_of(G) / G;
  Share q;
  const int g = threadIdx.x / G, HB = H < GPB ? H : GPB;
  q.K = GPB / HB;
  q.kk = g / HB;
  q.head = blockIdx.y * HB + g % HB;
  q.active = q.kk < q.K && q.head < H;
  return q;
}

// kE values as pairs, for the instructions that work on two at once
struct Row {
  Pair p[kE / 2];
  __device__ __forceinline__ void set(const float *f) {
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) p[i] = pair(f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ void get(float *f) const {
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) split(p[i], f[2 * i], f[2 * i + 1]);
  }
};
__device__ __forceinline__ Pair both(float a) { return pair(a, a); }
__device__ __forceinline__ float total(Pair p) {
  float a, b;
  split(p, a, b);
  return a + b;
}

// sum / d, rounded once (inv = 1 / d): a row of one value over and over, whose
// sum is exact, has exactly that mean.  sum * inv alone is a step off for one
// in eight of such rows, and 1 / sqrt(eps) makes 0.3 of it where the value is
// 16000 (1000 channels).
__device__ __forceinline__ float mean_of(float sum, float inv, float d) {
  const float m = sum * inv;
  return fmaf(fmaf(-d, m, sum), inv, m);
}

// How rows are read and written.
enum Access {
  kAligned,   // 16-byte vectors, rows start on 16-byte boundaries
  kShifted,   // 16-byte vectors; a row starts within one and ends within one
  kScalar     // one element at a time
};
template <typename T, int A>
constexpr int width() { return A == kScalar ? 1 : 16 / (int)sizeof(T); }

// The rows of NT tensors (x; x and dy) on their way to a group of G threads,
// thread l of which has every G-th vector from l on.
//
// A group walks over tokens; the next two tokens' vectors (one where two
// would not fit) are sent to each thread's own slots of shared memory
// ([slot][thread], nobody else reads them) while one token is computed.
// 2-byte elements cannot be sent so; they are loaded where they are used.
//
// kShifted: a row's first element stands at `shift` in its first vector.  A
// group's tokens are a multiple of V apart, so `shift`, and with it which
// columns a thread holds, is the same for all of them.
template <typename T, int A, int G, int NT>
struct Rows {
  static constexpr int V = width<T, A>();
  using raw_t = typename Vec<T, V>::type;
  static constexpr int NV = kE / V, B = block_of(G);
  static constexpr bool kAsync = sizeof(raw_t) >= 4;
  static constexpr int kStage = NT * NV * B;
  static constexpr int kAhead =
      2 * kStage * (int)sizeof(raw_t) <= 192 << 10 ? 2 : 1;
  static constexpr int kBytes = kAsync ? kAhead * kStage * (int)sizeof(raw_t)
                                       : 0;
  raw_t *slots;
  const T *src[NT];       // at the thread's first vector of token 0
  long long ld[NT];       // elements from one token to the next
  const T *end[NT];       // the tensor's end (kShifted)
  int n;                  // vectors of the row that are this thread's
  int shift;
  unsigned valid;         // which of its kE elements are (kShifted)
  int ntok;

  __device__ __forceinline__ void start(char *sm, const Share &q, int d,
                                        int ntok_, long long at) {
    slots = reinterpret_cast<raw_t *>(sm) + threadIdx.x;
    ntok = ntok_;
    const int l = threadIdx.x % G;
    shift = A == kShifted ? rows::shift(at, V) : 0;
    const int nv = q.active ? rows::vectors(shift, d, V) : 0;
    n = nv <= l ? 0 : min((nv - l + G - 1) / G, NV);
    if constexpr (A == kShifted) {
      valid = 0;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int c = column(e);
        if (q.active && c >= 0 && c < d) valid |= 1u << e;
      }
    }
  }
  __device__ __forceinline__ bool has(int e) const {
    return A == kShifted ? valid >> e & 1 : mine(e / V);
  }
  // the column of the thread's element e
  __device__ __forceinline__ int column(int e) const {
    return ((int)threadIdx.x % G + e / V * G) * V + e % V - shift;
  }
  // tensor i: `p` at column 0 of the group's head, token 0
  __device__ __forceinline__ void tensor(int i, const T *p, long long ld_,
                                         const T *end_) {
    src[i] = p + column(0);
    ld[i] = ld_;
    end[i] = end_;
  }
  __device__ __forceinline__ bool mine(int j) const { return j < n; }
  __device__ __forceinline__ const T *vec(int i, long long tok, int j) const {
    return src[i] + tok * ld[i] + j * G * V;
  }
  // END: the tensor may end within one of the token's vectors
  template <bool END>
  __device__ __forceinline__ void send_all(int stage, long long tok) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const T *p = vec(i, tok, j);
        int bytes = tok < ntok && mine(j) ? (int)sizeof(raw_t) : 0;
        if (END && bytes)
          bytes = rows::vector_bytes(end[i] - p, V, (int)sizeof(T));
        copy_async<sizeof(raw_t)>(slots + stage * kStage + (i * NV + j) * B, p,
                                  bytes);
      }
  }
  __device__ __forceinline__ void send(int stage, long long tok) {
    if constexpr (kAsync) {
      if (A == kShifted && rows::may_end(tok, ntok, V))
        send_all<true>(stage, tok);
      else
        send_all<false>(stage, tok);
      copies_sent();
    }
  }
  __device__ __forceinline__ void take(int stage, long long tok,
                                       Row (&r)[NT]) {
    if constexpr (kAsync) copies_landed_but<kAhead - 1>();
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float f[kE];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        raw_t v{};
        if constexpr (kAsync)
          v = slots[stage * kStage + (i * NV + j) * B];
        else if (tok < ntok && mine(j))
          v = load(reinterpret_cast<const raw_t *>(vec(i, tok, j)));
        unpack(v, f + j * V);
      }
      r[i].set(f);
      if (A == kShifted) mask(r[i]);      // (the neighbours' elements)
    }
  }
  // sets to 0 what is not of this row
  __device__ __forceinline__ void mask(Row &r) const {
    if (A == kShifted ? valid == (1u << kE) - 1 : n == NV) return;
    float f[kE];
    r.get(f);
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (!has(e)) f[e] = 0.f;
    r.set(f);
  }
  // `dst` as tensor()'s p
  __device__ __forceinline__ void store_row(T *dst, long long tok,
                                            long long ld_,
                                            const Row &r) const {
    if (tok >= ntok) return;
    float f[kE];
    r.get(f);
    dst += tok * ld_ + column(0);
    constexpr unsigned full = (1u << V) - 1;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (A != kShifted || (valid >> (j * V) & full) == full) {
        if (mine(j)) store<V>(dst + j * G * V, f + j * V);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (has(j * V + v)) store<1>(dst + j * G * V + v, f + j * V + v);
      }
    }
  }
  // a row of parameters, `none` where there are none
  __device__ __forceinline__ void params(const float *p, float none,
                                         Row &r) const {
    float f[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) f[e] = none;
    if (p) {
      if constexpr (A == kAligned) {
#pragma unroll
        for (int e = 0; e < kE; e += 4)
          if (has(e))
            unpack(load(reinterpret_cast<const float4 *>(p + column(e))),
                   f + e);
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e)
          if (has(e)) f[e] = load(p + column(e));
      }
    }
    r.set(f);
  }
  // the thread's part of a row of sums
  __device__ __forceinline__ void sums(float *p, const Row &r) const {
    float f[kE];
    r.get(f);
    if constexpr (A == kAligned) {
#pragma unroll
      for (int e = 0; e < kE; e += 4)
        if (has(e))
          *reinterpret_cast<float4 *>(p + column(e)) =
              make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (has(e)) p[column(e)] = f[e];
    }
  }
};

// ----------------------------------------------------------------- forward

template <typename T, int A, int G>
__global__ void __launch_bounds__(block_of(G), block_of(G) > 256 ? 1 : kFwdBlocks)
    gdr_norm_fwd_kernel(const T *x, long long ldx, const float *w,
                        const float *b, T *out, int ntok, int H, int d,
                        float eps) {
  using RW = Rows<T, A, G, 1>;
  prior_done();
  next_may_start();
  extern __shared__ __align__(128) char slots[];
  __shared__ float2 sm[2][block_of(G) / 32];
  const Share q = share<G>(H);
  const long long pc = (long long)q.head * d, ldo = (long long)H * d;
  const long long stride = (long long)gridDim.x * q.K;
  // (a block's steps are as many for all its groups)
  long long tb = (long long)blockIdx.x * q.K;
  RW rows;
  rows.start(slots, q, d, ntok, (tb + q.kk) * ldx + pc);
  rows.tensor(0, x + pc, ldx, x + ntok * ldo);
  const float df = (float)d, inv = 1.f / df;
  Row wr, br;
#pragma unroll
  for (int i = 0; i < RW::kAhead; ++i) rows.send(i, tb + q.kk + i * stride);
  rows.params(w ? w + pc : nullptr, 1.f, wr);
  rows.params(b ? b + pc : nullptr, 0.f, br);
  for (int it = 0; tb < ntok; tb += stride, it = (it + 1) % RW::kAhead) {
    const long long tok = tb + q.kk;
    Row r[1];
    rows.take(it, tok, r);
    rows.send(it, tok + RW::kAhead * stride);
    Pair s = both(0.f);
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) s = add2(s, r[0].p[i]);
    float mean = total(s), none = 0.f;
    group_sum<G, false>(mean, none, sm[0]);
    mean = mean_of(mean, inv, df);
    Row c;
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) c.p[i] = add2(r[0].p[i], both(-mean));
    rows.mask(c);
    s = both(0.f);
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) s = fma2(c.p[i], c.p[i], s);
    float var = total(s);
    group_sum<G, false>(var, none, sm[1]);
    const Pair rstd = both(1.f / sqrtf(var * inv + eps));
#pragma unroll
    for (int i = 0; i < kE / 2; ++i)
      c.p[i] = fma2(mul2(c.p[i], rstd), wr.p[i], br.p[i]);
    rows.store_row(out + pc, tok, ldo, c);
  }
}

// ---------------------------------------------------------------- backward

// Block (slice, head block).
template <typename T, int A, int G>
__global__ void __launch_bounds__(block_of(G), block_of(G) > 256 ? 1 : kBwdBlocks)
    gdr_norm_bwd_kernel(const T *x, long long ldx, const float *w,
                        const T *dy, T *dx, float *part_w, float *part_b,
                        bool direct, int ntok, int H, int d, float eps) {
  using RW = Rows<T, A, G, 2>;
  constexpr int B = block_of(G);
  prior_done();
  next_may_start();
  extern __shared__ __align__(128) char slots[];
  __shared__ float2 sm[2][B / 32];
  const Share q = share<G>(H);
  const long long pc = (long long)q.head * d, ldo = (long long)H * d;
  const long long stride = (long long)gridDim.x * q.K;
  long long tb = (long long)blockIdx.x * q.K;
  RW rows;
  rows.start(slots, q, d, ntok, (tb + q.kk) * ldx + pc);
  rows.tensor(0, x + pc, ldx, x + ntok * ldo);
  rows.tensor(1, dy + pc, ldo, dy + ntok * ldo);
  const float df = (float)d, inv = 1.f / df;
#pragma unroll
  for (int i = 0; i < RW::kAhead; ++i) rows.send(i, tb + q.kk + i * stride);
  Row wr, aw, ab;
  rows.params(w ? w + pc : nullptr, 1.f, wr);
#pragma unroll
  for (int i = 0; i < kE / 2; ++i) aw.p[i] = ab.p[i] = both(0.f);
  for (int it = 0; tb < ntok; tb += stride, it = (it + 1) % RW::kAhead) {
    const long long tok = tb + q.kk;
    Row r[2];                       // x, dy
    rows.take(it, tok, r);
    rows.send(it, tok + RW::kAhead * stride);
    Pair s = both(0.f), t = both(0.f);
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
      s = add2(s, r[0].p[i]);
      t = fma2(r[1].p[i], wr.p[i], t);
    }
    float mean = total(s), m1 = total(t);
    group_sum<G, true>(mean, m1, sm[0]);
    mean = mean_of(mean, inv, df);
    m1 *= inv;
#pragma unroll
    for (int i = 0; i < kE / 2; ++i)
      r[0].p[i] = add2(r[0].p[i], both(-mean));
    rows.mask(r[0]);
    s = t = both(0.f);
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
      s = fma2(r[0].p[i], r[0].p[i], s);
      t = fma2(mul2(r[1].p[i], wr.p[i]), r[0].p[i], t);
    }
    float var = total(s), m2 = total(t);
    group_sum<G, true>(var, m2, sm[1]);
    // (behind the last token a group computes on zeros, and without eps their
    // rstd would put a NaN into its sums)
    const float rstd = tok < ntok ? 1.f / sqrtf(var * inv + eps) : 0.f;
    m2 *= inv * rstd;
    Row o;
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
      const Pair xh = mul2(r[0].p[i], both(rstd));
      aw.p[i] = fma2(r[1].p[i], xh, aw.p[i]);
      ab.p[i] = add2(ab.p[i], r[1].p[i]);
      o.p[i] = mul2(fma2(xh, both(-m2),
                         fma2(r[1].p[i], wr.p[i], both(-m1))),
                    both(rstd));
    }
    rows.store_row(dx + pc, tok, ldo, o);
  }
  // the block's sums meet in shared memory (its groups of one head in order),
  // then those of the cluster's blocks, each block a part of the columns
  if (!part_w && !part_b) return;
  if (direct) {                         // a partial row per group
    if (!q.active) return;
    const long long o = ((long long)blockIdx.x * q.K + q.kk) * ldo + pc;
    if (part_w) rows.sums(part_w + o, aw);
    if (part_b) rows.sums(part_b + o, ab);
    return;
  }
  copies_landed();
  __syncthreads();
  constexpr int GE = G * kE;                        // room for a group's row
  float *cs = reinterpret_cast<float *>(slots);     // [2][B / G][GE]
  if (q.active) {
    float *mine = cs + threadIdx.x / G * GE;
    rows.sums(mine, aw);
    rows.sums(mine + B * kE, ab);
  }
  cg::cluster_group cl = cg::this_cluster();
  const int nc = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int HB = min(H, B / G), h0 = blockIdx.y * HB;
  const int cols = min(HB, H - h0) * d;
  const long long o = (long long)(blockIdx.x / nc) * ldo + (long long)h0 * d;
  __syncthreads();
  constexpr int V = A == kAligned ? 4 : 1;          // columns at a time
  if (nc == 1 || q.K > 1)
    for (int c = threadIdx.x * V; c < cols; c += B * V) {
      const int hb = HB > 1 ? c / d : 0;
      float *at = cs + hb * GE + (c - hb * d);
      float sum[2][V] = {};
#pragma unroll 4
      for (int k = 0; k < q.K; ++k)
#pragma unroll
        for (int w2 = 0; w2 < 2; ++w2) {
          float f[V];
          const float *from = at + k * HB * GE + w2 * B * kE;
          if constexpr (V == 4) {
            const float4 t = *reinterpret_cast<const float4 *>(from);
            f[0] = t.x, f[1] = t.y, f[2] = t.z, f[3] = t.w;
          } else {
            f[0] = *from;
          }
#pragma unroll
          for (int v = 0; v < V; ++v) sum[w2][v] += f[v];
        }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (nc > 1) {            // (no other thread reads these columns here)
          at[v] = sum[0][v];
          at[v + B * kE] = sum[1][v];
        } else {
          if (part_w) part_w[o + c + v] = sum[0][v];
          if (part_b) part_b[o + c + v] = sum[1][v];
        }
      }
    }
  if (nc == 1) return;
  cl.sync();
  for (int c = rank * B + threadIdx.x; c < cols; c += nc * B) {
    const int hb = HB > 1 ? c / d : 0, at = hb * GE + (c - hb * d);
    float sw = 0.f, sb = 0.f;
    for (int r = 0; r < nc; ++r) {
      const float *rs = cl.map_shared_rank(cs, r);
      sw += rs[at];
      sb += rs[at + B * kE];
    }
    if (part_w) part_w[o + c] = sw;
    if (part_b) part_b[o + c] = sb;
  }
  cl.sync();                // none ends while another reads its sums
}

// dst[c] = the sum over `slices` rows of part[.][c], c < n: 32 columns a
// block, 32 threads a column, always in the same order.  blockIdx.y chooses
// between the weight's and the bias's sums.
__global__ void __launch_bounds__(1024)
    gdr_norm_sum_kernel(const float *part_w, const float *part_b, float *dw,
                        float *db, int n, int slices) {
  __shared__ float sm[32][33];
  prior_done();
  next_may_start();
  const bool bias = blockIdx.y == 1 || !dw;
  const float *part = bias ? part_b : part_w;
  float *dst = bias ? db : dw;
  const int i = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + i;
  float s = 0.f;
  if (c < n) {
#pragma unroll 8
    for (int r = k; r < slices; r += 32) s += part[(long long)r * n + c];
  }
  sm[k][i] = s;
  __syncthreads();
  // one warp per column: lane = share
  s = sm[i][k];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  if (i == 0 && blockIdx.x * 32 + k < n) dst[blockIdx.x * 32 + k] = s;
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
  int access, G;           // how rows are read; threads per row
  int slices;              // blocks side by side over the tokens
  int cluster;             // of which this many add their sums
  int parts;               // partial rows of sums
  bool direct;             // ... one per group of threads, not per block
  int ntok, H, d;
  float eps;
};

// 16-byte vectors where every row starts on a 16-byte boundary, or where all
// tensors are contiguous, so that their rows start alike; else (tokens of x
// apart and unaligned) one element at a time.
int access_of(const NormParams &p, int es) {
  const int v = 16 / es;
  if (p.d % v == 0 && p.ldx % v == 0) return kAligned;
  return p.ldx == (long long)p.H * p.d && p.d + v - 1 <= kMaxDim ? kShifted
                                                                : kScalar;
}
// Threads per row.
int group_of(int d, int access, int es) {
  const int n = access == kShifted ? d + 16 / es - 1 : d;
  int g = 1;
  while (g * kE < n) g *= 2;
  return g;
}
struct Cut {
  int groups, hblocks;   // groups per head, head blocks
};
Cut cut_of(int H, int G) {
  const int gpb = block_of(G) / G;
  const int heads = H < gpb ? H : gpb;
  return {gpb / heads, (H + heads - 1) / heads};
}
// Blocks side by side over the tokens: as many in all as the GPU holds; where
// a group takes more than one token and they have to start alike, a multiple
// of 8.
int slices_of(const NormParams &p, int resident) {
  const Cut c = cut_of(p.H, p.G);
  const int want =
      (kSms * (block_of(p.G) > 256 ? 1 : resident) + c.hblocks - 1) / c.hblocks;
  const int most = (p.ntok + c.groups - 1) / c.groups;
  if (want >= most) return most;
  return p.access == kShifted ? (want > 8 ? want & ~7 : 8) : want;
}
// The backward pass of few tokens: one cluster of up to 8 blocks per head
// block, which ends with the whole sums and saves the second kernel and its
// scratch.  Else blocks on their own: clusters do not fill the GPU (32768
// tokens of 2048 channels, bf16: 124 us with 4 blocks each, 78 without).
void cut_bwd(NormParams *p) {
  const Cut c = cut_of(p->H, p->G);
  const int blocks = (p->ntok + c.groups - 1) / c.groups;
  p->direct = false;
  if (blocks <= 8) {
    p->slices = p->cluster = blocks;
    p->parts = 1;
  } else {
    p->slices = slices_of(*p, kBwdBlocks);
    p->cluster = 1;
    // Few groups leave it all to the second kernel; more add theirs block by
    // block first, for the second kernel's reading grows with its rows (333
    // rows of 1001, fp32, a row of sums per group 7.4 us, per block 12.3;
    // 8192 rows of 16 heads of 128, bf16, 1184 groups, 23.1 and 23.9; 2000
    // unaligned rows of 1001, 1184 groups, 18.6 and 16.5; 5000 rows of 8
    // heads of 64, 2368 groups, 14.8 and 10.7).
    p->direct = (long long)p->slices * c.groups <=
                    (p->access == kAligned ? 1280 : 512) ||
                c.groups == 1;
    p->parts = p->direct ? p->slices * c.groups : p->slices;
  }
}

template <typename T, int A, int G>
cudaError_t launch_fwd(const NormParams &p, cudaStream_t s) {
  auto *k = gdr_norm_fwd_kernel<T, A, G>;
  constexpr int bytes = Rows<T, A, G, 1>::kBytes;
  if constexpr (bytes > 24 << 10) {   // (static shared memory counts too)
    const cudaError_t e = cudaFuncSetAttribute(
        k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  return launch(k, dim3(p.slices, cut_of(p.H, G).hblocks), block_of(G), bytes,
                1, true, s, static_cast<const T *>(p.x), p.ldx, p.w, p.b,
                static_cast<T *>(p.out), p.ntok, p.H, p.d, p.eps);
}
template <typename T, int A, int G>
cudaError_t launch_bwd(const NormParams &p, cudaStream_t s) {
  auto *k = gdr_norm_bwd_kernel<T, A, G>;
  constexpr int slots = Rows<T, A, G, 2>::kBytes;
  constexpr int sums = 2 * block_of(G) * kE * (int)sizeof(float);
  constexpr int bytes = slots > sums ? slots : sums;
  if constexpr (bytes > 24 << 10) {   // (static shared memory counts too)
    const cudaError_t e = cudaFuncSetAttribute(
        k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  return launch(k, dim3(p.slices, cut_of(p.H, G).hblocks), block_of(G), bytes,
                p.cluster, true, s, static_cast<const T *>(p.x), p.ldx, p.w,
                static_cast<const T *>(p.dy), static_cast<T *>(p.out),
                p.part_w, p.part_b, p.direct, p.ntok, p.H, p.d, p.eps);
}

template <bool BWD, typename T, int A, int G>
cudaError_t launch(const NormParams &p, cudaStream_t s) {
  if constexpr (BWD)
    return launch_bwd<T, A, G>(p, s);
  else
    return launch_fwd<T, A, G>(p, s);
}
template <bool BWD, typename T, int A>
cudaError_t run_g(const NormParams &p, cudaStream_t s) {
  switch (p.G) {
    case 1: return launch<BWD, T, A, 1>(p, s);
    case 2: return launch<BWD, T, A, 2>(p, s);
    case 4: return launch<BWD, T, A, 4>(p, s);
    case 8: return launch<BWD, T, A, 8>(p, s);
    case 16: return launch<BWD, T, A, 16>(p, s);
    case 32: return launch<BWD, T, A, 32>(p, s);
    case 64: return launch<BWD, T, A, 64>(p, s);
    case 128: return launch<BWD, T, A, 128>(p, s);
    case 256: return launch<BWD, T, A, 256>(p, s);
    case 512: return launch<BWD, T, A, 512>(p, s);
    default: return launch<BWD, T, A, 1024>(p, s);
  }
}
template <bool BWD, typename T>
cudaError_t run_a(const NormParams &p, cudaStream_t s) {
  switch (p.access) {
    case kAligned: return run_g<BWD, T, kAligned>(p, s);
    case kShifted: return run_g<BWD, T, kShifted>(p, s);
    default: return run_g<BWD, T, kScalar>(p, s);
  }
}
template <bool BWD>
cudaError_t run(const NormParams &p, gdr_dtype dtype, cudaStream_t s) {
  return dtype == GDR_FP32 ? run_a<BWD, float>(p, s)
                           : run_a<BWD, __nv_bfloat16>(p, s);
}
void set_access(NormParams *p, gdr_dtype dtype) {
  const int es = dtype == GDR_FP32 ? 4 : 2;
  p->access = access_of(*p, es);
  p->G = group_of(p->d, p->access, es);
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
  set_access(&p, dtype);
  // (groups within a warp or two need no third block to hide their meetings,
  // and two disturb one another less: 32768 x 16 heads of 128, bf16, 45.7 us
  // against 49.6; 32768 rows of 2048, whose groups are four warps, 45.8
  // against 49.1 the other way round)
  p.slices = slices_of(p, p.G <= 64 && p.access == kAligned ? 2 : kFwdBlocks);
  const cudaError_t e = run<false>(p, dtype, stream);
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
  set_access(&p, dtype);
  cut_bwd(&p);
  // (one part: the sums are whole)
  const size_t one = (size_t)(4 * hd * p.parts + 255) & ~(size_t)255;
  const int narr = (d_weight ? 1 : 0) + (d_bias ? 1 : 0);
  void *ws = nullptr;
  p.part_w = d_weight;
  p.part_b = d_bias;
  if (narr && p.parts > 1) {
    st = scratch_get(&ws, one * narr, stream);
    if (st != GDR_OK) return st;
    char *at = static_cast<char *>(ws);
    if (d_weight) {
      p.part_w = reinterpret_cast<float *>(at);
      at += one;
    }
    if (d_bias) p.part_b = reinterpret_cast<float *>(at);
  }
  cudaError_t e = run<true>(p, dtype, stream);
  if (e == cudaSuccess && ws) {
    // (its launch overlaps the end of the first kernel)
    e = launch(gdr_norm_sum_kernel, dim3((unsigned)((hd + 31) / 32), narr),
               1024, 0, 1, true, stream, p.part_w, p.part_b, d_weight, d_bias,
               (int)hd, p.parts);
  }
  const cudaError_t f = ws ? scratch_put(ws, stream) : cudaSuccess;
  return (e == cudaSuccess && f == cudaSuccess) ? GDR_OK : GDR_ERR_CUDA;
}
