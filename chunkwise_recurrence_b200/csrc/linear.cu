// Gated linear recurrence of libgdr: the memory of the delta rule without the
// erase, with a vector state -- forward pass, single-token step, gradients.
//
// Per sequence and channel (tokens t in order, alpha_t = e^{log_alpha_t}):
//   h_t = alpha_t h_{t-1} + x_t,   out_t = h_t
// and backwards, with c_t = alpha_t G_t handed to the token before:
//   G_t = dout_t + c_{t+1},   dx_t = G_t,   dlog_alpha_t = G_t alpha_t h_{t-1}.
// Both are scans of affine maps y -> alpha y + b, which compose:
//   (alpha', b') o (alpha, b) = (alpha' alpha, alpha' b + b').
//
// One pass over the data.  A warp holds a tile of 32 tokens x 32 channels in
// registers: a thread has V consecutive channels (one 16-byte load of fp32)
// of R tokens in a row (R V = 32 values), scans them alone, and the
// warp's 32 / lanes-per-row runs are joined by shuffles.  Eight warps stack
// their tiles in time (256 tokens), and a cluster of up to 8 CTAs stacks
// theirs; the joins travel through shared and distributed shared memory, so
// nothing but x, log_alpha and the results touches HBM and no scratch, flag
// or spin-wait is needed.  Each thread then runs its tokens a second time
// from the state it now knows.
//
// Decays near 1 are held as alpha - 1 (decay_factor): rounding alpha itself
// to fp32 puts a systematic 2^-25 into every step, which a memory of 10^4
// tokens turns into 3e-4.  Composed decays are sums of log_alpha until they
// are applied, so that log_alpha = -inf clears the state exactly.

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstring>

#include "gdr_internal.h"

namespace gdr {
namespace {

namespace cg = cooperative_groups;

constexpr int kTok = GDR_LINEAR_CHUNK;   // tokens of a warp's tile
constexpr int kCh = 32;                  // channels of a warp's tile
constexpr int kWarps = 8;
constexpr int kMaxCluster = 8;
static_assert(kTok == 32, "a warp's tile is 32 tokens");

struct LinParams {
  const void *x;
  const float *la, *s0;
  void *out;        // forward; nullptr: only states and sT are written
  float *sT;
  float *states;    // chunk states: written (forward), read (backward)
  const void *dout;
  const float *dsT;
  void *dx;
  float *dla;       // channel gate, or scalar gate with one tile per head
  float *part;      // scalar gate: per channel tile [nct][ntok][H]
  float *ds0;
  const int32_t *cu;
  long long ldx;
  int T, ntok, nseq, H, d, D;
  int tiles;        // channel tiles in all
  int nct;          // channel tiles per head; 0: tiles cut H * d as one row
  int chains;       // tiles * nseq
};

// ---------------------------------------------------------------- elements

template <typename T, int V>
struct Raw;
template <>
struct Raw<float, 4> { using type = float4; };
template <>
struct Raw<float, 1> { using type = float; };
template <>
struct Raw<__nv_bfloat16, 4> { using type = uint2; };
template <>
struct Raw<__nv_bfloat16, 1> { using type = unsigned short; };

__device__ __forceinline__ void unpack(const float4 &r, float (&f)[4]) {
  f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w;
}
__device__ __forceinline__ void unpack(const float &r, float (&f)[1]) {
  f[0] = r;
}
__device__ __forceinline__ void unpack(const uint2 &r, float (&f)[4]) {
  f[0] = __uint_as_float(r.x << 16), f[1] = __uint_as_float(r.x & 0xffff0000u);
  f[2] = __uint_as_float(r.y << 16), f[3] = __uint_as_float(r.y & 0xffff0000u);
}
__device__ __forceinline__ void unpack(const unsigned short &r,
                                       float (&f)[1]) {
  f[0] = __uint_as_float((unsigned)r << 16);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ void store(float *p, const float (&f)[4]) {
  *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store(float *p, const float (&f)[1]) {
  *p = f[0];
}
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&f)[4]) {
  *reinterpret_cast<uint2 *>(p) =
      make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
}
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&f)[1]) {
  *p = __float2bfloat16_rn(f[0]);
}

// ------------------------------------------------------------------ decays

// The decay e^s in the form the state is multiplied by: for -1/8 < s <= 0
// (sign bit set, also at s = 0) the value is e^s - 1 to its own relative
// precision, by its Taylor series (the first term left out is under 5e-8 of
// the sum); elsewhere (sign bit clear) it is e^s.
__device__ __forceinline__ float decay_factor(float s) {
  float p = fmaf(s, 1.f / 120.f, 1.f / 24.f);
  p = fmaf(s, p, 1.f / 6.f);
  p = fmaf(s, p, 0.5f);
  p = fmaf(s, p, 1.f);
  const float near1 = -fabsf(s) * p;
  const float far1 = __expf(s);
  return (s > -0.125f && s <= 0.f) ? near1 : far1;
}
// e^s h, from decay_factor(s)
__device__ __forceinline__ float decay(float m, float h) {
  return fmaf(m, h, __float_as_int(m) < 0 ? h : 0.f);
}

// Tokens [*a, *a + *len) of sequence n.  Offsets that do not lie in order
// within [0, T] are pulled there: whatever they hold, no token outside the
// tensors is touched.
__device__ __forceinline__ void seq_range(const LinParams &p, int n, int *a,
                                          int *len) {
  if (p.cu) {
    const int lo = min(max(p.cu[n], 0), p.T);
    const int hi = min(max(p.cu[n + 1], lo), p.T);
    *a = lo;
    *len = hi - lo;
  } else {
    *a = n * p.T;
    *len = p.T;
  }
}

// What a warp's threads hold of one tile, and the joins inside the warp.
template <int V, int GATE>
struct Tile {
  static constexpr int kLanes = kCh / V;         // threads per token
  static constexpr int kSubs = 32 / kLanes;      // token runs per warp
  static constexpr int R = kTok / kSubs;         // tokens per run
  static constexpr int GV = GATE == GDR_GATE_CHANNEL ? V : 1;
};

template <int V, int GV>
struct Map {       // y -> e^s y + b per channel
  float s[GV], b[V];
};

// this = this o other (other is applied first)
template <int V, int GV, int GATE>
__device__ __forceinline__ void after(Map<V, GV> &f, const Map<V, GV> &g) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (GATE == GDR_GATE_NONE) {
      f.b[v] += g.b[v];
    } else {
      f.b[v] += decay(decay_factor(f.s[GV == V ? v : 0]), g.b[v]);
    }
  }
  if constexpr (GATE != GDR_GATE_NONE)
#pragma unroll
    for (int v = 0; v < GV; ++v) f.s[v] += g.s[v];
}

// Scan of the warp's runs, in time (REV = false) or against it: on return
// `f` maps over this run and all before it (in scan order), `ex` over those
// before it alone.
template <int V, int GV, int GATE, bool REV>
__device__ __forceinline__ void warp_scan(Map<V, GV> &f, Map<V, GV> &ex) {
  constexpr int L = kCh / V;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = L; off < 32; off <<= 1) {
    Map<V, GV> g;
#pragma unroll
    for (int v = 0; v < V; ++v)
      g.b[v] = REV ? __shfl_down_sync(~0u, f.b[v], off)
                   : __shfl_up_sync(~0u, f.b[v], off);
#pragma unroll
    for (int v = 0; v < GV; ++v)
      g.s[v] = REV ? __shfl_down_sync(~0u, f.s[v], off)
                   : __shfl_up_sync(~0u, f.s[v], off);
    const bool has = REV ? lane + off < 32 : lane >= off;
    if (has) after<V, GV, GATE>(f, g);
  }
  if constexpr (L < 32) {
    const bool first = REV ? lane + L >= 32 : lane < L;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float b = REV ? __shfl_down_sync(~0u, f.b[v], L)
                          : __shfl_up_sync(~0u, f.b[v], L);
      ex.b[v] = first ? 0.f : b;
    }
#pragma unroll
    for (int v = 0; v < GV; ++v) {
      const float s = REV ? __shfl_down_sync(~0u, f.s[v], L)
                          : __shfl_up_sync(~0u, f.s[v], L);
      ex.s[v] = first ? 0.f : s;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) ex.b[v] = 0.f;
#pragma unroll
    for (int v = 0; v < GV; ++v) ex.s[v] = 0.f;
  }
}

// The joins across the warps of a CTA and the CTAs of a cluster.  Thread
// (warp w, lane) looks after channel `lane` of the tile: it leaves with the
// value that enters warp w's tile, and `carry` moves on past all tiles of
// this step.  One barrier per step: the buffers alternate.
struct Joint {
  float2 warp[2][kWarps][kCh];
  float2 rank[2][kMaxCluster][kCh];
};

template <int GATE>
__device__ __forceinline__ float apply(float2 m, float y) {
  if constexpr (GATE == GDR_GATE_NONE) return y + m.y;
  return decay(decay_factor(m.x), y) + m.y;
}

// `edge`: this thread belongs to the run that holds the whole warp's map
// (the last in scan order).
template <int V, int GV, int GATE, bool REV>
__device__ __forceinline__ float block_join(Joint &jt, int buf,
                                            const Map<V, GV> &f, bool edge,
                                            int nc, int rank, float &carry) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = lane % (kCh / V);
  if (edge) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      jt.warp[buf][w][c * V + v] =
          make_float2(GATE == GDR_GATE_NONE ? 0.f : f.s[GV == V ? v : 0],
                      f.b[v]);
  }
  __syncthreads();
  float in = 0.f;
  if (nc == 1) {
    float y = carry;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int j = REV ? kWarps - 1 - i : i;
      if (j == w) in = y;
      y = apply<GATE>(jt.warp[buf][j][lane], y);
    }
    carry = y;
    return in;
  }
  float2 pre = make_float2(0.f, 0.f);   // the warps before this one
  const int nbefore = REV ? kWarps - 1 - w : w;
  for (int i = 0; i < nbefore; ++i) {
    const float2 m = jt.warp[buf][REV ? kWarps - 1 - i : i][lane];
    pre.y = apply<GATE>(m, pre.y);
    pre.x += m.x;
  }
  if (nbefore == kWarps - 1) {
    const float2 m = jt.warp[buf][w][lane];
    const float2 tot = make_float2(pre.x + m.x, apply<GATE>(m, pre.y));
    cg::cluster_group cl = cg::this_cluster();
    for (int r = 0; r < nc; ++r)
      cl.map_shared_rank(&jt.rank[buf][rank][lane], r)[0] = tot;
  }
  cg::this_cluster().sync();
  float y = carry;
  for (int r = 0; r < nc; ++r) {
    if (r == rank) in = y;
    y = apply<GATE>(jt.rank[buf][r][lane], y);
  }
  carry = y;
  return apply<GATE>(pre, in);
}

// The same for a warp on its own: lane's channel of the warp's map.
template <int V, int GV, int GATE, bool REV>
__device__ __forceinline__ float warp_join(const Map<V, GV> &f,
                                           float &carry) {
  constexpr int L = kCh / V;
  const int lane = threadIdx.x & 31;
  const int src = (REV ? 0 : 32 - L) + lane / V;
  float2 m = make_float2(0.f, 0.f);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float b = __shfl_sync(~0u, f.b[v], src);
    if (lane % V == v) m.y = b;
  }
  if constexpr (GATE != GDR_GATE_NONE) {
#pragma unroll
    for (int v = 0; v < GV; ++v) {
      const float s = __shfl_sync(~0u, f.s[v], src);
      if (GV == 1 || lane % V == v) m.x = s;
    }
  }
  const float in = carry;
  carry = apply<GATE>(m, carry);
  return in;
}

// A thread's place: its chain (sequence and channel tile), its channels.
struct Place {
  int n;            // sequence
  int ch;           // first of the thread's V channels
  int chl;          // channel `lane` of the tile
  bool has, hasl;   // whether those exist
  int head, ct;     // the tile's head and tile within it (nct > 0)
};
template <int V>
__device__ __forceinline__ Place place(const LinParams &p, int chain) {
  Place q;
  const int lane = threadIdx.x & 31;
  const int tile = chain % p.tiles;
  q.n = chain / p.tiles;
  int base, end;
  if (p.nct) {
    q.head = tile / p.nct;
    q.ct = tile - q.head * p.nct;
    base = q.head * p.d + q.ct * kCh;
    end = (q.head + 1) * p.d;
  } else {
    q.head = q.ct = 0;
    base = tile * kCh;
    end = p.D;
  }
  q.ch = base + (lane % (kCh / V)) * V;
  q.chl = base + lane;
  q.has = q.ch < end;
  q.hasl = q.chl < end;
  return q;
}

// ----------------------------------------------------------------- forward

// WPC = 8: a cluster of CTAs per chain, stacked in time; WPC = 1: a warp per
// chain.
template <typename T, int V, int GATE, int WPC>
__global__ void __launch_bounds__(kWarps * 32, 3)
    gdr_linear_fwd_kernel(const LinParams p) {
  using TL = Tile<V, GATE>;
  constexpr int R = TL::R, GV = TL::GV, L = TL::kLanes;
  using raw_t = typename Raw<T, V>::type;
  __shared__ Joint jt;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / L;
  int nc = 1, rank = 0, chain;
  if constexpr (WPC == 1) {
    chain = blockIdx.x * kWarps + w;
    if (chain >= p.chains) return;
  } else {
    nc = (int)cg::this_cluster().num_blocks();
    rank = (int)cg::this_cluster().block_rank();
    chain = blockIdx.x / nc;
    // no CTA writes into another's shared memory before that one has begun
    if (nc > 1) cg::this_cluster().sync();
  }
  const Place q = place<V>(p, chain);
  int tok0, len;
  seq_range(p, q.n, &tok0, &len);
  const long long so = (long long)q.n * p.D + q.chl;
  float carry = (p.s0 && q.hasl) ? p.s0[so] : 0.f;
  const int span = WPC == 1 ? kTok : kWarps * kTok * nc;
  const int off = WPC == 1 ? 0 : (rank * kWarps + w) * kTok;
  const int steps = (len + span - 1) / span;
  const int gcol = GATE == GDR_GATE_SCALAR ? q.ch / p.d : q.ch;
  const int gld = GATE == GDR_GATE_SCALAR ? p.H : p.D;

  for (int k = 0; k < steps; ++k) {
    const int t0 = k * span + off;       // the warp's first token
    const int t = t0 + sub * R;          // the thread's
    const long long tok = (long long)tok0 + t;
    raw_t xr[R];
    float m[R][GV];
    const T *xp = static_cast<const T *>(p.x) + tok * p.ldx + q.ch;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      xr[r] = raw_t{};
      if (q.has && t + r < len)
        xr[r] = __ldg(reinterpret_cast<const raw_t *>(xp + r * p.ldx));
    }
    if constexpr (GATE != GDR_GATE_NONE) {
      const float *gp = p.la + tok * gld + gcol;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        typename Raw<float, GV>::type g{};
        if (q.has && t + r < len)
          g = __ldg(reinterpret_cast<const typename Raw<float, GV>::type *>(
              gp + (long long)r * gld));
        unpack(g, m[r]);
      }
    }
    // the run on its own
    Map<V, GV> f, ex;
#pragma unroll
    for (int v = 0; v < V; ++v) f.b[v] = 0.f;
#pragma unroll
    for (int v = 0; v < GV; ++v) f.s[v] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float x[V];
      unpack(xr[r], x);
      if constexpr (GATE != GDR_GATE_NONE) {
#pragma unroll
        for (int v = 0; v < GV; ++v) {
          f.s[v] += m[r][v];
          m[r][v] = decay_factor(m[r][v]);
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
        f.b[v] = (GATE == GDR_GATE_NONE
                      ? f.b[v]
                      : decay(m[r][GV == V ? v : 0], f.b[v])) + x[v];
    }
    warp_scan<V, GV, GATE, false>(f, ex);
    float hin;
    if constexpr (WPC == 1)
      hin = warp_join<V, GV, GATE, false>(f, carry);
    else
      hin = block_join<V, GV, GATE, false>(jt, k & 1, f, sub == TL::kSubs - 1,
                                           nc, rank, carry);
    if (p.states && q.hasl && t0 < len) {
      const long long slot = (long long)(tok0 / kTok) + q.n + t0 / kTok;
      p.states[slot * p.D + q.chl] = hin;
    }
    if (p.out) {
      float h[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float y = __shfl_sync(~0u, hin, (lane % L) * V + v);
        h[v] = apply<GATE>(make_float2(ex.s[GV == V ? v : 0], ex.b[v]), y);
      }
      T *op = static_cast<T *>(p.out) + tok * p.D + q.ch;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x[V];
        unpack(xr[r], x);
#pragma unroll
        for (int v = 0; v < V; ++v)
          h[v] = (GATE == GDR_GATE_NONE ? h[v]
                                        : decay(m[r][GV == V ? v : 0], h[v])) +
                 x[v];
        if (q.has && t + r < len) store(op + (long long)r * p.D, h);
      }
    }
  }
  if (p.sT && q.hasl && (WPC == 1 || (rank == 0 && w == 0))) p.sT[so] = carry;
}

// ---------------------------------------------------------------- backward

// From the last token to the first.  Every warp has its tile's first state
// (the chunk states), so h is run forward inside the warp, leaving
// alpha_t h_{t-1} in registers; then c runs backward through the same joins
// as the forward pass.
template <typename T, int V, int GATE, int WPC>
__global__ void __launch_bounds__(kWarps * 32, 2)
    gdr_linear_bwd_kernel(const LinParams p) {
  using TL = Tile<V, GATE>;
  constexpr int R = TL::R, GV = TL::GV, L = TL::kLanes;
  using raw_t = typename Raw<T, V>::type;
  __shared__ Joint jt;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / L;
  int nc = 1, rank = 0, chain;
  if constexpr (WPC == 1) {
    chain = blockIdx.x * kWarps + w;
    if (chain >= p.chains) return;
  } else {
    nc = (int)cg::this_cluster().num_blocks();
    rank = (int)cg::this_cluster().block_rank();
    chain = blockIdx.x / nc;
    // no CTA writes into another's shared memory before that one has begun
    if (nc > 1) cg::this_cluster().sync();
  }
  const Place q = place<V>(p, chain);
  int tok0, len;
  seq_range(p, q.n, &tok0, &len);
  const long long so = (long long)q.n * p.D + q.chl;
  float carry = (p.dsT && q.hasl) ? p.dsT[so] : 0.f;
  const int block = WPC == 1 ? kTok : kWarps * kTok;
  const int nblk = (len + block - 1) / block;
  const int steps = (nblk + nc - 1) / nc;
  const int gcol = GATE == GDR_GATE_SCALAR ? q.ch / p.d : q.ch;
  const int gld = GATE == GDR_GATE_SCALAR ? p.H : p.D;

  for (int k = 0; k < steps; ++k) {
    const int blk = nblk - 1 - (k * nc + rank);
    // (a block before the first token: nothing of it exists)
    const int end = blk < 0 ? INT_MIN : len;
    const int t0 = blk * block + (WPC == 1 ? 0 : w * kTok);
    const int t = t0 + sub * R;
    const long long tok = (long long)tok0 + t;
    raw_t xr[R], dr[R];
    float m[R][GV];
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.f;
    if constexpr (GATE != GDR_GATE_NONE) {
      const T *xp = static_cast<const T *>(p.x) + tok * p.ldx + q.ch;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        xr[r] = raw_t{};
        if (q.has && t + r < end)
          xr[r] = __ldg(reinterpret_cast<const raw_t *>(xp + r * p.ldx));
      }
      const float *gp = p.la + tok * gld + gcol;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        typename Raw<float, GV>::type g{};
        if (q.has && t + r < end)
          g = __ldg(reinterpret_cast<const typename Raw<float, GV>::type *>(
              gp + (long long)r * gld));
        unpack(g, m[r]);
      }
      if (q.has && t0 < end) {
        const long long slot = (long long)(tok0 / kTok) + q.n + t0 / kTok;
        unpack(__ldg(reinterpret_cast<const typename Raw<float, V>::type *>(
                   p.states + slot * p.D + q.ch)),
               h);
      }
    }
    const T *dp = static_cast<const T *>(p.dout) + tok * p.D + q.ch;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      dr[r] = raw_t{};
      if (q.has && t + r < end)
        dr[r] = __ldg(
            reinterpret_cast<const raw_t *>(dp + (long long)r * p.D));
    }
    Map<V, GV> f, ex;
#pragma unroll
    for (int v = 0; v < V; ++v) f.b[v] = 0.f;
#pragma unroll
    for (int v = 0; v < GV; ++v) f.s[v] = 0.f;
    float ah[R][V];                      // alpha_t h_{t-1}
    if constexpr (GATE != GDR_GATE_NONE) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x[V];
        unpack(xr[r], x);
#pragma unroll
        for (int v = 0; v < GV; ++v) {
          f.s[v] += m[r][v];
          m[r][v] = decay_factor(m[r][v]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
          f.b[v] = decay(m[r][GV == V ? v : 0], f.b[v]) + x[v];
      }
      float ssum[GV];
#pragma unroll
      for (int v = 0; v < GV; ++v) ssum[v] = f.s[v];
      warp_scan<V, GV, GATE, false>(f, ex);
#pragma unroll
      for (int v = 0; v < V; ++v)
        h[v] = apply<GATE>(make_float2(ex.s[GV == V ? v : 0], ex.b[v]), h[v]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x[V];
        unpack(xr[r], x);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          ah[r][v] = decay(m[r][GV == V ? v : 0], h[v]);
          h[v] = ah[r][v] + x[v];
        }
      }
#pragma unroll
      for (int v = 0; v < GV; ++v) f.s[v] = ssum[v];
#pragma unroll
      for (int v = 0; v < V; ++v) f.b[v] = 0.f;
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      float g[V];
      unpack(dr[r], g);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        g[v] += f.b[v];
        f.b[v] = GATE == GDR_GATE_NONE ? g[v]
                                       : decay(m[r][GV == V ? v : 0], g[v]);
      }
    }
    warp_scan<V, GV, GATE, true>(f, ex);
    float cin;
    if constexpr (WPC == 1)
      cin = warp_join<V, GV, GATE, true>(f, carry);
    else
      cin = block_join<V, GV, GATE, true>(jt, k & 1, f, sub == 0, nc, rank,
                                          carry);
    float c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float y = __shfl_sync(~0u, cin, (lane % L) * V + v);
      c[v] = apply<GATE>(make_float2(ex.s[GV == V ? v : 0], ex.b[v]), y);
    }
    T *xo = static_cast<T *>(p.dx) + tok * p.D + q.ch;
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      float g[V];
      unpack(dr[r], g);
#pragma unroll
      for (int v = 0; v < V; ++v) g[v] += c[v];
      const bool live = q.has && t + r < end;
      if (live) store(xo + (long long)r * p.D, g);
      if constexpr (GATE == GDR_GATE_CHANNEL) {
        float dl[V];
#pragma unroll
        for (int v = 0; v < V; ++v) dl[v] = g[v] * ah[r][v];
        if (live) store(p.dla + (tok + r) * p.D + q.ch, dl);
      }
      if constexpr (GATE == GDR_GATE_SCALAR) {
        // the head's share of this tile, added in a fixed order
        float dl = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) dl = fmaf(g[v], ah[r][v], dl);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1)
          dl += __shfl_xor_sync(~0u, dl, o);
        if (live && lane % L == 0) {
          if (p.nct == 1)
            p.dla[(tok + r) * p.H + q.head] = dl;
          else
            p.part[((long long)q.ct * p.ntok + tok + r) * p.H + q.head] = dl;
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
        c[v] = GATE == GDR_GATE_NONE ? g[v]
                                     : decay(m[r][GV == V ? v : 0], g[v]);
    }
  }
  if (p.ds0 && q.hasl && (WPC == 1 || (rank == 0 && w == 0)))
    p.ds0[so] = carry;
}

// Scalar gate, heads of more than one channel tile: the tiles' shares of
// dlog_alpha, added in order.
__global__ void __launch_bounds__(256)
    gdr_linear_dla_kernel(const float *part, float *dla, long long n,
                          int nct) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float s = 0.f;
  for (int c = 0; c < nct; ++c) s += part[c * n + i];
  dla[i] = s;
}

// -------------------------------------------------------------------- step

template <typename T, int V, int GATE>
__global__ void __launch_bounds__(128)
    gdr_linear_step_kernel(const T *x, const float *la, const float *sin,
                           float *sout, T *out, long long ldx, int N, int H,
                           int d) {
  const int D = H * d, nv = D / V;
  const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
  if (i >= (long long)N * nv) return;
  const long long n = i / nv;
  const int ch = (int)(i - n * nv) * V;
  float xf[V], h[V];
  using raw_t = typename Raw<T, V>::type;
  using f_t = typename Raw<float, V>::type;
  unpack(__ldg(reinterpret_cast<const raw_t *>(x + n * ldx + ch)), xf);
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = 0.f;
  if (sin) unpack(*reinterpret_cast<const f_t *>(sin + n * D + ch), h);
  if constexpr (GATE == GDR_GATE_CHANNEL) {
    float g[V];
    unpack(__ldg(reinterpret_cast<const f_t *>(la + n * D + ch)), g);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = decay(decay_factor(g[v]), h[v]);
  } else if constexpr (GATE == GDR_GATE_SCALAR) {
    const float m = decay_factor(__ldg(la + n * H + ch / d));
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = decay(m, h[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] += xf[v];
  store(out + n * D + ch, h);
  store(sout + n * D + ch, h);
}

// ---------------------------------------------------------------- launches

// A chain is run by a warp where there are chains enough to fill the GPU so
// (or the sequences are too short to cut), else by a cluster of CTAs.
constexpr int kSms = 148;

int cluster_size(const LinParams &p, int resident) {
  const long long avg = p.ntok / (p.nseq > 0 ? p.nseq : 1);
  const long long blocks = (avg + kWarps * kTok - 1) / (kWarps * kTok);
  int nc = 1;
  while (nc * 2 <= kMaxCluster && nc * 2 <= blocks &&
         (long long)p.chains * nc * 2 <= (long long)kSms * resident)
    nc *= 2;
  return nc;
}

bool warp_chains(const LinParams &p) {
  const long long avg = p.ntok / (p.nseq > 0 ? p.nseq : 1);
  return avg <= 2 * kTok || p.chains >= kSms * 3 * kWarps;
}

template <typename K>
cudaError_t launch_chains(K kernel, const LinParams &p, int wpc, int nc,
                          cudaStream_t s) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(wpc == 1 ? (p.chains + kWarps - 1) / kWarps
                              : p.chains * nc);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = wpc == 1 ? 1 : nc;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T, int V, int GATE>
cudaError_t run_fwd(const LinParams &p, cudaStream_t s) {
  if (warp_chains(p))
    return launch_chains(gdr_linear_fwd_kernel<T, V, GATE, 1>, p, 1, 1, s);
  return launch_chains(gdr_linear_fwd_kernel<T, V, GATE, kWarps>, p, kWarps,
                       cluster_size(p, 3), s);
}
template <typename T, int V, int GATE>
cudaError_t run_bwd(const LinParams &p, cudaStream_t s) {
  if (warp_chains(p))
    return launch_chains(gdr_linear_bwd_kernel<T, V, GATE, 1>, p, 1, 1, s);
  return launch_chains(gdr_linear_bwd_kernel<T, V, GATE, kWarps>, p, kWarps,
                       cluster_size(p, 2), s);
}
template <typename T, int V, int GATE>
cudaError_t run_step(const LinParams &p, cudaStream_t s) {
  const long long n = (long long)p.nseq * (p.D / V);
  gdr_linear_step_kernel<T, V, GATE><<<(unsigned)((n + 127) / 128), 128, 0,
                                       s>>>(
      static_cast<const T *>(p.x), p.la, p.s0, p.sT,
      static_cast<T *>(p.out), p.ldx, p.nseq, p.H, p.d);
  return cudaGetLastError();
}

enum Op { kFwd, kBwd, kStep };

template <typename T, int V, int GATE>
cudaError_t run3(Op op, const LinParams &p, cudaStream_t s) {
  return op == kFwd ? run_fwd<T, V, GATE>(p, s)
                    : op == kBwd ? run_bwd<T, V, GATE>(p, s)
                                 : run_step<T, V, GATE>(p, s);
}
template <typename T, int V>
cudaError_t run2(Op op, int gate, const LinParams &p, cudaStream_t s) {
  switch (gate) {
    case GDR_GATE_NONE: return run3<T, V, GDR_GATE_NONE>(op, p, s);
    case GDR_GATE_SCALAR: return run3<T, V, GDR_GATE_SCALAR>(op, p, s);
    default: return run3<T, V, GDR_GATE_CHANNEL>(op, p, s);
  }
}
// Four channels a thread where rows keep 16-byte (fp32) alignment and a
// vector stays within a head; else one.
cudaError_t run(Op op, const gdr_opts &o, const LinParams &p, cudaStream_t s) {
  const bool v4 = p.D % 4 == 0 && p.ldx % 4 == 0 &&
                  (o.gate != GDR_GATE_SCALAR || p.d % 4 == 0);
  if (o.dtype == GDR_BF16)
    return v4 ? run2<__nv_bfloat16, 4>(op, o.gate, p, s)
              : run2<__nv_bfloat16, 1>(op, o.gate, p, s);
  return v4 ? run2<float, 4>(op, o.gate, p, s)
            : run2<float, 1>(op, o.gate, p, s);
}

// ------------------------------------------------------------------ checks

bool misaligned(const void *p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) != 0;
}

struct Span {
  const void *p;
  long long bytes;
};
// whether a buffer that is written meets any other
bool overlaps(const Span *w, int nw, const Span *r, int nr) {
  auto meet = [](const Span &a, const Span &b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p);
    const uintptr_t y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
  };
  for (int i = 0; i < nw; ++i) {
    for (int j = i + 1; j < nw; ++j)
      if (meet(w[i], w[j])) return true;
    for (int j = 0; j < nr; ++j)
      if (meet(w[i], r[j])) return true;
  }
  return false;
}

// Checks what the three entries share and fills the sizes.  *empty: nothing
// to do (no sequence, or no channel).
gdr_status check_common(const gdr_opts *opts, gdr_opts *o, LinParams *p,
                        const void *x, const float *log_alpha, int B, int T,
                        int H, int d, long long ldx, bool step, bool *empty) {
  o->dtype = GDR_BF16;
  o->gate = GDR_GATE_SCALAR;
  o->cu_seqlens = nullptr;
  o->num_seqs = 0;
  o->algo = GDR_ALGO_AUTO;
  if (opts) *o = *opts;
  if (B < 0 || T < 0 || H < 0 || d < 1) return GDR_ERR_INVALID_ARGUMENT;
  if (o->dtype != GDR_BF16 && o->dtype != GDR_FP32)
    return GDR_ERR_INVALID_ARGUMENT;
  if (o->gate != GDR_GATE_NONE && o->gate != GDR_GATE_SCALAR &&
      o->gate != GDR_GATE_CHANNEL)
    return GDR_ERR_INVALID_ARGUMENT;
  if (o->algo < GDR_ALGO_AUTO || o->algo > GDR_ALGO_RECURRENT)
    return GDR_ERR_INVALID_ARGUMENT;
  if (o->algo != GDR_ALGO_AUTO) return GDR_ERR_UNSUPPORTED;
  const bool packed = o->cu_seqlens != nullptr;
  if (packed && (step || B != 1 || o->num_seqs < 0))
    return GDR_ERR_INVALID_ARGUMENT;
  if (!packed && o->num_seqs != 0) return GDR_ERR_INVALID_ARGUMENT;
  if (o->gate == GDR_GATE_NONE && log_alpha) return GDR_ERR_INVALID_ARGUMENT;
  const long long D = (long long)H * d;
  if (H > 65535 || D > (1 << 24)) return GDR_ERR_UNSUPPORTED;
  const long long ntok = packed ? T : (long long)B * T;
  if (ntok > INT_MAX / 2) return GDR_ERR_UNSUPPORTED;
  if (ldx < D) return GDR_ERR_INVALID_ARGUMENT;
  std::memset(p, 0, sizeof(*p));
  p->nseq = packed ? o->num_seqs : B;
  p->T = T;
  p->ntok = (int)ntok;
  p->H = H;
  p->d = d;
  p->D = (int)D;
  p->ldx = ldx;
  p->cu = o->cu_seqlens;
  p->x = x;
  p->la = log_alpha;
  *empty = p->nseq == 0 || D == 0;
  if (!*empty && ntok > 0 && o->gate != GDR_GATE_NONE && !log_alpha)
    return GDR_ERR_INVALID_ARGUMENT;
  return GDR_OK;
}

// Cuts the channels into tiles; the chains have to fit the launch grid.
gdr_status cut(LinParams *p, bool per_head) {
  p->nct = per_head ? (p->d + kCh - 1) / kCh : 0;
  p->tiles = per_head ? p->H * p->nct : (p->D + kCh - 1) / kCh;
  const long long chains = (long long)p->tiles * p->nseq;
  if (chains > INT_MAX / kMaxCluster) return GDR_ERR_UNSUPPORTED;
  p->chains = (int)chains;
  return GDR_OK;
}

}  // namespace
}  // namespace gdr

extern "C" gdr_status gdr_linear_fwd(const void *x, long long ldx,
                                     const float *log_alpha,
                                     const float *initial_state, void *out,
                                     float *final_state, float *chunk_states,
                                     int B, int T, int H, int d,
                                     cudaStream_t stream,
                                     const gdr_opts *opts) {
  using namespace gdr;
  gdr_opts o;
  LinParams p;
  bool empty;
  gdr_status st = check_common(opts, &o, &p, x, log_alpha, B, T, H, d, ldx,
                               false, &empty);
  if (st != GDR_OK) return st;
  if (empty) return GDR_OK;
  if (p.ntok > 0 && (!x || !out)) return GDR_ERR_INVALID_ARGUMENT;
  const void *ptrs[] = {x, log_alpha, initial_state, out, final_state,
                        chunk_states};
  for (const void *q : ptrs)
    if (misaligned(q)) return GDR_ERR_INVALID_ARGUMENT;
  if (reinterpret_cast<uintptr_t>(p.cu) & 3u) return GDR_ERR_INVALID_ARGUMENT;
  const long long es = o.dtype == GDR_BF16 ? 2 : 4;
  const long long n = (long long)p.ntok * p.D;
  const long long sb = 4ll * p.nseq * p.D;
  const long long cb =
      4ll * (p.ntok / GDR_LINEAR_CHUNK + (long long)p.nseq) * p.D;
  const Span wr[] = {{out, n * es}, {final_state, sb}, {chunk_states, cb}};
  const Span rd[] = {
      {x, p.ntok ? ((p.ntok - 1) * ldx + p.D) * es : 0},
      {log_alpha, 4ll * p.ntok * (o.gate == GDR_GATE_SCALAR ? H : p.D)},
      {initial_state, sb}};
  if (overlaps(wr, 3, rd, 3)) return GDR_ERR_INVALID_ARGUMENT;
  p.s0 = initial_state;
  p.out = out;
  p.sT = final_state;
  p.states = chunk_states;
  st = cut(&p, false);
  if (st != GDR_OK) return st;
  return run(kFwd, o, p, stream) == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
}

extern "C" gdr_status gdr_linear_step(const void *x, long long ldx,
                                      const float *log_alpha,
                                      const float *state_in, float *state_out,
                                      void *out, int N, int H, int d,
                                      cudaStream_t stream,
                                      const gdr_opts *opts) {
  using namespace gdr;
  gdr_opts o;
  LinParams p;
  bool empty;
  gdr_status st = check_common(opts, &o, &p, x, log_alpha, N, 1, H, d, ldx,
                               true, &empty);
  if (st != GDR_OK) return st;
  if (empty) return GDR_OK;
  if (!x || !out || !state_out) return GDR_ERR_INVALID_ARGUMENT;
  const void *ptrs[] = {x, log_alpha, state_in, state_out, out};
  for (const void *q : ptrs)
    if (misaligned(q)) return GDR_ERR_INVALID_ARGUMENT;
  const long long es = o.dtype == GDR_BF16 ? 2 : 4;
  const long long n = (long long)N * p.D;
  // state_out may be state_in itself (each thread reads its channels before
  // it writes them)
  const Span wr[] = {{out, n * es}, {state_out, 4 * n}};
  const Span rd[] = {
      {x, ((N - 1) * ldx + p.D) * es},
      {log_alpha, 4ll * N * (o.gate == GDR_GATE_SCALAR ? H : p.D)},
      {state_in == state_out ? nullptr : state_in, 4 * n}};
  if (overlaps(wr, 2, rd, 3)) return GDR_ERR_INVALID_ARGUMENT;
  p.s0 = state_in;
  p.sT = state_out;
  p.out = out;
  return run(kStep, o, p, stream) == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
}

extern "C" gdr_status gdr_linear_backward(
    const void *x, long long ldx, const float *log_alpha,
    const float *initial_state, const float *chunk_states, const void *d_out,
    const float *d_final_state, void *dx, float *d_log_alpha,
    float *d_initial_state, int B, int T, int H, int d, cudaStream_t stream,
    const gdr_opts *opts) {
  using namespace gdr;
  gdr_opts o;
  LinParams p;
  bool empty;
  gdr_status st = check_common(opts, &o, &p, x, log_alpha, B, T, H, d, ldx,
                               false, &empty);
  if (st != GDR_OK) return st;
  if (o.gate == GDR_GATE_NONE && d_log_alpha) return GDR_ERR_INVALID_ARGUMENT;
  if (empty) return GDR_OK;
  if (p.ntok > 0 && (!x || !d_out || !dx ||
                     (o.gate != GDR_GATE_NONE && !d_log_alpha)))
    return GDR_ERR_INVALID_ARGUMENT;
  const void *ptrs[] = {x,     log_alpha, initial_state, chunk_states,
                        d_out, d_final_state, dx, d_log_alpha,
                        d_initial_state};
  for (const void *q : ptrs)
    if (misaligned(q)) return GDR_ERR_INVALID_ARGUMENT;
  if (reinterpret_cast<uintptr_t>(p.cu) & 3u) return GDR_ERR_INVALID_ARGUMENT;
  const long long es = o.dtype == GDR_BF16 ? 2 : 4;
  const long long n = (long long)p.ntok * p.D;
  const long long sb = 4ll * p.nseq * p.D;
  const long long lb = 4ll * p.ntok * (o.gate == GDR_GATE_SCALAR ? H : p.D);
  const long long cb =
      4ll * (p.ntok / GDR_LINEAR_CHUNK + (long long)p.nseq) * p.D;
  const Span wr[] = {{dx, n * es}, {d_log_alpha, lb}, {d_initial_state, sb}};
  const Span rd[] = {{x, p.ntok ? ((p.ntok - 1) * ldx + p.D) * es : 0},
                     {log_alpha, lb},
                     {initial_state, sb},
                     {chunk_states, cb},
                     {d_out, n * es},
                     {d_final_state, sb}};
  if (overlaps(wr, 3, rd, 6)) return GDR_ERR_INVALID_ARGUMENT;
  const bool scalar = o.gate == GDR_GATE_SCALAR;
  LinParams pf = p;
  st = cut(&pf, false);
  if (st == GDR_OK) st = cut(&p, scalar);
  if (st != GDR_OK) return st;
  // scratch: the chunk states where the caller has none (no gate needs
  // none), the channel tiles' shares of dlog_alpha
  const bool recompute = !chunk_states && o.gate != GDR_GATE_NONE;
  const bool parts = scalar && p.nct > 1;
  const size_t sbytes = recompute ? (size_t)((cb + 255) & ~255ll) : 0;
  const size_t bytes = sbytes + (parts ? (size_t)lb * p.nct : 0);
  void *ws = nullptr;
  if (bytes) {
    st = scratch_get(&ws, bytes, stream);
    if (st != GDR_OK) return st;
  }
  p.states = const_cast<float *>(chunk_states);
  cudaError_t e = cudaSuccess;
  if (recompute) {
    p.states = static_cast<float *>(ws);
    pf.s0 = initial_state;
    pf.states = p.states;
    e = run(kFwd, o, pf, stream);
  }
  p.dout = d_out;
  p.dsT = d_final_state;
  p.dx = dx;
  p.dla = d_log_alpha;
  p.part = reinterpret_cast<float *>(static_cast<char *>(ws) + sbytes);
  p.ds0 = d_initial_state;
  if (e == cudaSuccess) e = run(kBwd, o, p, stream);
  if (e == cudaSuccess && parts && p.ntok > 0) {
    const long long nh = (long long)p.ntok * H;
    gdr_linear_dla_kernel<<<(unsigned)((nh + 255) / 256), 256, 0, stream>>>(
        p.part, d_log_alpha, nh, p.nct);
    e = cudaGetLastError();
  }
  const cudaError_t f = ws ? scratch_put(ws, stream) : cudaSuccess;
  return (e == cudaSuccess && f == cudaSuccess) ? GDR_OK : GDR_ERR_CUDA;
}
