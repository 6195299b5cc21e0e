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
// One pass over the data.  A thread holds 8 tokens of 4 channels in registers
// and scans them alone; the runs of a warp (if it has more than one) are
// joined by shuffles, those of a CTA's four warps in shared memory, and those
// of up to eight CTAs, stacked in time as a cluster, in distributed shared
// memory.  Each thread then runs its tokens a second time from the state it
// now knows.  Nothing but x, log_alpha and the results touches HBM, and the
// only waits are a cluster's, for its own CTAs.
//
// Decays near 1 are held as alpha - 1: rounding alpha itself to fp32 puts a
// systematic 2^-25 into every step, which a memory of 10^4 tokens turns into
// 3e-4.  A run's decay is made from its sum of log_alpha; runs, warps and CTAs
// compose factors (joining sums and taking e^s anew at every join cost a
// quarter of the instructions: 93 us for 8 x 4096 x 2048).  log_alpha = -inf
// is a factor of exactly 0.
//
// Bound by HBM: forward 2 + 4 + 2 bytes a token and channel (bf16, a decay per
// channel), backward 2 + 4 + 2 + 2 + 4 and half a byte of chunk states.  What
// it takes to get near: inputs sent for one step ahead (cp.async into slots
// that only their thread reads), 19 (forward) and 35 (backward) instructions
// a value through packed fp32 pairs, four CTAs of four warps an SM so that
// one's joins hide behind the others' arithmetic, and no cluster-wide barrier.
// Measured in short runs (us, share of the 6.53 TB/s a copy reaches; batch x
// tokens x channels, decay per channel, bf16 unless said):
//   forward  8 x 4096 x 2048  85 (0.97); fp32 4 x 4096 x 2048 73 (0.84);
//            64 x 512 x 2048 84 (0.98); 1 x 65536 x 2048 201 (0.82)
//   backward 8 x 4096 x 2048 163 (0.91); fp32 4 x 4096 x 2048 121 (0.87);
//            1 x 65536 x 2048 350 (0.85)
//   no decay, 8 x 4096 x 2048: forward 51 (0.80), backward 58 (0.70); fp32
//            4 x 4096 x 2048: backward 47 (0.87)
// One long sequence is 64 chains cut over 8 CTAs each; every step of 1024
// tokens then waits for the slowest of the eight and for the exchange, about
// 0.5 us of 3.1.  Longer runs of the forward pass draw the full 1000 W and
// the clock falls to 1.78 GHz (8 x 4096 x 2048: 91 to 100 us from one GPU to
// another).  A decay per head leaves half the bytes and most of the
// arithmetic: 65 us of 42 forward, 110 of 67 backward (fp32 4 x 4096 x 2048:
// 49 of 41 and 82 of 64).  Decays below e^-1 anywhere in a warp's tile take it
// through the dearer form of decay_factor: 8 x 4096 x 2048 with log_alpha = -2
// 122 forward and 184 backward, -0.01 and -8 at random 135 and 203.  Rows that
// are not aligned (H d odd) take twice the instructions: 8 x 2000 x 3030 136
// to 139 us (0.44).

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstdlib>
#include <cstring>

#include "gdr_internal.h"
#include "sm100.cuh"
#include "streaming.cuh"

namespace gdr {

__device__ unsigned g_linear_error;

namespace {

namespace cg = cooperative_groups;
using namespace sm100;
using namespace streaming;

constexpr int kV = 4;            // channels of a thread
constexpr int kR = 8;            // tokens of a thread's run
constexpr int kWarps = 4;        // warps of a CTA, four CTAs to an SM
constexpr int kMaxCluster = 8;
constexpr long long kWaitCycles = 1ll << 31;   // ~1 s: never reached
// GDR_FAULT_INJECT_LINEAR_TIMEOUT=1: no maps are sent between CTAs, and the
// wait for them gives up after this many cycles (tests of the timeout path)
constexpr long long kInjectWaitCycles = 1ll << 20;
static_assert(kR == GDR_LINEAR_CHUNK, "a chunk is a run");
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
  int nc;           // CTAs per chain
  // bound of a wait for the other CTAs' maps; failure injection: none are sent
  long long wait_cycles;
  bool mute;
};

// ---------------------------------------------------------------- elements

// Four channels of a token as loaded: 16 bytes of fp32, 8 of bf16.
template <typename T>
struct Raw;
template <>
struct Raw<float> { using type = float4; };
template <>
struct Raw<__nv_bfloat16> { using type = uint2; };

__device__ __forceinline__ void unpack(const float4 &r, float (&f)[kV]) {
  f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w;
}
__device__ __forceinline__ void unpack(const uint2 &r, float (&f)[kV]) {
  f[0] = __uint_as_float(r.x << 16), f[1] = __uint_as_float(r.x & 0xffff0000u);
  f[2] = __uint_as_float(r.y << 16), f[3] = __uint_as_float(r.y & 0xffff0000u);
}
// Forgets what the compiler knows about a loaded value, so that it does not
// keep the unpacked elements in registers from one pass to the next.
__device__ __forceinline__ void renew(uint2 &r) {
  asm volatile("" : "+r"(r.x), "+r"(r.y));
}
__device__ __forceinline__ void renew(float4 &) {}

// A thread's first n <= 4 channels, as one vector (VEC: n is 4 or 0) or one
// by one where rows are not aligned for that.
template <bool VEC>
__device__ __forceinline__ void store(float *p, const float (&f)[kV], int n) {
  if constexpr (VEC) {
    if (n > 0)
      *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int v = 0; v < kV; ++v)
      if (n > v) p[v] = f[v];
  }
}
template <bool VEC>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&f)[kV],
                                      int n) {
  if constexpr (VEC) {
    if (n > 0)
      *reinterpret_cast<uint2 *>(p) =
          make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
  } else {
#pragma unroll
    for (int v = 0; v < kV; ++v)
      if (n > v) p[v] = __float2bfloat16_rn(f[v]);
  }
}

// ------------------------------------------------------------------ decays

// e^x, results below 2^-126 as 0; off by 2 + 1.2 |x| steps of 2^-23 at most
__device__ __forceinline__ float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
// e^s - 1 for kTight <= s <= 0: s times a least-maximum-error polynomial of
// (e^s - 1) / s (fitted by reweighted least squares; off by 1.4e-7 of e^s - 1
// at most, evaluated in fp32, and exact for s -> 0)
constexpr float kTight = -1.f;
__device__ __forceinline__ float expm1_tight(float s) {
  float p = fmaf(s, 1.283806487e-4f, 1.298663556e-3f);
  p = fmaf(s, p, 8.273095824e-3f);
  p = fmaf(s, p, 4.164557904e-2f);
  p = fmaf(s, p, 1.666630954e-1f);
  p = fmaf(s, p, 4.999997616e-1f);
  p = fmaf(s, p, 1.f);
  return s * p;
}

__device__ __forceinline__ Pair expm1_tight(Pair s) {
  Pair p = fma2(s, pair(1.283806487e-4f, 1.283806487e-4f),
                pair(1.298663556e-3f, 1.298663556e-3f));
  p = fma2(s, p, pair(8.273095824e-3f, 8.273095824e-3f));
  p = fma2(s, p, pair(4.164557904e-2f, 4.164557904e-2f));
  p = fma2(s, p, pair(1.666630954e-1f, 1.666630954e-1f));
  p = fma2(s, p, pair(4.999997616e-1f, 4.999997616e-1f));
  p = fma2(s, p, pair(1.f, 1.f));
  return mul2(s, p);
}

// The decay e^s in one of two forms.  Tight (kTight <= s <= 0, the usual
// decays): e^s - 1.  Any: for -1/8 < s <= 0 (sign bit set, also at s = 0)
// e^s - 1, else (sign bit clear) e^s, which keeps its digits however small it
// is; dearer to make and to apply.
template <bool TIGHT>
__device__ __forceinline__ float decay_factor(float s) {
  if constexpr (TIGHT) return expm1_tight(s);
  return s > -0.125f && s <= 0.f ? -fabsf(expm1_tight(s)) : exp_fast(s);
}
// e^s h, from decay_factor<TIGHT>(s)
template <bool TIGHT>
__device__ __forceinline__ float decay(float m, float h) {
  if constexpr (TIGHT) return fmaf(m, h, h);
  return fmaf(m, h, __float_as_int(m) < 0 ? h : 0.f);
}
template <int GATE, bool TIGHT>
__device__ __forceinline__ float decayed(float m, float h) {
  if constexpr (GATE == GDR_GATE_NONE) return h;
  return decay<TIGHT>(m, h);
}
// y <- e^s y + x over a thread's channels, from their factors m
template <int GV, int GATE, bool TIGHT>
__device__ __forceinline__ void advance(float (&y)[kV], const float (&m)[GV],
                                        const float (&x)[kV]) {
  if constexpr (TIGHT) {
#pragma unroll
    for (int v = 0; v < kV; v += 2) {
      Pair h = pair(y[v], y[v + 1]);
      if constexpr (GATE != GDR_GATE_NONE)
        h = fma2(pair(m[GV == kV ? v : 0], m[GV == kV ? v + 1 : 0]), h, h);
      split(add2(h, pair(x[v], x[v + 1])), y[v], y[v + 1]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < kV; ++v)
      y[v] = decayed<GATE, false>(m[GV == kV ? v : 0], y[v]) + x[v];
  }
}
// y <- e^s y
template <int GV, int GATE, bool TIGHT>
__device__ __forceinline__ void decay_all(float (&y)[kV],
                                          const float (&m)[GV]) {
  if constexpr (GATE == GDR_GATE_NONE) return;
  if constexpr (TIGHT) {
#pragma unroll
    for (int v = 0; v < kV; v += 2) {
      const Pair h = pair(y[v], y[v + 1]);
      split(fma2(pair(m[GV == kV ? v : 0], m[GV == kV ? v + 1 : 0]), h, h),
            y[v], y[v + 1]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < kV; ++v)
      y[v] = decayed<GATE, false>(m[GV == kV ? v : 0], y[v]);
  }
}
__device__ __forceinline__ void add_all(float (&y)[kV], const float (&x)[kV]) {
#pragma unroll
  for (int v = 0; v < kV; v += 2)
    split(add2(pair(y[v], y[v + 1]), pair(x[v], x[v + 1])), y[v], y[v + 1]);
}
// One token's log-decays into factors, added to the run's sums.
template <int GV, int GATE, bool TIGHT>
__device__ __forceinline__ void factors(float (&m)[GV], float (&sum)[GV]) {
  if constexpr (GATE == GDR_GATE_NONE) return;
  if constexpr (TIGHT && GV == kV) {
#pragma unroll
    for (int v = 0; v < GV; v += 2) {
      const Pair s = pair(m[v], m[v + 1]);
      split(add2(pair(sum[v], sum[v + 1]), s), sum[v], sum[v + 1]);
      split(expm1_tight(s), m[v], m[v + 1]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < GV; ++v) {
      sum[v] += m[v];
      m[v] = decay_factor<TIGHT>(m[v]);
    }
  }
}

// The factor (any form) of one decay after another: where both are held as
// alpha - 1 so is the product, unless it is far from 1.
__device__ __forceinline__ float compose(float a, float b) {
  const float m = fmaf(a, b, a + b);
  const float p = decay<false>(a, 1.f) * decay<false>(b, 1.f);
  return (__float_as_int(a) & __float_as_int(b)) < 0 && m > -0.5f ? -fabsf(m)
                                                                  : p;
}
// the factor that changes nothing, in both forms
constexpr float kNoDecay = -0.f;

// the map (factor in any form, b): y -> e^s y + b
template <int GATE>
__device__ __forceinline__ float apply(float2 m, float y) {
  return decayed<GATE, false>(m.x, y) + m.y;
}

template <bool B>
struct Bool { static constexpr bool value = B; };

__device__ __forceinline__ float min3(float a, float b, float c) {
  float y;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Whether every log-decay the warp holds is tight.
template <int GV, int GATE>
__device__ __forceinline__ bool is_tight(const float (&s)[kR][GV]) {
  if constexpr (GATE == GDR_GATE_NONE) return true;
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int r = 0; r < kR; r += 2)
#pragma unroll
    for (int v = 0; v < GV; ++v) {
      lo = min3(lo, s[r][v], s[r + 1][v]);
      hi = max3(hi, s[r][v], s[r + 1][v]);
    }
  return __all_sync(~0u, lo >= kTight && hi <= 0.f);
}
// The same for its runs' sums, given that each decay is.
template <int GV, int GATE>
__device__ __forceinline__ bool is_tight_run(const float (&s)[GV], bool each) {
  if constexpr (GATE == GDR_GATE_NONE) return true;
  float lo = s[0];
#pragma unroll
  for (int v = 1; v < GV; ++v) lo = fminf(lo, s[v]);
  return __all_sync(~0u, each && lo >= kTight);
}

// ------------------------------------------------------------------- tiles

// A warp's tile: kLanes threads side by side over 4 kLanes channels, and
// kSubs = 32 / kLanes runs of 8 tokens.
template <int LANES, int GATE>
struct Tile {
  static constexpr int kCh = kV * LANES;
  static constexpr int kSubs = 32 / LANES;
  static constexpr int kTok = kR * kSubs;
  // decays per thread and token (a thread's channels share a scalar one)
  static constexpr int GV = GATE == GDR_GATE_CHANNEL ? kV : 1;
};

template <int GV>
struct Map {       // y -> e^s y + b per channel of a thread
  float s[GV], b[kV];   // s: the sum of log-decays, then the factor
};
// From the sums to the factors.
template <int GV, int GATE>
__device__ __forceinline__ void to_factors(Map<GV> &f, bool tight) {
  if constexpr (GATE == GDR_GATE_NONE) return;
  if (!tight) {
#pragma unroll
    for (int v = 0; v < GV; ++v) f.s[v] = decay_factor<false>(f.s[v]);
  } else if constexpr (GV == kV) {
#pragma unroll
    for (int v = 0; v < GV; v += 2)
      split(expm1_tight(pair(f.s[v], f.s[v + 1])), f.s[v], f.s[v + 1]);
  } else {
    f.s[0] = expm1_tight(f.s[0]);
  }
}
// y <- the map at y
template <int GV, int GATE, bool TIGHT>
__device__ __forceinline__ void apply_all(float (&y)[kV], const Map<GV> &f) {
  advance<GV, GATE, TIGHT>(y, f.s, f.b);
}

// Scan of the warp's runs, in time (REV = false) or against it: on return
// `f` maps over this run and all before it (in scan order), `ex` over those
// before it alone.
template <int LANES, int GV, int GATE, bool REV>
__device__ __forceinline__ void warp_scan(Map<GV> &f, Map<GV> &ex,
                                          bool tight) {
  if constexpr (LANES < 32) {
    const int lane = threadIdx.x & 31;
    auto from = [](float x, int off) {
      return REV ? __shfl_down_sync(~0u, x, off) : __shfl_up_sync(~0u, x, off);
    };
    auto stage = [&](int off, auto tc) {
      const bool has = REV ? lane + off < 32 : lane >= off;
      float y[kV];
#pragma unroll
      for (int v = 0; v < kV; ++v) y[v] = from(f.b[v], off);
      apply_all<GV, GATE, tc.value>(y, f);
#pragma unroll
      for (int v = 0; v < kV; ++v)
        if (has) f.b[v] = y[v];
      if constexpr (GATE != GDR_GATE_NONE) {
#pragma unroll
        for (int v = 0; v < GV; ++v) {
          const float g = from(f.s[v], off);
          const float m = tc.value ? fmaf(f.s[v], g, f.s[v] + g)
                                   : compose(f.s[v], g);
          if (has) f.s[v] = m;
        }
      }
    };
    auto all = [&](auto tc) {
      stage(LANES, tc);
      if constexpr (LANES < 16) stage(2 * LANES, tc);
    };
    if (tight) all(Bool<true>{}); else all(Bool<false>{});
    const bool first = REV ? lane + LANES >= 32 : lane < LANES;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const float b = from(f.b[v], LANES);
      ex.b[v] = first ? 0.f : b;
    }
    if constexpr (GATE != GDR_GATE_NONE) {
#pragma unroll
      for (int v = 0; v < GV; ++v) {
        const float m = from(f.s[v], LANES);
        ex.s[v] = first ? kNoDecay : m;
      }
      // (from here on in any form)
      if (tight) {
#pragma unroll
        for (int v = 0; v < GV; ++v) f.s[v] = -fabsf(f.s[v]);
      }
    }
  }
}
// y, the value that enters the warp's tile, moved on to this thread's run.
template <int LANES, int GV, int GATE>
__device__ __forceinline__ void enter(float (&y)[kV], const Map<GV> &ex,
                                      bool tight) {
  if constexpr (LANES < 32) {
    if (tight)
      apply_all<GV, GATE, true>(y, ex);
    else
      apply_all<GV, GATE, false>(y, ex);
  }
}

// A thread's place: its sequence, its channels.
struct Place {
  int n;            // sequence
  int base, end;    // channels of the tile: [base, min(base + CH, end))
  int ch, nch;      // the thread's first channel, and how many it has
  int head, ct;     // the tile's head and tile within it (nct > 0)
};
template <int LANES>
__device__ __forceinline__ Place place(const LinParams &p, int chain) {
  Place q;
  const int c = (threadIdx.x & 31) % LANES;
  const int tile = chain % p.tiles;
  q.n = chain / p.tiles;
  q.head = q.ct = 0;
  if (p.nct) {
    q.head = tile / p.nct;
    q.ct = tile - q.head * p.nct;
    q.base = q.head * p.d + q.ct * kV * LANES;
    q.end = (q.head + 1) * p.d;
  } else {
    q.base = tile * kV * LANES;
    q.end = p.D;
  }
  q.ch = q.base + c * kV;
  q.nch = min(max(q.end - q.ch, 0), kV);
  return q;
}

// The inputs of one step where rows are aligned for vectors: a thread's own 8
// tokens of 4 channels are fetched into the thread's own slots of shared
// memory while the step before is computed.  Slots are [token][thread], so
// that a warp's accesses are contiguous; nobody else reads them.  Where x is
// all there is, at 2 bytes a value, one step's is too little to keep HBM busy
// and goes two steps ahead (forward, bf16, no decay, 8 x 4096 x 2048: one step
// ahead 55.9 us, two 51.8; with a decay per head 65.2 and 64.0, but 1 x 4096
// 13.4 and 13.9; fp32 without one 1 x 32768 100.7 and 108.3).
template <typename T, int GATE, bool BWD>
struct Slots {
  using raw_t = typename Raw<T>::type;
  static constexpr bool kX = !BWD || GATE != GDR_GATE_NONE;
  static constexpr int GV = GATE == GDR_GATE_CHANNEL ? kV : 1;
  static constexpr bool kGate = GATE == GDR_GATE_CHANNEL;
  static constexpr bool kState = BWD && GATE != GDR_GATE_NONE;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kSlots = kR * kThreads;
  static constexpr int kRaw = (int)sizeof(raw_t);
  static constexpr bool kTwo =
      !BWD && GATE == GDR_GATE_NONE && sizeof(T) == 2;
  static constexpr int kBytes = kSlots * (16 * kGate + kRaw * (kX + BWD)) *
                                    (1 + kTwo) +
                                16 * kThreads * kState;
  // at the thread's first token of the step to fetch; distances between
  // tokens, in elements
  const T *x, *dout;
  const float *la, *states;
  int ldx, ldg, ldd;
  bool has;                // whether the thread has channels (4 or none)
  float sc[kR];            // scalar decays of the step to come

  __device__ __forceinline__ void start(const LinParams &p, const Place &q,
                                        int tok0, int t) {
    ldx = (int)p.ldx;
    ldg = GATE == GDR_GATE_SCALAR ? p.H : p.D;
    ldd = p.D;
    has = q.nch > 0;
    const long long tok = (long long)tok0 + t;
    x = static_cast<const T *>(p.x) + tok * ldx + q.ch;
    dout = static_cast<const T *>(p.dout) + tok * ldd + q.ch;
    la = p.la + tok * ldg +
         (GATE == GDR_GATE_CHANNEL ? q.ch : p.nct ? q.head : q.ch / p.d);
    // (t is a multiple of 8, and so is what it moves on by)
    states = p.states + ((long long)(tok0 / kR) + q.n + t / kR) * ldd + q.ch;
  }
  __device__ __forceinline__ void move(int tokens) {
    x += (long long)tokens * ldx;
    la += (long long)tokens * ldg;
    if constexpr (BWD) {
      dout += (long long)tokens * ldd;
      states += (long long)(tokens / kR) * ldd;
    }
  }

  static __device__ __forceinline__ raw_t *xs(char *sm) {
    return reinterpret_cast<raw_t *>(sm) + threadIdx.x;
  }
  static __device__ __forceinline__ raw_t *ds(char *sm) {
    return xs(sm) + (kX ? kSlots : 0);
  }
  static __device__ __forceinline__ float4 *gs(char *sm) {
    return reinterpret_cast<float4 *>(sm + kSlots * kRaw * (kX + BWD)) +
           threadIdx.x;
  }
  // sends for the 8 tokens from t on, those before `end`
  template <bool FULL>
  __device__ __forceinline__ void send_all(char *sm, int t, int end) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const bool ok = FULL || (t + r < end && has);
      if constexpr (!BWD)
        copy_async<kRaw>(xs(sm) + r * kThreads, x + (long long)r * ldx,
                         ok ? kRaw : 0);
      if constexpr (BWD)
        copy_async<kRaw>(ds(sm) + r * kThreads, dout + (long long)r * ldd,
                         ok ? kRaw : 0);
      if constexpr (kGate)
        copy_async<16>(gs(sm) + r * kThreads, la + (long long)r * ldg,
                       ok ? 16 : 0);
    }
    if constexpr (kState)
      copy_async<16>(gs(sm) + kSlots * kGate, states,
                     t < end && has ? 16 : 0);
  }
  __device__ __forceinline__ void send(char *sm, int t, int end) {
    if (!BWD && t + kR <= end && has)
      send_all<true>(sm, t, end);
    else
      send_all<false>(sm, t, end);
  }
  // fetches step k, which begins at this thread's token t; kTwo: x of step
  // k + 1, `span` tokens on (that of step k has been sent before)
  __device__ __forceinline__ void fetch(char *slots, int k, int t, int end,
                                        int span) {
    if constexpr (GATE == GDR_GATE_SCALAR) {
#pragma unroll
      for (int r = 0; r < kR; ++r)
        sc[r] = t + r < end && has ? load(la + (long long)r * ldg) : 0.f;
    }
    if constexpr (kTwo) {
      x += (long long)span * ldx;
      send(step(slots, k + 1), t + span, end);
      x -= (long long)span * ldx;
      copies_sent();
    } else {
      send(slots, t, end);
    }
  }
  __device__ __forceinline__ void first(char *slots, int t, int end,
                                        int span) {
    if constexpr (kTwo) {
      send(slots, t, end);
      copies_sent();
    }
    fetch(slots, 0, t, end, span);
  }
  static __device__ __forceinline__ char *step(char *slots, int k) {
    return slots + (kTwo && (k & 1) ? kBytes / 2 : 0);
  }
  // x of the backward pass comes on its own: it is read where it is used, to
  // spare registers, and so is still in its slots when the rest is fetched
  __device__ __forceinline__ void fetch_x(char *sm, const T *at, int t,
                                          int end) const {
    if constexpr (BWD && kX) {
#pragma unroll
      for (int r = 0; r < kR; ++r)
        copy_async<kRaw>(xs(sm) + r * kThreads, at + (long long)r * ldx,
                         t + r < end && has ? kRaw : 0);
    }
  }
  __device__ __forceinline__ raw_t x_at(char *sm, int r) const {
    return xs(sm)[r * kThreads];
  }
  __device__ __forceinline__ void take(char *slots, int k, raw_t (&xr)[kR],
                                       raw_t (&dr)[kR], float (&m)[kR][GV],
                                       float (&h)[kV]) const {
    if constexpr (kTwo)
      copies_landed_but<1>();
    else
      copies_landed();
    char *sm = step(slots, k);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      if constexpr (!BWD) xr[r] = x_at(sm, r);
      if constexpr (BWD) dr[r] = ds(sm)[r * kThreads];
      if constexpr (kGate) unpack(gs(sm)[r * kThreads], m[r]);
      if constexpr (GATE == GDR_GATE_SCALAR) m[r][0] = sc[r];
    }
    if constexpr (kState) unpack(gs(sm)[kSlots * kGate], h);
  }
};

// The inputs and results of one step where rows are not aligned: a warp's
// tile of 32 tokens by 32 channels goes through shared memory row by row, a
// lane to a channel (of bf16, a lane to a 4-byte word, since a row may start
// in the middle of one), and from there to the threads that compute it and
// back.  Nothing is fetched ahead.
template <typename T, int GATE, bool BWD>
struct Rows {
  using raw_t = typename Raw<T>::type;
  static constexpr bool kX = !BWD || GATE != GDR_GATE_NONE;
  static constexpr int GV = GATE == GDR_GATE_CHANNEL ? kV : 1;
  static constexpr bool kGate = GATE == GDR_GATE_CHANNEL;
  static constexpr bool kState = BWD && GATE != GDR_GATE_NONE;
  static constexpr int kRow = 32;                      // tokens and channels
  // words of a row in shared memory: of bf16 16, and one for an odd start
  static constexpr int kPitch = sizeof(T) == 4 ? 32 : 17;
  static constexpr int kTile = kRow * kPitch * 4;      // of x or dout
  static constexpr int kTileG = kGate ? kRow * 32 * 4 : 0;
  static constexpr int kTileS = kState ? 4 * 32 * 4 : 0;
  static constexpr int kWarp = kTile * (kX + BWD) + kTileG + kTileS;
  static constexpr int kBytes = kWarp * kWarps;
  // at the tile's first channel of the sequence's first token
  const T *x, *dout;
  const float *la, *states;
  T *out;
  float *dla;
  int ldx, ldg, ldd, n;    // n: channels of the tile that exist
  int t0, end;             // the tile's tokens: t0 .. t0 + 31, those < end
  int tn, endn;            // of the step to come

  __device__ __forceinline__ int lane() const { return threadIdx.x & 31; }
  __device__ __forceinline__ int sub() const { return lane() / 8; }
  __device__ __forceinline__ int col() const { return lane() % 8; }

  __device__ __forceinline__ void start(const LinParams &p, const Place &q,
                                        int tok0, int) {
    ldx = (int)p.ldx;
    ldg = GATE == GDR_GATE_SCALAR ? p.H : p.D;
    ldd = p.D;
    n = min(q.end - q.base, kRow);
    x = static_cast<const T *>(p.x) + (long long)tok0 * ldx + q.base;
    dout = static_cast<const T *>(p.dout) + (long long)tok0 * ldd + q.base;
    la = p.la + (long long)tok0 * ldg +
         (GATE == GDR_GATE_CHANNEL ? q.base : q.head);
    states = p.states + ((long long)(tok0 / kR) + q.n) * ldd + q.base;
    out = static_cast<T *>(BWD ? p.dx : p.out) + (long long)tok0 * ldd +
          q.base;
    dla = p.dla + (long long)tok0 * ldd + q.base;
  }
  __device__ __forceinline__ void move(int) {}
  __device__ __forceinline__ void first(char *sm, int t, int e, int) {
    fetch(sm, 0, t, e, 0);
  }
  __device__ __forceinline__ void fetch(char *, int, int t, int e, int) {
    tn = t - sub() * kR;
    endn = e;
    if (tn + lane() < e) {
      if constexpr (kX) soon(x, ldx);
      if constexpr (BWD) soon(dout, ldd);
      if constexpr (kGate) soon(la, ldg);
    }
  }
  __device__ __forceinline__ void fetch_x(char *, const T *, int, int) const {}

  __device__ __forceinline__ char *base(char *sm) const {
    return sm + (threadIdx.x >> 5) * kWarp;
  }
  __device__ __forceinline__ char *ds(char *sm) const {
    return base(sm) + (kX ? kTile : 0);
  }
  __device__ __forceinline__ float *gs(char *sm) const {
    return reinterpret_cast<float *>(base(sm) + kTile * (kX + BWD));
  }
  // ROWS rows of fp32, the first `have` of them
  template <int ROWS>
  __device__ __forceinline__ void rows(float *dst, const float *src, int ld,
                                       int have) const {
    src += lane();
    dst += lane();
    float v[ROWS];
    if (have == ROWS && n == kRow) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) v[r] = load(src + (long long)r * ld);
    } else {
      if (lane() >= n) have = 0;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        v[r] = 0.f;
        if (r < have) v[r] = load(src + (long long)r * ld);
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) dst[r * 32] = v[r];
  }
  // the same of bf16, two rows at a time; a lane's rows all start alike.  Of
  // a word whose second half is beyond the tile only the first is read.
  template <int ROWS>
  __device__ __forceinline__ void rows(float *dst, const __nv_bfloat16 *src,
                                       int ld, int have) const {
    auto word = [&](int r, int j, int &bytes) {
      const uintptr_t at =
          reinterpret_cast<uintptr_t>(src + (long long)r * ld);
      bytes = r < have ? (int)(at & 2) + 2 * n - 4 * j : 0;
      return reinterpret_cast<const char *>(at & ~(uintptr_t)3) + 4 * j;
    };
    auto read = [&](const char *p, int bytes) {
      uint32_t v = 0;
      if (bytes >= 4) v = load(reinterpret_cast<const uint32_t *>(p));
      if (bytes == 2) v = load(reinterpret_cast<const unsigned short *>(p));
      return v;
    };
    const int r0 = lane() / 16, j = lane() % 16;
    int bytes, bytes1;
    const char *p = word(r0, j, bytes);
    const char *p1 = word(lane(), 16, bytes1);
    uint32_t *d = reinterpret_cast<uint32_t *>(dst);
    uint32_t v[ROWS / 2];
    if (have == ROWS && n == kRow) {       // (then words 0 .. 15 are whole)
#pragma unroll
      for (int r = 0; r < ROWS; r += 2)
        v[r / 2] = load(
            reinterpret_cast<const uint32_t *>(p + (long long)r * (2 * ld)));
    } else {
#pragma unroll
      for (int r = 0; r < ROWS; r += 2)
        v[r / 2] = read(p + (long long)r * (2 * ld),
                        r + r0 < have ? bytes : 0);
    }
    d[lane() * kPitch + 16] = read(p1, bytes1);
    d += r0 * kPitch + j;
#pragma unroll
    for (int r = 0; r < ROWS; r += 2) d[r * kPitch] = v[r / 2];
  }
  // brings row `lane` of the next step's tile into L2
  template <typename E>
  __device__ __forceinline__ void soon(const E *src, int ld) const {
    const E *row = src + (long long)(tn + lane()) * ld;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(row) : "memory");
    asm volatile("prefetch.global.L2 [%0];" ::"l"(row + n - 1) : "memory");
  }
  // the thread's 4 channels of its token r, of the tile that starts at `src`
  // (a tile's first token has an even index, and so has each thread's)
  __device__ __forceinline__ raw_t at(const char *tile, const T *src, int ld,
                                      int r) const {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(tile) +
                        (sub() * kR + r) * kPitch;
    if constexpr (sizeof(T) == 4) {
      return *reinterpret_cast<const float4 *>(w + col() * 4);
    } else {
      w += col() * 2;
      const bool odd =
          (((int)reinterpret_cast<uintptr_t>(src) >> 1) ^ (r & ld)) & 1;
      return odd ? make_uint2(__funnelshift_r(w[0], w[1], 16),
                              __funnelshift_r(w[1], w[2], 16))
                 : make_uint2(w[0], w[1]);
    }
  }
  __device__ __forceinline__ raw_t x_at(char *sm, int r) const {
    return at(base(sm), x, ldx, r);
  }
  __device__ __forceinline__ void take(char *sm, int, raw_t (&xr)[kR],
                                       raw_t (&dr)[kR], float (&m)[kR][GV],
                                       float (&h)[kV]) {
    t0 = tn;
    end = endn;
    const int have = end > t0 ? min(end - t0, kRow) : 0;
    const long long at0 = have > 0 ? t0 : 0;
    __syncwarp();          // the step before is out of shared memory
    if constexpr (kX)
      rows<kRow>(reinterpret_cast<float *>(base(sm)), x + at0 * ldx, ldx,
                 have);
    if constexpr (BWD)
      rows<kRow>(reinterpret_cast<float *>(ds(sm)), dout + at0 * ldd, ldd,
                 have);
    if constexpr (kGate) rows<kRow>(gs(sm), la + at0 * ldg, ldg, have);
    if constexpr (kState)
      rows<4>(gs(sm) + kTileG / 4, states + at0 / kR * ldd, ldd,
              (have + kR - 1) / kR);
    if constexpr (GATE == GDR_GATE_SCALAR) {
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const int row = sub() * kR + r;
        m[r][0] = row < have ? load(la + (at0 + row) * ldg) : 0.f;
      }
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      if constexpr (!BWD) xr[r] = x_at(sm, r);
      if constexpr (BWD) dr[r] = at(ds(sm), dout, ldd, r);
      if constexpr (kGate)
        unpack(*reinterpret_cast<const float4 *>(
                   gs(sm) + (sub() * kR + r) * 32 + col() * 4),
               m[r]);
    }
    if constexpr (kState)
      unpack(*reinterpret_cast<const float4 *>(gs(sm) + kTileG / 4 +
                                               sub() * 32 + col() * 4),
             h);
    __syncwarp();          // the tiles of dout (x) and of the decays are free
  }
  // results: into the tiles of dout (forward: x) and of the decays ...
  __device__ __forceinline__ void put(char *sm, int r, const float (&f)[kV]) {
    T *d = reinterpret_cast<T *>(BWD ? ds(sm) : base(sm));
    store<true>(d + (sub() * kR + r) * kRow + col() * kV, f, kV);
  }
  __device__ __forceinline__ void put_la(char *sm, int r,
                                         const float (&f)[kV]) {
    store<true>(gs(sm) + (sub() * kR + r) * kRow + col() * kV, f, kV);
  }
  // ... and out, row by row
  __device__ __forceinline__ void flush(char *sm) {
    const T *d = reinterpret_cast<const T *>(BWD ? ds(sm) : base(sm)) + lane();
    const float *g = gs(sm) + lane();
    const int have = lane() < n ? min(end - t0, kRow) : 0;
    T *o = out + (long long)t0 * ldd + lane();
    float *og = dla + (long long)t0 * ldd + lane();
    __syncwarp();
    if (n == kRow && end - t0 >= kRow) {
#pragma unroll
      for (int r = 0; r < kRow; ++r) {
        o[(long long)r * ldd] = d[r * kRow];
        if constexpr (BWD && kGate) og[(long long)r * ldd] = g[r * kRow];
      }
      return;
    }
#pragma unroll 4
    for (int r = 0; r < kRow; ++r)
      if (r < have) {
        o[(long long)r * ldd] = d[r * kRow];
        if constexpr (BWD && kGate) og[(long long)r * ldd] = g[r * kRow];
      }
  }
};

template <typename T, bool VEC, int GATE, bool BWD>
struct InputsOf { using type = Rows<T, GATE, BWD>; };
template <typename T, int GATE, bool BWD>
struct InputsOf<T, true, GATE, BWD> { using type = Slots<T, GATE, BWD>; };
template <typename T, bool VEC, int GATE, bool BWD>
using Inputs = typename InputsOf<T, VEC, GATE, BWD>::type;

// The joins across the warps of a CTA and the CTAs of a cluster.
template <int CH, int NW>
struct __align__(128) Joint {
  float2 warp[NW][CH];                   // each warp's map
  float in[NW][CH];                      // what enters each warp's tile
  float2 rank[2][kMaxCluster][CH];       // each CTA's map; alternating, since
                                         // a CTA may be a step ahead
  uint64_t full[2];                      // mbarriers: a step's maps are here
};

// --- exchange between the CTAs of a cluster.  A map goes to every CTA as an
// asynchronous remote store that counts its bytes down on the receiver's
// mbarrier: no cluster-wide barrier (whose release would wait for all the
// results still on their way to memory) in the loop.  Bytes for step k + 2
// cannot arrive before step k was read: their sender has first received step
// k + 1 from this CTA, which sends it after that reading.
__device__ __forceinline__ uint32_t remote(const void *p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(a)
      : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void send_map(uint32_t dst, float2 m,
                                         uint32_t bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], "
      "{%1, %2}, [%3];" ::"r"(dst),
      "f"(m.x), "f"(m.y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ bool maps_here(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], "
      "%2;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}


// Every warp's map into shared memory (`edge`: this thread's run holds it).
template <int GV, int GATE, typename J>
__device__ __forceinline__ void post(J &jt, const Map<GV> &f, int c,
                                     bool edge) {
  const int w = threadIdx.x >> 5;
  if (edge) {
#pragma unroll
    for (int v = 0; v < kV; ++v)
      jt.warp[w][c * kV + v] =
          make_float2(GATE == GDR_GATE_NONE ? 0.f : f.s[GV == kV ? v : 0],
                      f.b[v]);
  }
  __syncthreads();
}

// Runs the posted maps: thread i < CH looks after channel i and carries its
// value (`carry`) from step to step.  Leaves jt.in for everyone.
template <int CH, int GATE, bool REV, bool CL, typename J>
__device__ __forceinline__ void run_maps(J &jt, int step, int nc, int rank,
                                         long long &limit, bool mute,
                                         float &carry) {
  const int i = threadIdx.x, buf = step & 1;
  if constexpr (!CL) {
    if (i < CH) {
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const int j = REV ? kWarps - 1 - k : k;
        jt.in[j][i] = carry;
        carry = apply<GATE>(jt.warp[j][i], carry);
      }
    }
  } else {
    float2 pre[kWarps];                  // the maps of the warps before
    if (i < CH) {
      // (after an expired wait nothing more is sent, expected or waited for)
      if (i == 0 && limit > 0)
        mbar_arrive_expect_tx(&jt.full[buf], nc * CH * (int)sizeof(float2));
      float2 m = make_float2(kNoDecay, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float2 g = jt.warp[REV ? kWarps - 1 - k : k][i];
        pre[k] = m;
        m = make_float2(compose(m.x, g.x), apply<GATE>(g, m.y));
      }
      if (!mute && limit > 0) {
        const uint32_t off = smem_u32(&jt.rank[buf][rank][i]) -
                             smem_u32(&jt.full[buf]);
        for (int r = 0; r < nc; ++r) {
          const uint32_t bar = remote(&jt.full[buf], r);
          send_map(bar + off, m, bar);
        }
      }
      // bounded: after one wait that expires no other is waited for, so that
      // every CTA gets to the end, where the cluster meets once more
      if (limit > 0) {
        const long long start = clock64();
        while (!maps_here(&jt.full[buf], (step >> 1) & 1))
          if (clock64() - start > limit) {
            limit = 0;
            atomicExch(&g_linear_error, 1u);
            break;
          }
      }
      float y = 0.f;
#pragma unroll (REV ? 1 : kMaxCluster)
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < nc) {
          if (r == rank) y = carry;
          carry = apply<GATE>(jt.rank[buf][r][i], carry);
        }
#pragma unroll
      for (int k = 0; k < kWarps; ++k)
        jt.in[REV ? kWarps - 1 - k : k][i] = apply<GATE>(pre[k], y);
    }
  }
  __syncthreads();
}

// No CTA writes into another's shared memory before that one has begun and
// set up its mbarriers (nor after it has ended: the kernels end with another
// meeting).
template <typename J>
__device__ __forceinline__ void meet_first(J &jt) {
  if (threadIdx.x == 0) {
    mbar_init(&jt.full[0], 1);
    mbar_init(&jt.full[1], 1);
    fence_mbar_init();
  }
  cg::this_cluster().sync();
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

// ----------------------------------------------------------------- forward

// WPC = kWarps: a chain (sequence and channel tile) by a CTA, or by a cluster
// of them (CL), stacked in time; WPC = 1: by a warp.
template <typename T, int LANES, bool VEC, int GATE, int WPC, bool CL>
__global__ void __launch_bounds__(kWarps * 32, 4)
    gdr_linear_fwd_kernel(const LinParams p) {
  using TL = Tile<LANES, GATE>;
  constexpr int GV = TL::GV, CH = TL::kCh;
  prior_done();
  next_may_start();
  using IN = Inputs<T, VEC, GATE, false>;
  using raw_t = typename IN::raw_t;
  extern __shared__ __align__(128) char slots[];
  __shared__ __align__(128) Joint<WPC == 1 ? 1 : CH, WPC> jt;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LANES, c = lane % LANES;
  int nc = 1, rank = 0, chain;
  if constexpr (WPC == 1) {
    chain = blockIdx.x * kWarps + w;
    if (chain >= p.chains) return;
  } else {
    nc = p.nc;
    if constexpr (CL) rank = (int)cg::this_cluster().block_rank();
    chain = blockIdx.x / nc;
    if constexpr (CL) meet_first(jt);
  }
  const Place q = place<LANES>(p, chain);
  int tok0, len;
  seq_range(p, q.n, &tok0, &len);
  // the channel this thread carries the state of
  const int own = WPC == 1 ? lane : threadIdx.x;
  long long limit = p.wait_cycles;
  const bool owns = own < CH && q.base + own < q.end;
  const long long so = (long long)q.n * p.D + q.base + own;
  float carry = (p.s0 && owns) ? p.s0[so] : 0.f;
  constexpr int kBlock = WPC * TL::kTok;
  const int span = kBlock * nc;
  const int steps = (len + span - 1) / span;
  // the thread's first token within the block's first step
  const int t00 =
      rank * kBlock + (WPC == 1 ? 0 : w * TL::kTok) + sub * kR;
  IN in;
  in.start(p, q, tok0, t00);
  if (steps > 0) in.first(slots, t00, len, span);
  T *op = static_cast<T *>(p.out) + ((long long)tok0 + t00) * p.D + q.ch;
  float *sp =
      p.states + ((long long)(tok0 / kR) + q.n + t00 / kR) * p.D + q.ch;

  for (int k = 0; k < steps; ++k) {
    const int t = k * span + t00;                      // the thread's
    raw_t xr[kR], dr[kR];
    float m[kR][GV], none[kV];
    in.move(span);
    in.take(slots, k, xr, dr, m, none);
    if (k + 1 < steps) in.fetch(slots, k + 1, t + span, len, span);
    // the run on its own
    Map<GV> f, ex;
#pragma unroll
    for (int v = 0; v < kV; ++v) f.b[v] = 0.f;
#pragma unroll
    for (int v = 0; v < GV; ++v) f.s[v] = 0.f;
    const bool tight = is_tight<GV, GATE>(m);
    auto alone = [&](auto tc) {
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float x[kV];
        unpack(xr[r], x);
        factors<GV, GATE, tc.value>(m[r], f.s);
        advance<GV, GATE, tc.value>(f.b, m[r], x);
      }
    };
    if (tight) alone(Bool<true>{}); else alone(Bool<false>{});
    const bool runs = is_tight_run<GV, GATE>(f.s, tight);
    to_factors<GV, GATE>(f, runs);
    warp_scan<LANES, GV, GATE, false>(f, ex, runs);
    // what enters the warp's tile
    float h[kV];
    if constexpr (WPC == 1) {
      float2 mine = make_float2(0.f, 0.f);
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const int src = 32 - LANES + lane / kV;
        const bool me = lane % kV == v;
        const float b = __shfl_sync(~0u, f.b[v], src);
        const float s = __shfl_sync(~0u, f.s[GV == kV ? v : 0], src);
        if (me) mine = make_float2(s, b);
        h[v] = __shfl_sync(~0u, carry, c * kV + v);
      }
      carry = apply<GATE>(mine, carry);
    } else {
      post<GV, GATE>(jt, f, c, sub == TL::kSubs - 1);
      run_maps<CH, GATE, false, CL>(jt, k, nc, rank, limit, p.mute, carry);
#pragma unroll
      for (int v = 0; v < kV; ++v) h[v] = jt.in[w][c * kV + v];
    }
    enter<LANES, GV, GATE>(h, ex, runs);
    if (p.states) {
      store<VEC>(sp, h, t < len ? q.nch : 0);
      sp += (long long)(span / kR) * p.D;
    }
    if (p.out) {
      auto again = [&](auto tc, auto full) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          float x[kV];
          renew(xr[r]);
          unpack(xr[r], x);
          advance<GV, GATE, tc.value>(h, m[r], x);
          if constexpr (VEC) {
            if (full.value || (t + r < len && q.nch > 0))
              store<true>(op + (long long)r * p.D, h, kV);
          } else {
            in.put(slots, r, h);
          }
        }
      };
      if (!tight)
        again(Bool<false>{}, Bool<false>{});
      else if (t + kR <= len && q.nch == kV)
        again(Bool<true>{}, Bool<true>{});
      else
        again(Bool<true>{}, Bool<false>{});
      if constexpr (!VEC) in.flush(slots);
      op += (long long)span * p.D;
    }
  }
  if (p.sT && owns && rank == 0) p.sT[so] = carry;
  if constexpr (CL) cg::this_cluster().sync();
}

// ---------------------------------------------------------------- backward

// Sums v[0 .. 7] over the LANES (8 or 16) threads of a token run, thread c of
// which ends with one of the sums in v[0]; returns which.  In every round
// each thread hands half of its values to a partner and adds the partner's
// to the other half.
template <int LANES>
__device__ __forceinline__ int sum_tokens(float (&v)[kR], int c) {
  int which = 0;
#pragma unroll
  for (int n = kR / 2, o = LANES / 2; n > 0; n >>= 1, o >>= 1) {
    const bool up = c & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(~0u, give, o);
    }
    which += up ? n : 0;
  }
  if constexpr (LANES == 16) v[0] += __shfl_xor_sync(~0u, v[0], 1);
  return which;
}

// From the last token to the first.  Every thread runs h forward over its
// tokens from their chunk state, leaving alpha_t h_{t-1} in registers; then c
// runs backward through the same joins as the forward pass.
template <typename T, int LANES, bool VEC, int GATE, int WPC, bool CL>
__global__ void __launch_bounds__(kWarps * 32, 4)
    gdr_linear_bwd_kernel(const LinParams p) {
  using TL = Tile<LANES, GATE>;
  constexpr int GV = TL::GV, CH = TL::kCh;
  prior_done();
  next_may_start();
  using IN = Inputs<T, VEC, GATE, true>;
  using raw_t = typename IN::raw_t;
  extern __shared__ __align__(128) char slots[];
  __shared__ __align__(128) Joint<WPC == 1 ? 1 : CH, WPC> jt;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LANES, c = lane % LANES;
  int nc = 1, rank = 0, chain;
  if constexpr (WPC == 1) {
    chain = blockIdx.x * kWarps + w;
    if (chain >= p.chains) return;
  } else {
    nc = p.nc;
    if constexpr (CL) rank = (int)cg::this_cluster().block_rank();
    chain = blockIdx.x / nc;
    if constexpr (CL) meet_first(jt);
  }
  const Place q = place<LANES>(p, chain);
  int tok0, len;
  seq_range(p, q.n, &tok0, &len);
  const int own = WPC == 1 ? lane : threadIdx.x;
  long long limit = p.wait_cycles;
  const bool owns = own < CH && q.base + own < q.end;
  const long long so = (long long)q.n * p.D + q.base + own;
  float carry = (p.dsT && owns) ? p.dsT[so] : 0.f;
  constexpr int kBlock = WPC * TL::kTok;
  const int nblk = (len + kBlock - 1) / kBlock;
  const int steps = (nblk + nc - 1) / nc;
  // the first token of the block's and of the thread's step k; blocks before
  // the first token hold none (end below all tokens)
  auto block_at = [&](int k) { return (nblk - 1 - (k * nc + rank)) * kBlock; };
  auto end_at = [&](int tb) { return tb < 0 ? INT_MIN : len; };
  const int off = (WPC == 1 ? 0 : w * TL::kTok) + sub * kR;
  IN in;
  in.start(p, q, tok0, block_at(0) + off);
  if (steps > 0) {
    in.first(slots, block_at(0) + off, end_at(block_at(0)), 0);
    in.fetch_x(slots, in.x, block_at(0) + off, end_at(block_at(0)));
  }
  T *xo = static_cast<T *>(p.dx) +
          ((long long)tok0 + block_at(0) + off) * p.D + q.ch;

  for (int k = 0; k < steps; ++k) {
    const int tb = block_at(k), end = end_at(tb);
    const int t = tb + off;
    const long long tok = (long long)tok0 + t;
    raw_t xr[kR], dr[kR];
    float m[kR][GV], h[kV];
    in.move(-kBlock * nc);
    in.take(slots, k, xr, dr, m, h);
    const int tn = block_at(k + 1);
    if (k + 1 < steps) in.fetch(slots, k + 1, tn + off, end_at(tn), 0);
    Map<GV> f, ex;
#pragma unroll
    for (int v = 0; v < kV; ++v) f.b[v] = 0.f;
#pragma unroll
    for (int v = 0; v < GV; ++v) f.s[v] = 0.f;
    const bool tight = is_tight<GV, GATE>(m);
    float ah[kR][kV];                    // alpha_t h_{t-1}
    auto both = [&](auto tc) {
      if constexpr (GATE != GDR_GATE_NONE) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          float x[kV];
          unpack(in.x_at(slots, r), x);
          factors<GV, GATE, tc.value>(m[r], f.s);
          decay_all<GV, GATE, tc.value>(h, m[r]);
#pragma unroll
          for (int v = 0; v < kV; ++v) ah[r][v] = h[v];
          add_all(h, x);
        }
      }
#pragma unroll
      for (int r = kR - 1; r >= 0; --r) {
        float g[kV];
        unpack(dr[r], g);
        add_all(f.b, g);
        decay_all<GV, GATE, tc.value>(f.b, m[r]);
      }
    };
    if (tight) both(Bool<true>{}); else both(Bool<false>{});
    if (k + 1 < steps) in.fetch_x(slots, in.x, tn + off, end_at(tn));
    const bool runs = is_tight_run<GV, GATE>(f.s, tight);
    to_factors<GV, GATE>(f, runs);
    warp_scan<LANES, GV, GATE, true>(f, ex, runs);
    float cy[kV];
    if constexpr (WPC == 1) {
      float2 mine = make_float2(0.f, 0.f);
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const int src = lane / kV;
        const bool me = lane % kV == v;
        const float b = __shfl_sync(~0u, f.b[v], src);
        const float s = __shfl_sync(~0u, f.s[GV == kV ? v : 0], src);
        if (me) mine = make_float2(s, b);
        cy[v] = __shfl_sync(~0u, carry, c * kV + v);
      }
      carry = apply<GATE>(mine, carry);
    } else {
      post<GV, GATE>(jt, f, c, sub == 0);
      run_maps<CH, GATE, true, CL>(jt, k, nc, rank, limit, p.mute, carry);
#pragma unroll
      for (int v = 0; v < kV; ++v) cy[v] = jt.in[w][c * kV + v];
    }
    enter<LANES, GV, GATE>(cy, ex, runs);
    float dl8[kR];                       // G alpha h, summed over channels
    auto again = [&](auto tc) {
#pragma unroll
      for (int r = kR - 1; r >= 0; --r) {
        float g[kV];
        renew(dr[r]);
        unpack(dr[r], g);
        add_all(cy, g);
        [[maybe_unused]] const int n = t + r < end ? q.nch : 0;
        if constexpr (VEC)
          store<true>(xo + (long long)r * p.D, cy, n);
        else
          in.put(slots, r, cy);
        if constexpr (GATE == GDR_GATE_CHANNEL) {
          float dl[kV];
#pragma unroll
          for (int v = 0; v < kV; ++v) dl[v] = cy[v] * ah[r][v];
          if constexpr (VEC)
            store<true>(p.dla + (tok + r) * p.D + q.ch, dl, n);
          else
            in.put_la(slots, r, dl);
        }
        if constexpr (GATE == GDR_GATE_SCALAR) {
          Pair t = mul2(pair(cy[0], cy[1]), pair(ah[r][0], ah[r][1]));
          t = fma2(pair(cy[2], cy[3]), pair(ah[r][2], ah[r][3]), t);
          float lo, hi;
          split(t, lo, hi);
          dl8[r] = lo + hi;
        }
        decay_all<GV, GATE, tc.value>(cy, m[r]);
      }
    };
    if (tight) again(Bool<true>{}); else again(Bool<false>{});
    if constexpr (GATE == GDR_GATE_SCALAR) {
      // the head's share of this tile, added over the threads of a token in a
      // fixed order; each thread ends with one token's sum
      const int r = sum_tokens<LANES>(dl8, c);
      if (t + r < end && (LANES == 8 || c % 2 == 0)) {
        const long long to = tok + r;
        if (p.nct == 1)
          p.dla[to * p.H + q.head] = dl8[0];
        else
          p.part[((long long)q.ct * p.ntok + to) * p.H + q.head] = dl8[0];
      }
    }
    if constexpr (!VEC) in.flush(slots);
    xo -= (long long)kBlock * nc * p.D;
  }
  if (p.ds0 && owns && rank == 0) p.ds0[so] = carry;
  if constexpr (CL) cg::this_cluster().sync();
}

// Scalar gate, heads of more than one channel tile: the tiles' shares of
// dlog_alpha, added in order; tokens outside every sequence (in order, as they
// have to be, before the first or behind the last) have none.
__global__ void __launch_bounds__(256)
    gdr_linear_dla_kernel(const float *part, float *dla, long long n, int nct,
                          const int32_t *cu, int nseq, int H) {
  prior_done();
  next_may_start();
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  if (cu && (i < (long long)cu[0] * H || i >= (long long)cu[nseq] * H)) return;
  float s = 0.f;
  for (int c = 0; c < nct; ++c) s += part[c * n + i];
  dla[i] = s;
}

// -------------------------------------------------------------------- step

__device__ __forceinline__ float to_float(float f) { return f; }
__device__ __forceinline__ float to_float(__nv_bfloat16 f) {
  return __bfloat162float(f);
}

// A thread has four channels (VEC) or one.
template <typename T, bool VEC, int GATE>
__global__ void __launch_bounds__(128)
    gdr_linear_step_kernel(const T *x, const float *la, const float *sin,
                           float *sout, T *out, long long ldx, int N, int H,
                           int d) {
  constexpr int V = VEC ? kV : 1;
  const int D = H * d, nv = D / V;
  prior_done();
  next_may_start();
  const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
  if (i >= (long long)N * nv) return;
  const long long n = i / nv;
  const int ch = (int)(i - n * nv) * V;
  float xf[kV], h[kV] = {0.f, 0.f, 0.f, 0.f};
  if constexpr (VEC)
    unpack(load(reinterpret_cast<const typename Raw<T>::type *>(
               x + n * ldx + ch)),
           xf);
  else
    xf[0] = to_float(x[n * ldx + ch]);
  if (sin) {   // (may be sout)
    const float *sp = sin + n * D + ch;
    if constexpr (VEC)
      unpack(*reinterpret_cast<const float4 *>(sp), h);
    else
      h[0] = *sp;
  }
  if constexpr (GATE != GDR_GATE_NONE) {
    float g[kV];
    if constexpr (GATE == GDR_GATE_CHANNEL) {
      if constexpr (VEC)
        unpack(load(reinterpret_cast<const float4 *>(la + n * D + ch)), g);
      else
        g[0] = load(la + n * D + ch);
    } else {
      g[0] = load(la + n * H + ch / d);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      h[v] = decay<false>(
          decay_factor<false>(g[GATE == GDR_GATE_CHANNEL ? v : 0]), h[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] += xf[v];
  store<VEC>(out + n * D + ch, h, 1);
  store<VEC>(sout + n * D + ch, h, 1);
}

// ---------------------------------------------------------------- launches

enum Op { kFwd, kBwd, kStep };

// How a call is cut.
struct Plan {
  bool vec;        // rows are aligned for vectors of four channels
  int lanes, wpc;  // a warp's tile is 4 lanes channels wide; warps per chain
  int nc;          // CTAs per chain
  bool early;      // see launch()
};

constexpr int kSms = 148;
gdr_status plan(Op op, const gdr_opts &o, LinParams *p, Plan *pl) {
  const bool bf16 = o.dtype == GDR_BF16, bwd = op == kBwd;
  // one vector must not span two decays
  pl->vec = p->D % kV == 0 && p->ldx % kV == 0 &&
            (o.gate != GDR_GATE_SCALAR || p->d % kV == 0);
  // 64 channels by 16 tokens in the backward pass of bf16, whose tiles then
  // take one shuffle round fewer; of fp32 they would leave room for fewer
  // CTAs, and the forward pass is as fast either way but makes twice the
  // chains
  const int wide = bwd && bf16 && pl->vec ? 16 : 8;
  const int btok = kWarps * kR * 32 / wide;
  // Packed sequences' lengths are on the GPU, so a call is cut by their mean.
  // One long sequence among many short ones is then cut like the short ones:
  // 16384 tokens of 2048 channels, bf16, alone take 55 us forward and 147 in a
  // training step, with 1000 sequences of ten tokens 704 us and 2.4 ms.
  const int avg = p->ntok / p->nseq;
  auto cut = [&](int lanes) {
    pl->lanes = lanes;
    const int ch = kV * lanes;
    // a scalar decay's gradient is summed per head, so its tiles keep to one;
    // so do those of rows that are not aligned
    const bool per_head = o.gate == GDR_GATE_SCALAR && (bwd || !pl->vec);
    p->nct = per_head ? (p->d + ch - 1) / ch : 0;
    p->tiles = per_head ? p->H * p->nct : (p->D + ch - 1) / ch;
    return (long long)p->tiles * p->nseq;
  };
  // Sequences too short for a CTA's tile are run by single warps.  So are, in
  // the forward pass, those up to half as long again, if they alone fill the
  // GPU (32768 tokens of 2048 channels, bf16: 96 tokens each 91 us against
  // 121, 192 tokens 95 against 101, 256 tokens 96 against 84).
  long long chains = cut(8);
  const bool short_seqs =
      2 * avg <= btok || (!bwd && pl->vec && 2 * avg <= 3 * btok &&
                          chains >= 4ll * kSms * kWarps);
  pl->wpc = short_seqs ? 1 : kWarps;
  if (!short_seqs) chains = cut(wide);
  if (chains > INT_MAX / kMaxCluster) return GDR_ERR_UNSUPPORTED;
  p->chains = (int)chains;
  // CTAs per chain: the more, the more of a long sequence is under way at
  // once, but a step then waits for all of them.  Best as long as the launch
  // stays about this big, in CTAs per SM (of which four fit, six without a
  // decay): forward, bf16, 512 chains of 4096 tokens: 1 CTA 85 us, 8 CTAs 113;
  // 64 chains of 65536: 1 CTA 557 us, 8 CTAs 201; backward, a decay per
  // channel, bf16, 1, 2, 4 and 8 CTAs: 256 chains of 4096 167, 208, 175, 163;
  // 288 178, 225, 203, 184; 384 266, 288, 249, 244; 512 403, 349, 324, 321; of
  // 1024 tokens 256 46, 49, 46, 52; 384 71, 68, 66, 74; 512 103, 88, 85, 97 (so
  // this rule is within a seventh of the best of each); a decay per head, 512
  // chains of 2048: 1 CTA 92, 2 101, 8 119.  fp32 gains from more as long as
  // each still has eight steps (forward, a decay per channel, 512 chains of
  // 4096: 1 CTA 148, 4 131; of 1024: 1 CTA 38, 4 41).  Where the decays are
  // most of the traffic, and of fp32, a launch a little larger than what fits
  // loses to a smaller one, its last blocks running almost alone (backward,
  // fp32, 160 chains of 16384: 4 CTAs 371, 2 334).
  const bool channel = o.gate == GDR_GATE_CHANNEL;
  const int few = o.gate == GDR_GATE_NONE ? 6
                  : !bwd                  ? (channel && !bf16 ? 3 : 4)
                  : channel               ? (bf16 ? 14 : 7)
                                          : (bf16 ? 6 : 4);
  const int many = bf16 ? few : bwd ? 7 : 14;
  pl->nc = 1;
  if (pl->wpc > 1)
    while (pl->nc < kMaxCluster && pl->nc * btok < avg &&
           chains * pl->nc * 2 <=
               (16 * pl->nc * btok <= avg ? many : few) * kSms)
      pl->nc *= 2;
  if (bwd && (channel || !bf16) && pl->nc > 1 && chains * pl->nc > 4 * kSms &&
      2 * chains * pl->nc <= 11 * kSms)
    pl->nc /= 2;
  // Blocks that take their places while the launch before ends start sooner,
  // but are not spread evenly, which long ones feel, and those of a launch
  // that leaves room (2048 channels, bf16, a decay per channel, us a call
  // without and with: forward 8 x 512 tokens 16.7 and 13.8, 8 x 1024 25.4 and
  // 23.7, 8 x 4096 84.6 and 88.3; backward 8 x 512 33.6 and 32.4, 1 x 65536
  // 350 and 393; both of 1 x 4000, 256 blocks of the backward pass, 45.7 and
  // 56.4; of 2 x 1350 x 256, 128 blocks, 20.7 and 18.0).
  const long long blocks = chains * pl->nc;
  pl->early = avg <= 8 * pl->nc * btok &&
              (blocks <= kSms || blocks >= 3 * kSms);
  return GDR_OK;
}

template <typename K>
cudaError_t launch_chains(K kernel, int slots, const LinParams &p,
                          const Plan &pl, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, slots);
  if (e != cudaSuccess) return e;
  LinParams q = p;
  q.nc = pl.nc;
  return launch(kernel,
                dim3(pl.wpc == 1 ? (p.chains + kWarps - 1) / kWarps
                                 : p.chains * pl.nc),
                kWarps * 32, slots, pl.nc, pl.early, s, q);
}

template <typename T, bool VEC, int GATE, bool WARP, bool CL>
cudaError_t run4(Op op, const LinParams &p, const Plan &pl, cudaStream_t s) {
  constexpr int kWpc = WARP ? 1 : kWarps;
  constexpr int kWide = !WARP && VEC && sizeof(T) == 2 ? 16 : 8;   // as plan()
  return op == kFwd
             ? launch_chains(gdr_linear_fwd_kernel<T, 8, VEC, GATE, kWpc, CL>,
                             Inputs<T, VEC, GATE, false>::kBytes, p, pl, s)
             : launch_chains(
                   gdr_linear_bwd_kernel<T, kWide, VEC, GATE, kWpc, CL>,
                   Inputs<T, VEC, GATE, true>::kBytes, p, pl, s);
}
template <typename T, bool VEC, int GATE>
cudaError_t run3(Op op, const LinParams &p, const Plan &pl, cudaStream_t s) {
  if (op == kStep) {
    const long long n = (long long)p.nseq * (p.D / (VEC ? kV : 1));
    return launch(gdr_linear_step_kernel<T, VEC, GATE>,
                  dim3((unsigned)((n + 127) / 128)), 128, 0, 1, true,
                  s,
                  static_cast<const T *>(p.x), p.la, p.s0, p.sT,
                  static_cast<T *>(p.out), p.ldx, p.nseq, p.H, p.d);
  }
  return pl.wpc == 1  ? run4<T, VEC, GATE, true, false>(op, p, pl, s)
         : pl.nc == 1 ? run4<T, VEC, GATE, false, false>(op, p, pl, s)
                      : run4<T, VEC, GATE, false, true>(op, p, pl, s);
}
template <typename T, bool VEC>
cudaError_t run2(Op op, int gate, const LinParams &p, const Plan &pl,
                 cudaStream_t s) {
  switch (gate) {
    case GDR_GATE_NONE: return run3<T, VEC, GDR_GATE_NONE>(op, p, pl, s);
    case GDR_GATE_SCALAR: return run3<T, VEC, GDR_GATE_SCALAR>(op, p, pl, s);
    default: return run3<T, VEC, GDR_GATE_CHANNEL>(op, p, pl, s);
  }
}
cudaError_t run(Op op, const gdr_opts &o, const LinParams &p, const Plan &pl,
                cudaStream_t s) {
  if (o.dtype == GDR_BF16)
    return pl.vec ? run2<__nv_bfloat16, true>(op, o.gate, p, pl, s)
                  : run2<__nv_bfloat16, false>(op, o.gate, p, pl, s);
  return pl.vec ? run2<float, true>(op, o.gate, p, pl, s)
                : run2<float, false>(op, o.gate, p, pl, s);
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
  if (ldx > INT_MAX / 2) return GDR_ERR_UNSUPPORTED;
  std::memset(p, 0, sizeof(*p));
  const char *inj = std::getenv("GDR_FAULT_INJECT_LINEAR_TIMEOUT");
  p->mute = inj && inj[0] == '1';
  p->wait_cycles = p->mute ? kInjectWaitCycles : kWaitCycles;
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

}  // namespace

cudaError_t linear_read_error(unsigned *word, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_linear_error, sizeof(unsigned));
  if (e != cudaSuccess) return e;
  if (clear && *word) {
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(g_linear_error, &zero, sizeof(unsigned));
  }
  return e;
}

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
  Plan pl;
  st = plan(kFwd, o, &p, &pl);
  if (st != GDR_OK) return st;
  return run(kFwd, o, p, pl, stream) == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
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
  Plan pl;
  st = plan(kStep, o, &p, &pl);
  if (st != GDR_OK) return st;
  return run(kStep, o, p, pl, stream) == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
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
  Plan plf, pl;
  st = plan(kFwd, o, &pf, &plf);
  if (st == GDR_OK) st = plan(kBwd, o, &p, &pl);
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
    e = run(kFwd, o, pf, plf, stream);
  }
  p.dout = d_out;
  p.dsT = d_final_state;
  p.dx = dx;
  p.dla = d_log_alpha;
  p.part = reinterpret_cast<float *>(static_cast<char *>(ws) + sbytes);
  p.ds0 = d_initial_state;
  if (e == cudaSuccess) e = run(kBwd, o, p, pl, stream);
  if (e == cudaSuccess && parts && p.ntok > 0) {
    const long long nh = (long long)p.ntok * H;   // (within memory: < 2^39)
    e = streaming::launch(gdr_linear_dla_kernel,
                          dim3((unsigned)((nh + 255) / 256)), 256, 0, 1, true,
                          stream, p.part, d_log_alpha, nh, p.nct, p.cu,
                          p.nseq, H);
  }
  const cudaError_t f = ws ? scratch_put(ws, stream) : cudaSuccess;
  return (e == cudaSuccess && f == cudaSuccess) ? GDR_OK : GDR_ERR_CUDA;
}
