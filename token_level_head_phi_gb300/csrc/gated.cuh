// Linear recurrence with gates of each token and channel: what its kernels share.
//   h_t = a_t h_{t-1} + c_t u_t,   u_t = x_t sigma(i_t)
//   a_t = exp(log_decay sigma(r_t)) or sigma(r_t),   c_t = sqrt(1 - a_t^2), 1 - a_t or 1
// and its gradients: with G_t = dout_t + a_{t+1} G_{t+1},
//   dlog a_t = G_t (a_t h_{t-1} + u_t dc_t / dlog a_t),   du_t = G_t c_t.
// Both recurrences are scans of the maps h -> A h + H, which compose.
//
// A CTA takes 64 channels of one sequence, in tiles of 64 tokens: a warp 8
// tokens, a lane two channels, whose values are one register pair and one
// instruction.  Each warp forms the map of its 8 tokens in registers, the maps
// meet in shared memory behind one barrier, and a second walk over the same
// tokens writes the results from the state that the warp starts with.  Every
// input is read once.  Where sequences and channels are few, a cluster of CTAs
// takes successive tiles of the same channels at once and exchanges the tiles'
// maps through distributed shared memory.
#pragma once

#include "common.cuh"
#include "ops.h"
#include "pack.cuh"

namespace mhla {

constexpr int kGatedTok = 8;        // tokens of a warp
constexpr int kGatedWarps = 8;      // warps of a CTA
constexpr int kGatedTile = kGatedTok * kGatedWarps;
constexpr int kGatedSlab = 64;      // channels of a CTA
constexpr int kGatedCluster = 8;    // most CTAs of a cluster
static_assert(kGatedTile == MHLA_GATED_MARK, "a tile starts at a mark");
// CTAs that an SM holds: their registers, and the shared memory of float32's
// backward pass.
constexpr int gated_resident(bool f32, bool backward) { return backward ? (f32 ? 1 : 2) : (f32 ? 2 : 3); }

struct GatedArgs {
  const void *x, *r, *i, *dout;
  void *out, *dx, *dr, *di;
  mhla_strides sx, sr, si, so, sdo, sdx, sdr, sdi;
  const float* g;  // log_decay [D]
  const int32_t* lengths;
  const float *state_in, *dstate_out;
  float *state_out, *dstate_in;
  float* marks;    // [B][n_marks][D]
  float* partial;  // [B][cluster][D], sums for log_decay's gradient
  int B, N, D, n_marks, slabs;
  int scale;
  int vec;  // both channels of a lane in one access
};

// Launches return a status.
mhla_status launch_gated_fwd(const GatedArgs& a, int dtype, int kind, cudaStream_t s);
mhla_status launch_gated_bwd(const GatedArgs& a, int dtype, int kind, cudaStream_t s);
mhla_status launch_gated_step(const GatedArgs& a, int dtype, int kind, cudaStream_t s);

#ifdef __CUDACC__

// What the gates of two channels make, as pairs of float32.
struct Gates {
  uint64_t gap;   // 1 - a
  uint64_t s;     // sigma(r)
  uint64_t less;  // 1 - sigma(r)
  uint64_t q;     // sigma(i); 1 without an input gate
};

// sigma(r) = 1 / (1 + 2^-(r log2 e)), one reciprocal for both gates; the
// powers stay below 2^62, so their product does not overflow and sigma not
// below 2^-62.
//
// a is formed as 1 + expm1(log a): its rounding (2^-25 next to 1) is multiplied
// with itself over all the tokens that a slow channel remembers, so a float32
// exponential's last bit, which errs to one side, would show (the final state
// of 32k tokens 4.5e-6 off instead of 3e-7).  expm1 is its Taylor series above
// -1/4 (the first term left out is x^7 / 5040, 5e-8 of the sum) and 2^(x log2
// e) - 1 below.  `g`: log_decay, at most 0.
template <int KIND, bool IN>
__device__ __forceinline__ Gates gates_of(uint64_t r, uint64_t i, uint64_t g) {
  const uint64_t one = splat(1.f), minus = splat(-1.f);
  Gates o;
  const float2 f = unpair(mul2(r, splat(-kLog2e)));
  const uint64_t e = pair(ex2(least(f.x, 62.f)), ex2(least(f.y, 62.f))), e1 = add2(e, one);
  if constexpr (IN) {
    const float2 h = unpair(mul2(i, splat(-kLog2e)));
    const uint64_t k1 = add2(pair(ex2(least(h.x, 62.f)), ex2(least(h.y, 62.f))), one);
    const float2 d = unpair(mul2(e1, k1));
    const uint64_t inv = pair(rcp(d.x), rcp(d.y));
    o.s = mul2(inv, k1);
    o.q = mul2(inv, e1);
  } else {
    const float2 d = unpair(e1);
    o.s = pair(rcp(d.x), rcp(d.y));
    o.q = one;
  }
  o.less = mul2(e, o.s);
  if constexpr (KIND == MHLA_GATED_DECAY) {
    const uint64_t x = mul2(g, o.s);
    uint64_t t = fma2(x, splat(-1.f / 720.f), splat(-1.f / 120.f));
    t = fma2(x, t, splat(-1.f / 24.f));
    t = fma2(x, t, splat(-1.f / 6.f));
    t = fma2(x, t, splat(-0.5f));
    t = fma2(x, t, minus);
    const float2 near = unpair(mul2(x, t)), at = unpair(x), y = unpair(mul2(x, splat(kLog2e)));
    const float2 far = unpair(fma2(pair(ex2(y.x), ex2(y.y)), minus, one));
    o.gap = pair(at.x > -0.25f ? near.x : far.x, at.y > -0.25f ? near.y : far.y);
  } else {
    o.gap = o.less;
  }
  return o;
}

__device__ __forceinline__ uint64_t decay_of(uint64_t gap) { return fma2(gap, splat(-1.f), splat(1.f)); }

__device__ __forceinline__ int gated_length(const GatedArgs& p, int b) {
  if (!p.lengths) return p.N;
  const int n = p.lengths[b];
  return n < 0 ? 0 : n > p.N ? p.N : n;
}

// Two neighbouring channels of a row.
template <typename T>
using Two = Pack<T, 2>;
__device__ __forceinline__ uint64_t wide(const Two<__nv_bfloat16>& x) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(x.v);
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint64_t wide(const Two<float>& x) { return pair(x.v[0], x.v[1]); }
__device__ __forceinline__ Two<__nv_bfloat16> narrow(uint64_t x, __nv_bfloat16) {
  const float2 f = unpair(x);
  const __nv_bfloat162 y = __floats2bfloat162_rn(f.x, f.y);
  Two<__nv_bfloat16> o;
  *reinterpret_cast<uint32_t*>(o.v) = *reinterpret_cast<const uint32_t*>(&y);
  return o;
}
__device__ __forceinline__ Two<float> narrow(uint64_t x, float) {
  const float2 f = unpair(x);
  Two<float> o;
  o.v[0] = f.x;
  o.v[1] = f.y;
  return o;
}

// A lane's two channels.
struct Lane {
  int ch, n;  // n: of them inside the row
  __device__ __forceinline__ Lane(int slab, int D) {
    ch = slab * kGatedSlab + 2 * (threadIdx.x & 31);
    n = min(max(D - ch, 0), 2);
  }
  // entries of a float32 vector; zeros where it is NULL and outside
  __device__ __forceinline__ uint64_t get(const float* p) const {
    return pair(p && n > 0 ? p[ch] : 0.f, p && n > 1 ? p[ch + 1] : 0.f);
  }
  __device__ __forceinline__ void put(float* p, uint64_t v) const {
    const float2 f = unpair(v);
    if (n > 0) p[ch] = f.x;
    if (n > 1) p[ch + 1] = f.y;
  }
};

// ------------------------------------------------------- clusters of CTAs

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ int cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The map h -> A h + H of two channels.
struct __align__(16) Map {
  uint64_t A, H;
};
__device__ __forceinline__ Map same() { return Map{splat(1.f), splat(0.f)}; }
__device__ __forceinline__ Map then(Map first, Map next) {
  return Map{mul2(next.A, first.A), fma2(next.A, first.H, next.H)};
}
__device__ __forceinline__ uint64_t through(Map m, uint64_t h) { return fma2(m.A, h, m.H); }
__device__ __forceinline__ Map load_map(const Map* p) {
  const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
  return Map{v.x, v.y};
}
__device__ __forceinline__ void store_map(Map* p, Map m) { *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(m.A, m.H); }

// Stores m to the same place of CTA `rank`'s shared memory.
__device__ __forceinline__ void send(Map* place, int rank, Map m) {
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(place);
  uint32_t there;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(mine), "r"(rank));
  asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(there), "l"(m.A), "l"(m.H) : "memory");
}

// What a warp of CTA `rank` (of `ranks`) starts its tokens with, and what all
// the cluster's tiles make of `carry`.  REVERSE: the last warp of the last CTA
// comes first.  `turn` alternates, so one barrier a call is enough.
template <bool REVERSE>
struct Scan {
  Map maps[2][kGatedWarps][32];
  Map tiles[2][kGatedCluster][32];

  __device__ __forceinline__ uint64_t run(int turn, int rank, int ranks, Map map, uint64_t* carry) {
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    store_map(&maps[turn][w][l], map);
    __syncthreads();
    Map before = same(), all = before;
#pragma unroll
    for (int i = 0; i < kGatedWarps; ++i) {
      const int v = REVERSE ? kGatedWarps - 1 - i : i;
      if (v == w) before = all;
      all = then(all, load_map(&maps[turn][v][l]));
    }
    uint64_t start = *carry;
    if (ranks == 1) {
      *carry = through(all, start);
      return through(before, start);
    }
    if (w < ranks) send(&tiles[turn][rank][l], w, all);
    cluster_arrive();
    cluster_wait();
    const int place = REVERSE ? ranks - 1 - rank : rank;  // of this CTA in the order
    uint64_t h = start;
#pragma unroll
    for (int i = 0; i < kGatedCluster; ++i) {
      if (i == place) start = h;
      if (i < ranks) h = through(load_map(&tiles[turn][REVERSE ? ranks - 1 - i : i][l]), h);
    }
    *carry = h;
    return through(before, start);
  }
};

#endif

// CTAs of a cluster: the power of two with the fewest rounds of tiles, counted
// over the waves of CTAs that the GPU holds at once; of equal ones the smallest.
inline int gated_cluster(int64_t units, int tokens, int resident) {
  const int64_t slots = (int64_t)kOpsSms * resident, tiles = ((int64_t)tokens + kGatedTile - 1) / kGatedTile;
  int64_t best = 0;
  int c = 1;
  for (int n = 1; n <= kGatedCluster; n *= 2) {
    const int64_t cost = (units * n + slots - 1) / slots * ((tiles + n - 1) / n);
    if (n == 1 || cost < best) {
      best = cost;
      c = n;
    }
  }
  return c;
}

#ifdef __CUDACC__
template <typename K>
mhla_status launch_gated_clusters(K kernel, const GatedArgs& a, int resident, size_t smem, cudaStream_t s) {
  const int64_t units = (int64_t)a.B * a.slabs;
  const int cluster = gated_cluster(units, a.N, resident);
  if (units * cluster > 0x7fffffff) return MHLA_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cluster));
  cfg.blockDim = dim3(32 * kGatedWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e == cudaSuccess ? launch_status() : record_cuda_error(e);
}

// f.template go<T, KIND, IN>() for the arguments.
template <typename F>
mhla_status with_gates(const GatedArgs& a, int dtype, int kind, F&& f) {
  if (dtype == MHLA_DTYPE_BF16) {
    if (kind == MHLA_GATED_DECAY)
      return a.i ? f.template go<__nv_bfloat16, MHLA_GATED_DECAY, true>()
                 : f.template go<__nv_bfloat16, MHLA_GATED_DECAY, false>();
    return a.i ? f.template go<__nv_bfloat16, MHLA_GATED_SIGMOID, true>()
               : f.template go<__nv_bfloat16, MHLA_GATED_SIGMOID, false>();
  }
  if (kind == MHLA_GATED_DECAY)
    return a.i ? f.template go<float, MHLA_GATED_DECAY, true>() : f.template go<float, MHLA_GATED_DECAY, false>();
  return a.i ? f.template go<float, MHLA_GATED_SIGMOID, true>() : f.template go<float, MHLA_GATED_SIGMOID, false>();
}
#endif

}  // namespace mhla
