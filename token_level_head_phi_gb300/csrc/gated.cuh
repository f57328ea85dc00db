// Linear recurrence with gates of each token and channel: what its kernels share.
//   h_t = a_t h_{t-1} + c_t u_t,   u_t = x_t sigma(i_t)
//   a_t = exp(log_decay sigma(r_t)) or sigma(r_t),   c_t = sqrt(1 - a_t^2), 1 - a_t or 1
// and its gradients: with G_t = dout_t + a_{t+1} G_{t+1},
//   dlog a_t = G_t (a_t h_{t-1} + u_t dc_t / dlog a_t),   du_t = G_t c_t.
// Both recurrences are scans of the maps h -> A h + H, which compose.
//
// A CTA takes 64 channels of one sequence, tile by tile: a warp 16 tokens (8 in
// the backward pass and of float32), a lane two channels, whose values are one
// register pair and one instruction.  Each warp forms the map of its tokens,
// takes the state from the warp before it, hands its own on and then walks over
// the same tokens again for the results: the warps of a CTA run after one
// another without a barrier for all of them.  Every input is read once, by
// asynchronous copies into shared memory of the warp's own, a round ahead.
// Where sequences and channels are few, a cluster of CTAs takes successive tiles
// of the same channels at once and exchanges the tiles' maps through distributed
// shared memory.  Rows of whole 16 bytes have kernels of their own, without the
// code for others (64 x 512 tokens of 4096 channels backward 470 us with it, 389
// without).
#pragma once

#include "common.cuh"
#include "ops.h"
#include "pack.cuh"

namespace mhla {

constexpr int kGatedWarps = 8;    // warps of a CTA
constexpr int kGatedSlab = 64;    // channels of a CTA
constexpr int kGatedCluster = 8;  // most CTAs of a cluster
// tokens of a warp and of a CTA's tile
template <bool F32, bool BACKWARD>
constexpr int kGatedTok = BACKWARD || F32 ? 8 : 16;
// A kernel for rows that start at pairs or at single elements of bf16; of float32
// each has one of its own (5 x 1999 x 1009 backward 101 us, in one 115; bf16 pairs,
// 1010 channels, 71 us in one, 85 apart, where registers spill).
constexpr int kGatedNarrow = -1;
inline int gated_tile(bool f32, bool backward) { return kGatedWarps * (backward || f32 ? 8 : 16); }
// CTAs that an SM holds: for their registers, and the shared memory of float32's
// backward pass.
constexpr int gated_resident(bool f32) { return f32 ? 1 : 2; }

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
  int vec;  // rows start at multiples of 16 bytes (2), of a pair of elements (1) or of one (0)
};

// Launches return a status.
mhla_status launch_gated_fwd(const GatedArgs& a, int dtype, int kind, cudaStream_t s);
mhla_status launch_gated_bwd(const GatedArgs& a, int dtype, int kind, cudaStream_t s);
mhla_status launch_gated_step(const GatedArgs& a, int dtype, int kind, cudaStream_t s);

#ifdef __CUDACC__

// What the gates of two channels make, as pairs of float32.
struct Gates {
  float2 a;
  float2 m;     // a - 1
  float2 s;     // sigma(r)
  float2 less;  // 1 - sigma(r)
  float2 q;     // sigma(i); not set without an input gate
};

// sigma(r) = 1 / (1 + 2^-(r log2 e)), one reciprocal for both gates.  r is taken
// as at least -43 (least_gate), so the powers' product does not overflow, and
// sigma as at least 2e-19.
//
// Next to 1, a is formed as 1 + expm1(log a): its rounding (2^-25 there) is
// multiplied with itself over all the tokens that a slow channel remembers, so a
// float32 exponential's last bit, which errs to one side, would show (the final
// state of 32k tokens 4.5e-6 off instead of 3e-7).  Above log a = -1/8, expm1 is y
// times a cubic in y = log2 a, fitted for the least largest relative error (2e-8)
// with ln 2 as its first coefficient.  Below, a is the power itself, so that a small
// one has all of its digits, and m = a - 1; sigmoids likewise, where 1 - sigma is
// formed by itself: 1 - (1 - sigma) down to 7/8, sigma below.  `g2`: log_decay log2
// e, at most 0.
template <int KIND, bool IN>
__device__ __forceinline__ Gates gates_of(float2 r, float2 i, float2 g2) {
  Gates o;
  const float2 f = mulc(r, kLog2e);
  const float2 e = make_float2(ex2(-f.x), ex2(-f.y)), e1 = addc(e, 1.f);
  if constexpr (IN) {
    const float2 h = mulc(i, kLog2e);
    const float2 k1 = addc(make_float2(ex2(-h.x), ex2(-h.y)), 1.f);
    const float2 d = mul2(e1, k1);
    const float2 inv = make_float2(rcp(d.x), rcp(d.y));
    o.s = mul2(inv, k1);
    o.q = mul2(inv, e1);
  } else {
    o.s = make_float2(rcp(e1.x), rcp(e1.y));
  }
  o.less = mul2(e, o.s);
  if constexpr (KIND == MHLA_GATED_DECAY) {
    const float2 y = mul2(o.s, g2);  // log2 a
    float2 t = fma2(y, splat(9.17151198e-3f), splat(5.54584153e-2f));
    t = fmac(y, t, 0.240225211f);
    t = fmac(y, t, 0.693147182f);
    const float2 near = mul2(y, t), slow = addc(near, 1.f);
    const float2 power = make_float2(ex2(y.x), ex2(y.y)), gap = addc(power, -1.f);
    const bool one = y.x > -0.1803369f, two = y.y > -0.1803369f;
    o.a = make_float2(one ? slow.x : power.x, two ? slow.y : power.y);
    o.m = make_float2(one ? near.x : gap.x, two ? near.y : gap.y);
  } else {
    const float2 slow = add2(splat(1.f), make_float2(-o.less.x, -o.less.y));
    o.a = make_float2(o.less.x < 0.125f ? slow.x : o.s.x, o.less.y < 0.125f ? slow.y : o.s.y);
    o.m = make_float2(-o.less.x, -o.less.y);
  }
  return o;
}

// c of two channels: sqrt(1 - a^2), or k0 + k1 m: 1 or 1 - a.
template <bool NORM>
__device__ __forceinline__ float2 factor(float2 m, float2 k1, float2 k0) {
  if constexpr (!NORM) return fma2(m, k1, k0);
  const float2 v = mul2(m, addc(m, 2.f));
  return make_float2(root(-v.x), root(-v.y));
}

__device__ __forceinline__ int gated_length(const GatedArgs& p, int b) {
  if (!p.lengths) return p.N;
  const int n = p.lengths[b];
  return n < 0 ? 0 : n > p.N ? p.N : n;
}

// Two neighbouring channels of a row.
template <typename T>
using Two = Pack<T, 2>;
__device__ __forceinline__ float2 wide(const Two<__nv_bfloat16>& x) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(x.v);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 wide(const Two<float>& x) { return make_float2(x.v[0], x.v[1]); }
__device__ __forceinline__ Two<__nv_bfloat16> narrow(float2 x, __nv_bfloat16) {
  const __nv_bfloat162 y = __floats2bfloat162_rn(x.x, x.y);
  Two<__nv_bfloat16> o;
  *reinterpret_cast<uint32_t*>(o.v) = *reinterpret_cast<const uint32_t*>(&y);
  return o;
}
__device__ __forceinline__ Two<float> narrow(float2 x, float) {
  Two<float> o;
  o.v[0] = x.x;
  o.v[1] = x.y;
  return o;
}

// A gate's value, NaN kept, not below where sigma is taken to end.
__device__ __forceinline__ float2 least_gate(const Two<__nv_bfloat16>& x) {
  const __nv_bfloat162 end = __float2bfloat162_rn(-43.f);
  const __nv_bfloat162 y = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(x.v), end);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&y);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 least_gate(const Two<float>& x) {
  return make_float2(most(x.v[0], -43.f), most(x.v[1], -43.f));
}

// A lane's two channels.
struct Lane {
  int ch, n;  // n: of them inside the row
  __device__ __forceinline__ Lane(int slab, int D) {
    ch = slab * kGatedSlab + 2 * (threadIdx.x & 31);
    n = min(max(D - ch, 0), 2);
  }
  // entries of a float32 vector; zeros where it is NULL and outside
  __device__ __forceinline__ float2 get(const float* p) const {
    return make_float2(p && n > 0 ? p[ch] : 0.f, p && n > 1 ? p[ch + 1] : 0.f);
  }
  __device__ __forceinline__ void put(float* p, float2 v) const {
    if (n > 0) p[ch] = v.x;
    if (n > 1) p[ch + 1] = v.y;
  }
};

// ------------------------------------------------- a warp's shared memory

// TOK rows of a slab, of one warp.
template <typename T, int TOK>
struct Rows {
  Two<T> v[TOK][32];
  __device__ __forceinline__ T* single(int row, int i) { return &v[row][i / 2].v[i % 2]; }
  __device__ __forceinline__ const T* single(int row, int i) const { return &v[row][i / 2].v[i % 2]; }
  static constexpr int kPiece = 16 / sizeof(T), kPieces = kGatedSlab / kPiece;  // of a row
  static constexpr int kAtOnce = 32 / kPieces;                                  // rows of one access of the warp
};

// A lane's way through the rows of a slab in global memory.
template <typename T, typename P>
struct Walk {
  // of the lane: its piece of one of the first rows (vec 2); of the first row its
  // two channels (1), or one of two elements that are 32 apart (0)
  P* at;
  int64_t stride;
  using R1 = Rows<T, 1>;

  __device__ __forceinline__ Walk(P* slab, int64_t stride, int vec) : stride(stride) {
    const int l = threadIdx.x & 31;
    at = slab + (vec == 2 ? l / R1::kPieces * stride + l % R1::kPieces * R1::kPiece : vec == 1 ? 2 * l : l);
  }

  // Starts copies of the rows from `t0` on; zeros where they have no `rows` or
  // the row ends (`cols` entries).  `fast`: there are TOK whole ones, vec is 2.
  template <int TOK>
  __device__ __forceinline__ void fetch(Rows<T, TOK>& to, int t0, bool fast, int rows, int cols, int vec) const {
    const int l = threadIdx.x & 31;
    const T* from = at + t0 * stride;
    if (fast) {
      Two<T>* place = &to.v[l / R1::kPieces][l % R1::kPieces * (R1::kPiece / 2)];
#pragma unroll
      for (int i = 0; i < TOK / R1::kAtOnce; ++i, from += R1::kAtOnce * stride)
        copy_async<16>(place + i * R1::kAtOnce * 32, from, 16);
    } else if (vec == 2) {
      const int row = l / R1::kPieces, col = l % R1::kPieces * R1::kPiece;
      const int left = min(max(cols - col, 0), R1::kPiece) * (int)sizeof(T);
      for (int i = 0; i < TOK / R1::kAtOnce; ++i, from += R1::kAtOnce * stride) {
        Two<T>* place = &to.v[row + i * R1::kAtOnce][col / 2];
        if (row + i * R1::kAtOnce < rows && left)
          copy_async<16>(place, from, left);
        else
          *reinterpret_cast<uint4*>(place) = make_uint4(0, 0, 0, 0);
      }
    } else if (vec == 1) {
      // columns that are not there are lanes of their own, whose values nobody uses
      const int n = min(max(cols - 2 * l, 0), 2) * (int)sizeof(T);
      if (n && rows >= TOK) {
#pragma unroll
        for (int i = 0; i < TOK; ++i, from += stride) copy_async<2 * sizeof(T)>(&to.v[i][l], from, n);
      } else if (n) {
        const T* some = from;
#pragma unroll 4
        for (int i = 0; i < TOK; ++i, from += stride)
          copy_async<2 * sizeof(T)>(&to.v[i][l], i < rows ? from : some, i < rows ? n : 0);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        const T* at = from + c;
        if (c + l >= cols) continue;
        if constexpr (sizeof(T) == 4) {
          if (rows >= TOK) {
#pragma unroll
            for (int i = 0; i < TOK; ++i, at += stride) copy_async<4>(to.single(i, c + l), at, 4);
          } else {
            const T* some = at;
#pragma unroll 4
            for (int i = 0; i < TOK; ++i, at += stride)
              copy_async<4>(to.single(i, c + l), i < rows ? at : some, i < rows ? 4 : 0);
          }
        } else if (rows >= TOK) {  // no copies of 2 bytes: all rows into registers, then on
          T v[TOK];
#pragma unroll
          for (int i = 0; i < TOK; ++i, at += stride) v[i] = *at;
#pragma unroll
          for (int i = 0; i < TOK; ++i) *to.single(i, c + l) = v[i];
        } else {
#pragma unroll 4
          for (int i = 0; i < TOK; ++i, at += stride) *to.single(i, c + l) = i < rows ? *at : from_f32<T>(0.f);
        }
      }
    }
  }

  // Writes the rows from `t0` on, as far as there are `rows` and columns.
  template <int TOK>
  __device__ __forceinline__ void write(const Rows<T, TOK>& from, int t0, bool fast, int rows, int cols,
                                        int vec) const {
    const int l = threadIdx.x & 31;
    P* to = at + t0 * stride;
    if (vec == 2) {
      __syncwarp();
      const int row = l / R1::kPieces, col = l % R1::kPieces * R1::kPiece;
      const Two<T>* place = &from.v[row][col / 2];
      if (fast) {
#pragma unroll
        for (int i = 0; i < TOK / R1::kAtOnce; ++i, to += R1::kAtOnce * stride)
          __stcs(reinterpret_cast<uint4*>(to), *reinterpret_cast<const uint4*>(place + i * R1::kAtOnce * 32));
      } else {
        for (int i = 0; i < TOK / R1::kAtOnce; ++i, to += R1::kAtOnce * stride) {
          Pack<T, R1::kPiece> o;
          *reinterpret_cast<uint4*>(o.v) = *reinterpret_cast<const uint4*>(place + i * R1::kAtOnce * 32);
          if (row + i * R1::kAtOnce < rows) o.store(to, col + R1::kPiece <= cols, cols - col);
        }
      }
      __syncwarp();  // before the next copies arrive here
    } else if (vec == 1) {
      const bool whole = 2 * l + 1 < cols;
      if (2 * l >= cols) return;
      Two<T> v[TOK];
#pragma unroll
      for (int i = 0; i < TOK; ++i) v[i] = from.v[i][l];
      if (rows >= TOK && whole) {
#pragma unroll
        for (int i = 0; i < TOK; ++i, to += stride) v[i].store(to, true);
      } else {
#pragma unroll
        for (int i = 0; i < TOK; ++i, to += stride)
          if (i < rows) v[i].store(to, whole, cols - 2 * l);
      }
    } else {
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        P* at = to + c;
        if (c + l >= cols) continue;
        T v[TOK];
#pragma unroll
        for (int i = 0; i < TOK; ++i) v[i] = *from.single(i, c + l);
        if (rows >= TOK) {
#pragma unroll
          for (int i = 0; i < TOK; ++i, at += stride) *at = v[i];
        } else {
#pragma unroll
          for (int i = 0; i < TOK; ++i, at += stride)
            if (i < rows) *at = v[i];
        }
      }
      __syncwarp();
    }
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
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The map h -> A h + H of two channels.
struct __align__(16) Map {
  float2 A, H;
};
__device__ __forceinline__ Map same() { return Map{splat(1.f), splat(0.f)}; }
__device__ __forceinline__ Map then(Map first, Map next) {
  return Map{mul2(next.A, first.A), fma2(next.A, first.H, next.H)};
}
__device__ __forceinline__ float2 through(Map m, float2 h) { return fma2(m.A, h, m.H); }
__device__ __forceinline__ Map load_map(const Map* p) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  return Map{make_float2(v.x, v.y), make_float2(v.z, v.w)};
}
__device__ __forceinline__ void store_map(Map* p, Map m) {
  *reinterpret_cast<float4*>(p) = make_float4(m.A.x, m.A.y, m.H.x, m.H.y);
}

// Stores m to the same place of CTA `rank`'s shared memory.
__device__ __forceinline__ void send(Map* place, int rank, Map m) {
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(place);
  uint32_t there;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(mine), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(there), "f"(m.A.x), "f"(m.A.y), "f"(m.H.x),
               "f"(m.H.y)
               : "memory");
}

// Barrier `id` (1 .. 15) between two warps of a CTA: one has written, the other
// reads.
__device__ __forceinline__ void hand_over(int id) {
  asm volatile("barrier.cta.arrive.aligned %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ void take_over(int id) {
  asm volatile("barrier.cta.sync.aligned %0, 64;" ::"r"(id) : "memory");
}

#endif

// Clusters of n = 1 .. 8 CTAs that the GPU holds at once, with one or two CTAs to
// an SM: as cudaOccupancyMaxActiveClusters says, since a cluster stays inside a
// part of the GPU.
inline int gated_clusters(int n, int resident) {
  static constexpr int held[2][kGatedCluster] = {{152, 76, 46, 36, 28, 23, 15, 15}, {304, 152, 97, 74, 58, 46, 38, 36}};
  return held[resident - 1][n - 1];
}

// CTAs of a cluster: the number with the least time, counted in rounds of tiles
// over the waves of clusters that the GPU holds at once; of equal ones the
// smallest.  A round takes 1.8 us (backward 2.4) of a CTA alone on its SM, 3.2
// (3.9) of two alone on one SM and 4.1 to 5.2 (4.7) in a cluster, whose warps wait
// for the maps of all of its tiles.  5 x 1999 tokens of 1024 channels forward take 29
// us alone, 32 in pairs, 25 in threes and 28 in eights; backward 76, 74, 53 and
// 59; 16 x 256 tokens forward 8.5 alone and 13 in pairs; 3 x 777 of 321 float32
// channels 30 alone, 12 in sixes and 16 in eights, of which only 15 fit.
inline int gated_cluster(int64_t units, int tokens, bool f32, bool backward) {
  const int tile = gated_tile(f32, backward), resident = gated_resident(f32);
  const int64_t tiles = ((int64_t)tokens + tile - 1) / tile;
  int64_t best = 0;
  int c = 1;
  for (int n = 1; n <= kGatedCluster; ++n) {
    const int held = gated_clusters(n, resident);
    int round = 8;
    if (n > 1)
      round = backward ? 15 : 20;
    else if (resident > 1 && units > kOpsSms)
      round = backward ? 13 : 14;
    const int64_t cost = (units + held - 1) / held * ((tiles + n - 1) / n) * round;
    if (n == 1 || cost < best) {
      best = cost;
      c = n;
    }
  }
  return c;
}

#ifdef __CUDACC__
template <typename K>
mhla_status launch_gated_clusters(K kernel, const GatedArgs& a, bool f32, bool backward, size_t smem, cudaStream_t s) {
  const int64_t units = (int64_t)a.B * a.slabs;
  const int cluster = gated_cluster(units, a.N, f32, backward);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return record_cuda_error(e);
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
  e = cudaLaunchKernelEx(&cfg, kernel, a);
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
