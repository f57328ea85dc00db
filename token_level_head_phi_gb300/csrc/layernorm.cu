// Layer norm over the last axis, forward and backward ("Layer Normalization",
// section 3): y = (x - mean) rstd w + b.
//
// Forward: a row is held in the registers of G threads (part of a warp, a
// warp or a CTA), read once, and its variance is the mean square deviation
// from the finished mean, so a large mean cancels nothing.  Backward: with
// g = w dy and xh = (x - mean) rstd,
//   dx = rstd (g - mean(g) - xh mean(g xh)),  dw = sum dy xh,  db = sum dy;
// G threads keep the same columns for every row they take, sum dw and db in
// registers, combine inside the CTA through shared memory and write one
// partial row per CTA; a second kernel adds the partial rows in order, so the
// sums do not depend on timing.  Bound: memory (one read of each input, one
// write of each output).  Measured, bf16: 2M rows of 64 forward 90 us = 6.0 TB/s
// (91 % of a copy); 65536 rows of 1024 backward 76 us = 5.3 TB/s (79 %), 8 us
// of it for the second kernel.
#include <cmath>

#include "common.cuh"
#include "ops.h"
#include "tc_host.h"

namespace mhla {
namespace {

struct NormArgs {
  const void *x, *dy, *w, *b;
  void* y;  // dx in the backward pass
  float *mean, *rstd;
  int64_t rows, sx, sy, sdy;
  int cols;
  int w_f32;
  float eps, inv_cols;
  float* partial;  // [CTAs][2][cols] or nullptr
};

// VEC consecutive elements; VEC * sizeof(T) is 16 bytes or VEC is 1.
template <typename T, int VEC>
struct Raw {
  alignas(sizeof(T) * VEC) T v[VEC];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 1)
      v[0] = p[0];
    else
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
  }
  // streaming: read once
  __device__ __forceinline__ void load_once(const T* p) {
    if constexpr (VEC == 1)
      v[0] = p[0];
    else
      *reinterpret_cast<uint4*>(v) = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC == 1)
      p[0] = v[0];
    else
      __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(v));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = from_f32<T>(0.f);
  }
};

// VEC entries of weight or bias from column c on.
template <int VEC>
__device__ __forceinline__ void load_param(const void* p, int is_f32, int c, float (&o)[VEC]) {
  if (is_f32) {
    const float* f = static_cast<const float*>(p) + c;
    if constexpr (VEC % 4 == 0) {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        const float4 t = reinterpret_cast<const float4*>(f)[i];
        o[4 * i] = t.x, o[4 * i + 1] = t.y, o[4 * i + 2] = t.z, o[4 * i + 3] = t.w;
      }
    } else {
      o[0] = f[0];
    }
  } else {
    const __nv_bfloat16* f = static_cast<const __nv_bfloat16*>(p) + c;
    if constexpr (VEC % 4 == 0) {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        const uint2 t = reinterpret_cast<const uint2*>(f)[i];
        o[4 * i] = __uint_as_float(t.x << 16), o[4 * i + 1] = __uint_as_float(t.x & 0xffff0000u);
        o[4 * i + 2] = __uint_as_float(t.y << 16), o[4 * i + 3] = __uint_as_float(t.y & 0xffff0000u);
      }
    } else {
      o[0] = __bfloat162float(f[0]);
    }
  }
}

// Sums of R rows' pairs over the G threads of a row (every thread gets them).
// G > 32: the whole CTA, behind one barrier through `sh`, which the caller
// alternates between uses.
template <int G, int R>
__device__ __forceinline__ void row_sums2(float2 (&v)[R], float2 (*sh)[32]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1) {
      v[r].x += __shfl_xor_sync(0xffffffffu, v[r].x, o);
      v[r].y += __shfl_xor_sync(0xffffffffu, v[r].y, o);
    }
  if constexpr (G > 32) {
    constexpr int W = G / 32;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if ((threadIdx.x & 31) == 0) sh[r][threadIdx.x >> 5] = v[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v[r] = sh[r][(threadIdx.x & 31) & (W - 1)];
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) {
        v[r].x += __shfl_xor_sync(0xffffffffu, v[r].x, o);
        v[r].y += __shfl_xor_sync(0xffffffffu, v[r].y, o);
      }
    }
  }
}

template <int G>
__device__ __forceinline__ float row_sum(float v, float* sh) {
#pragma unroll
  for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh[(threadIdx.x & 31) & (W - 1)];
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// Threads of a CTA: a whole row for G > 32, several rows otherwise.
template <int G>
constexpr int norm_threads = G > 32 ? G : 128;

// A row in the registers of G threads, E vectors each; R rows at a time per
// group so that short rows keep enough loads in flight.
template <typename T, int VEC, int G, int E, int R>
__global__ void __launch_bounds__(norm_threads<G>) norm_fwd_kernel(const NormArgs a) {
  constexpr int kThreads = norm_threads<G>;
  constexpr int kGroups = kThreads / G;
  __shared__ float sh[2][32];
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const int nv = a.cols / VEC;
  const int64_t row0 = (int64_t)blockIdx.x * (kGroups * R) + group;
  Raw<T, VEC> raw[R][E];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t row = row0 + r * kGroups;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = lane + e * G;
      if (row < a.rows && i < nv)
        raw[r][e].load_once(static_cast<const T*>(a.x) + row * a.sx + (int64_t)i * VEC);
      else
        raw[r][e].zero();
    }
  }
  float mean[R], rstd[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += to_f32(raw[r][e].v[j]);
    mean[r] = row_sum<G>(s, sh[0]) * a.inv_cols;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (lane + e * G < nv)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d = to_f32(raw[r][e].v[j]) - mean[r];
          s = fmaf(d, d, s);
        }
    rstd[r] = rsqrtf(row_sum<G>(s, sh[1]) * a.inv_cols + a.eps);
    const int64_t row = row0 + r * kGroups;
    if (lane == 0 && row < a.rows) {
      if (a.mean) a.mean[row] = mean[r];
      if (a.rstd) a.rstd[row] = rstd[r];
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = lane + e * G;
    if (i >= nv) continue;
    float w[VEC], b[VEC];
    if (a.w) load_param<VEC>(a.w, a.w_f32, i * VEC, w);
    if (a.b) load_param<VEC>(a.b, a.w_f32, i * VEC, b);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = row0 + r * kGroups;
      if (row >= a.rows) continue;
      Raw<T, VEC> o;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float y = (to_f32(raw[r][e].v[j]) - mean[r]) * rstd[r];
        if (a.w) y *= w[j];
        if (a.b) y += b[j];
        o.v[j] = from_f32<T>(y);
      }
      o.store(static_cast<T*>(a.y) + row * a.sy + (int64_t)i * VEC);
    }
  }
}

// Rows longer than a CTA's registers: one CTA per row, three passes over it
// (the second and third mostly from L2).
template <typename T, int VEC>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(const NormArgs a) {
  __shared__ float sh[2][32];
  const int nv = a.cols / VEC;
  const T* x = static_cast<const T*>(a.x) + blockIdx.x * a.sx;
  T* y = static_cast<T*>(a.y) + blockIdx.x * a.sy;
  Raw<T, VEC> raw;
  float s = 0.f;
  for (int i = threadIdx.x; i < nv; i += 1024) {
    raw.load(x + (int64_t)i * VEC);
#pragma unroll
    for (int j = 0; j < VEC; ++j) s += to_f32(raw.v[j]);
  }
  const float mean = row_sum<1024>(s, sh[0]) * a.inv_cols;
  s = 0.f;
  for (int i = threadIdx.x; i < nv; i += 1024) {
    raw.load(x + (int64_t)i * VEC);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float d = to_f32(raw.v[j]) - mean;
      s = fmaf(d, d, s);
    }
  }
  const float rstd = rsqrtf(row_sum<1024>(s, sh[1]) * a.inv_cols + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[blockIdx.x] = mean;
    if (a.rstd) a.rstd[blockIdx.x] = rstd;
  }
  for (int i = threadIdx.x; i < nv; i += 1024) {
    raw.load(x + (int64_t)i * VEC);
    float w[VEC], b[VEC];
    if (a.w) load_param<VEC>(a.w, a.w_f32, i * VEC, w);
    if (a.b) load_param<VEC>(a.b, a.w_f32, i * VEC, b);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      float t = (to_f32(raw.v[j]) - mean) * rstd;
      if (a.w) t *= w[j];
      if (a.b) t += b[j];
      raw.v[j] = from_f32<T>(t);
    }
    raw.store(y + (int64_t)i * VEC);
  }
}

template <int G>
constexpr int norm_bwd_threads = G > 32 ? G : 256;

// dx of a row in the registers of G threads; dw and db of their columns over
// every row that the group takes.
template <typename T, int VEC, int G, int E, int R>
__global__ void __launch_bounds__(norm_bwd_threads<G>) norm_bwd_kernel(const NormArgs a) {
  constexpr int kThreads = norm_bwd_threads<G>;
  constexpr int kGroups = kThreads / G;
  __shared__ float2 sh[2][R][32];
  extern __shared__ float acc[];  // [2][cols], only for partial sums of several groups
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const int nv = a.cols / VEC;
  float dw[E][VEC], db[E][VEC];
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[e][j] = db[e][j] = 0.f;

  float w[E][VEC];  // of this thread's columns
#pragma unroll
  for (int e = 0; e < E; ++e) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[e][j] = 1.f;
    if (a.w && lane + e * G < nv) load_param<VEC>(a.w, a.w_f32, (lane + e * G) * VEC, w[e]);
  }

  // The next rows are on their way while the current ones are reduced and
  // written: their raw registers are free once xh and g are formed.
  Raw<T, VEC> rx[R][E], rg[R][E];
  float mean[R], rstd[R];
  auto fetch = [&](int64_t base) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = base + group + r * kGroups;
      const bool live = row < a.rows;
      mean[r] = live ? a.mean[row] : 0.f;
      rstd[r] = live ? a.rstd[row] : 0.f;
      const T* x = static_cast<const T*>(a.x) + row * a.sx + lane * VEC;
      const T* dy = static_cast<const T*>(a.dy) + row * a.sdy + lane * VEC;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (live && lane + e * G < nv) {
          rx[r][e].load_once(x + e * G * VEC);
          rg[r][e].load_once(dy + e * G * VEC);
        } else {  // adds nothing to any sum
          rx[r][e].zero();
          rg[r][e].zero();
        }
      }
    }
  };
  int turn = 0;  // alternates the exchange slots, so one barrier per turn is enough
  const int64_t stride = (int64_t)gridDim.x * (kGroups * R);
  int64_t base = (int64_t)blockIdx.x * (kGroups * R);
  if (base < a.rows) fetch(base);
  // every thread of the CTA makes the same number of turns
  for (; base < a.rows; base += stride) {
    float xh[R][E][VEC], g[R][E][VEC], scale[R];
    float2 sum[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      sum[r] = make_float2(0.f, 0.f);
      scale[r] = rstd[r];
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d = to_f32(rg[r][e].v[j]), z = (to_f32(rx[r][e].v[j]) - mean[r]) * rstd[r];
          dw[e][j] = fmaf(d, z, dw[e][j]);
          db[e][j] += d;
          xh[r][e][j] = z;
          g[r][e][j] = d * w[e][j];
          sum[r].x += g[r][e][j];
          sum[r].y = fmaf(g[r][e][j], z, sum[r].y);
        }
    }
    if (base + stride < a.rows) fetch(base + stride);
    row_sums2<G, R>(sum, sh[turn]);
    turn ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = base + group + r * kGroups;
      if (row >= a.rows) continue;
      const float c1 = sum[r].x * a.inv_cols * scale[r], c2 = sum[r].y * a.inv_cols * scale[r];
      T* dx = static_cast<T*>(a.y) + row * a.sy + lane * VEC;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (lane + e * G >= nv) continue;
        Raw<T, VEC> o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) o.v[j] = from_f32<T>(fmaf(g[r][e][j], scale[r], -fmaf(xh[r][e][j], c2, c1)));
        o.store(dx + e * G * VEC);
      }
    }
  }
  if (!a.partial) return;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // norm_reduce_kernel, which waits for all of this

  // groups that share a warp hold the same columns in lanes G apart
  if constexpr (G < 32) {
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
#pragma unroll
        for (int o = 16; o >= G; o >>= 1) {
          dw[e][j] += __shfl_xor_sync(0xffffffffu, dw[e][j], o);
          db[e][j] += __shfl_xor_sync(0xffffffffu, db[e][j], o);
        }
  }
  float* out = a.partial + (int64_t)blockIdx.x * 2 * a.cols;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = lane + e * G;
      if (i >= nv) continue;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        out[i * VEC + j] = dw[e][j];
        out[a.cols + i * VEC + j] = db[e][j];
      }
    }
  } else {
    const int warp = threadIdx.x >> 5;
    const bool first = (threadIdx.x & 31) < G;  // one copy per warp
    for (int wv = 0; wv < kThreads / 32; ++wv) {
      if (warp == wv && first) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int i = lane + e * G;
          if (i >= nv) continue;
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int c = i * VEC + j;
            acc[c] = wv ? acc[c] + dw[e][j] : dw[e][j];
            acc[a.cols + c] = wv ? acc[a.cols + c] + db[e][j] : db[e][j];
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * a.cols; c += kThreads) out[c] = acc[c];
  }
}

// Rows longer than a CTA's registers: dx with one CTA per row.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(const NormArgs a) {
  __shared__ float2 sh[1][32];
  const int nv = a.cols / VEC;
  const T* x = static_cast<const T*>(a.x) + blockIdx.x * a.sx;
  const T* dy = static_cast<const T*>(a.dy) + blockIdx.x * a.sdy;
  T* dx = static_cast<T*>(a.y) + blockIdx.x * a.sy;
  const float mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
  float2 sum[1] = {make_float2(0.f, 0.f)};
  float2& s = sum[0];
  Raw<T, VEC> rx, rg;
  float w[VEC];
  for (int i = threadIdx.x; i < nv; i += 1024) {
    rx.load(x + (int64_t)i * VEC);
    rg.load(dy + (int64_t)i * VEC);
    if (a.w) load_param<VEC>(a.w, a.w_f32, i * VEC, w);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float xh = (to_f32(rx.v[j]) - mean) * rstd;
      float g = to_f32(rg.v[j]);
      if (a.w) g *= w[j];
      s.x += g;
      s.y = fmaf(g, xh, s.y);
    }
  }
  row_sums2<1024, 1>(sum, sh);
  const float c1 = s.x * a.inv_cols, c2 = s.y * a.inv_cols;
  for (int i = threadIdx.x; i < nv; i += 1024) {
    rx.load(x + (int64_t)i * VEC);
    rg.load(dy + (int64_t)i * VEC);
    if (a.w) load_param<VEC>(a.w, a.w_f32, i * VEC, w);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float xh = (to_f32(rx.v[j]) - mean) * rstd;
      float g = to_f32(rg.v[j]);
      if (a.w) g *= w[j];
      rx.v[j] = from_f32<T>(rstd * (g - c1 - xh * c2));
    }
    rx.store(dx + (int64_t)i * VEC);
  }
}

// dw and db of long rows: a thread per column, each grid row a share of the rows.
template <typename T>
__global__ void __launch_bounds__(256) norm_bwd_columns_kernel(const NormArgs a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float dw = 0.f, db = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float g = to_f32(static_cast<const T*>(a.dy)[row * a.sdy + c]);
    const float xh = (to_f32(static_cast<const T*>(a.x)[row * a.sx + c]) - a.mean[row]) * a.rstd[row];
    dw = fmaf(g, xh, dw);
    db += g;
  }
  float* out = a.partial + (int64_t)blockIdx.y * 2 * a.cols;
  out[c] = dw;
  out[a.cols + c] = db;
}

// Adds the partial rows: 32 columns per CTA, 32 threads to a column, each
// every 32nd row in order, then the 32 sums in order.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* partial, int parts, int cols, float* dweight,
                                                           float* dbias) {
  __shared__ float sh[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;  // over [2][cols]
  float s = 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c < 2 * cols)
#pragma unroll 12
    for (int p = ty; p < parts; p += 32) s += partial[(int64_t)p * 2 * cols + c];
  sh[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && c < 2 * cols) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += sh[i][tx];
    if (c < cols) {
      if (dweight) dweight[c] = t;
    } else if (dbias) {
      dbias[c - cols] = t;
    }
  }
}

// ---------------------------------------------------------------- dispatch

// Runs f.template go<VEC, G, E, R>() with the smallest group of threads that
// holds a row: 16-byte vectors where rows allow it (VEC = 16 / sizeof(T)),
// single elements otherwise.
template <typename T, typename F>
mhla_status with_fwd_shape(int cols, bool vec, F&& f) {
  constexpr int W = 16 / sizeof(T);
  if (vec) {
    const int nv = cols / W;
    if (nv <= 2) return f.template go<W, 2, 1, 4>();
    if (nv <= 4) return f.template go<W, 4, 1, 4>();
    if (nv <= 8) return f.template go<W, 8, 1, 4>();
    if (nv <= 16) return f.template go<W, 16, 1, 4>();
    if (nv <= 32) return f.template go<W, 32, 1, 4>();
    if (nv <= 64) return f.template go<W, 32, 2, 2>();
    if (nv <= 128) return f.template go<W, 32, 4, 1>();
    if (nv <= 512) return f.template go<W, 128, 4, 1>();
    if (nv <= 1024) return f.template go<W, 256, 4, 1>();
    if (nv <= 2048) return f.template go<W, 512, 4, 1>();
    return f.template go_long<W>();
  }
  if (cols <= 8) return f.template go<1, 8, 1, 4>();
  if (cols <= 32) return f.template go<1, 32, 1, 4>();
  if (cols <= 128) return f.template go<1, 32, 4, 1>();
  if (cols <= 512) return f.template go<1, 32, 16, 1>();
  if (cols <= 2048) return f.template go<1, 128, 16, 1>();
  if (cols <= 8192) return f.template go<1, 512, 16, 1>();
  return f.template go_long<1>();
}

template <typename T, typename F>
mhla_status with_bwd_shape(int cols, bool vec, F&& f) {
  constexpr int W = 16 / sizeof(T);
  if (vec) {
    const int nv = cols / W;
    if (nv <= 2) return f.template go<W, 2, 1, 2>();
    if (nv <= 4) return f.template go<W, 4, 1, 2>();
    if (nv <= 8) return f.template go<W, 8, 1, 2>();
    if (nv <= 16) return f.template go<W, 16, 1, 2>();
    if (nv <= 32) return f.template go<W, 32, 1, 2>();
    if (nv <= 64) return f.template go<W, 64, 1, 2>();
    if (nv <= 128) return f.template go<W, 128, 1, 2>();
    if (nv <= 256) return f.template go<W, 256, 1, 2>();
    if (nv <= 512) return f.template go<W, 512, 1, 1>();
    if (nv <= 1024) return f.template go<W, 512, 2, 1>();
    if (nv <= 2048) return f.template go<W, 512, 4, 1>();
    return f.template go_long<W>();
  }
  if (cols <= 8) return f.template go<1, 8, 1, 2>();
  if (cols <= 32) return f.template go<1, 32, 1, 2>();
  if (cols <= 128) return f.template go<1, 32, 4, 2>();
  if (cols <= 512) return f.template go<1, 128, 4, 2>();
  if (cols <= 2048) return f.template go<1, 256, 8, 1>();
  if (cols <= 8192) return f.template go<1, 512, 16, 1>();
  return f.template go_long<1>();
}

template <typename T>
struct Forward {
  const NormArgs& a;
  cudaStream_t s;
  template <int VEC, int G, int E, int R>
  mhla_status go() {
    constexpr int rows = norm_threads<G> / G * R;
    const int64_t blocks = (a.rows + rows - 1) / rows;
    norm_fwd_kernel<T, VEC, G, E, R><<<(unsigned)blocks, norm_threads<G>, 0, s>>>(a);
    return launch_status();
  }
  template <int VEC>
  mhla_status go_long() {
    norm_fwd_long_kernel<T, VEC><<<(unsigned)a.rows, 1024, 0, s>>>(a);
    return launch_status();
  }
};

// Partial rows of dw and db that the backward pass of these sizes writes:
// one for each of the CTAs that are resident at once (512 to 640 threads on
// every SM), or 64 shares of the rows.
constexpr int kLongShares = 64;
struct Parts {
  const NormArgs& a;
  int64_t n = 0;
  template <int VEC, int G, int E, int R>
  mhla_status go() {
    constexpr int rows = norm_bwd_threads<G> / G * R;
    constexpr int64_t per_sm = (norm_bwd_threads<G> <= 128 ? 640 : 512) / norm_bwd_threads<G>;  // registers allow it
    n = (a.rows + rows - 1) / rows;
    if (n > per_sm * kOpsSms) n = per_sm * kOpsSms;
    return MHLA_OK;
  }
  template <int VEC>
  mhla_status go_long() {
    n = a.rows < kLongShares ? a.rows : kLongShares;
    return MHLA_OK;
  }
};

template <typename T>
struct Backward {
  const NormArgs& a;
  cudaStream_t s;
  int64_t parts;
  template <int VEC, int G, int E, int R>
  mhla_status go() {
    const size_t smem = norm_bwd_threads<G> > G && a.partial ? 2 * sizeof(float) * (size_t)a.cols : 0;
    norm_bwd_kernel<T, VEC, G, E, R><<<(unsigned)parts, norm_bwd_threads<G>, smem, s>>>(a);
    return launch_status();
  }
  template <int VEC>
  mhla_status go_long() {
    // the column sums first: dx may overwrite dy or x
    if (a.partial)
      norm_bwd_columns_kernel<T><<<dim3((unsigned)((a.cols + 255) / 256), (unsigned)parts), 256, 0, s>>>(a);
    norm_bwd_long_kernel<T, VEC><<<(unsigned)a.rows, 1024, 0, s>>>(a);
    return launch_status();
  }
};

mhla_status check_params(const mhla_layernorm_params* p) {
  if (!p || p->rows < 0 || p->cols < 1 || !ops_dtype_ok(p->dtype) || !ops_dtype_ok(p->weight_dtype))
    return MHLA_ERR_INVALID_ARG;
  if (!std::isfinite(p->eps) || p->eps < 0.f) return MHLA_ERR_INVALID_ARG;
  if (p->cols > (1 << 20) || p->rows > 0x7fffffff) return MHLA_ERR_UNSUPPORTED;
  return MHLA_OK;
}

RowTensor matrix(const void* ptr, const mhla_layernorm_params* p, int64_t stride) {
  return row_tensor(ptr, 1, 1, p->rows, mhla_strides{0, 0, stride}, p->cols, ops_elem(p->dtype));
}

bool param_aligned(const void* ptr) { return (uintptr_t)ptr % 16 == 0; }

NormArgs args_of(const mhla_layernorm_params* p) {
  NormArgs a = {};
  a.rows = p->rows;
  a.cols = p->cols;
  a.w_f32 = p->weight_dtype == MHLA_DTYPE_F32;
  a.eps = p->eps;
  a.inv_cols = 1.f / (float)p->cols;
  return a;
}

// Partial rows whatever the pointers' alignment: the larger of what the
// vector and the scalar kernels write.
int64_t most_parts(const mhla_layernorm_params* p) {
  const NormArgs a = args_of(p);
  Parts v{a}, e{a};
  const int w = 16 / (int)ops_elem(p->dtype);
  if (p->dtype == MHLA_DTYPE_BF16) {
    if (p->cols % w == 0) with_bwd_shape<__nv_bfloat16>(p->cols, true, v);
    with_bwd_shape<__nv_bfloat16>(p->cols, false, e);
  } else {
    if (p->cols % w == 0) with_bwd_shape<float>(p->cols, true, v);
    with_bwd_shape<float>(p->cols, false, e);
  }
  return v.n > e.n ? v.n : e.n;
}

}  // namespace
}  // namespace mhla

extern "C" {

mhla_status mhla_layernorm_forward(const void* x, const void* weight, const void* bias,
                                   const mhla_layernorm_params* p, void* y, float* mean, float* rstd, void* stream) {
  using namespace mhla;
  mhla_status st = check_params(p);
  if (st != MHLA_OK) return st;
  if (p->rows == 0) return MHLA_OK;
  const RowTensor tx = matrix(x, p, p->x_stride), ty = matrix(y, p, p->y_stride);
  const size_t we = ops_elem(p->weight_dtype);
  const RowTensor others[4] = {flat_tensor(weight, weight ? p->cols : 0, we), flat_tensor(bias, bias ? p->cols : 0, we),
                               flat_tensor(mean, mean ? p->rows : 0, 4), flat_tensor(rstd, rstd ? p->rows : 0, 4)};
  if (!row_tensor_ok(tx, true) || !row_tensor_ok(ty, true)) return MHLA_ERR_INVALID_ARG;
  for (const RowTensor& t : others)
    if (!row_tensor_ok(t, false) || !row_tensors_apart(t, ty)) return MHLA_ERR_INVALID_ARG;
  if (!row_tensors_same(tx, ty) && !row_tensors_apart(tx, ty)) return MHLA_ERR_INVALID_ARG;
  for (int i = 2; i < 4; ++i) {  // mean and rstd are written
    if (!row_tensors_apart(others[i], tx) || !row_tensors_apart(others[i], others[0]) ||
        !row_tensors_apart(others[i], others[1]))
      return MHLA_ERR_INVALID_ARG;
  }
  if (!row_tensors_apart(others[2], others[3])) return MHLA_ERR_INVALID_ARG;
  NormArgs a = args_of(p);
  a.x = x;
  a.y = y;
  a.w = weight;
  a.b = bias;
  a.mean = mean;
  a.rstd = rstd;
  a.sx = p->x_stride;
  a.sy = p->y_stride;
  const int w = 16 / (int)ops_elem(p->dtype);
  const bool vec = p->cols % w == 0 && row_alignment(tx, 16) == 16 && row_alignment(ty, 16) == 16 &&
                   param_aligned(weight) && param_aligned(bias);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->dtype == MHLA_DTYPE_BF16) return with_fwd_shape<__nv_bfloat16>(p->cols, vec, Forward<__nv_bfloat16>{a, s});
  return with_fwd_shape<float>(p->cols, vec, Forward<float>{a, s});
}

mhla_status mhla_layernorm_backward_workspace_bytes(const mhla_layernorm_params* p, size_t* bytes) {
  using namespace mhla;
  if (!bytes) return MHLA_ERR_INVALID_ARG;
  const mhla_status st = check_params(p);
  if (st != MHLA_OK) return st;
  *bytes = (size_t)most_parts(p) * 2 * sizeof(float) * (size_t)p->cols;
  return MHLA_OK;
}

mhla_status mhla_layernorm_backward(const void* dy, const void* x, const void* weight, const float* mean,
                                    const float* rstd, const mhla_layernorm_params* p, void* dx, float* dweight,
                                    float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace mhla;
  mhla_status st = check_params(p);
  if (st != MHLA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t we = ops_elem(p->weight_dtype);
  const RowTensor tw = flat_tensor(weight, weight ? p->cols : 0, we);
  const RowTensor tdw = flat_tensor(dweight, dweight ? p->cols : 0, 4), tdb = flat_tensor(dbias, dbias ? p->cols : 0, 4);
  if (!row_tensor_ok(tdw, true) || !row_tensor_ok(tdb, true) || !row_tensors_apart(tdw, tdb) ||
      !row_tensors_apart(tdw, tw) || !row_tensors_apart(tdb, tw))
    return MHLA_ERR_INVALID_ARG;
  if (p->rows == 0) {  // an empty sum
    cudaError_t e = cudaSuccess;
    if (dweight) e = cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)p->cols, s);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, sizeof(float) * (size_t)p->cols, s);
    return e == cudaSuccess ? MHLA_OK : record_cuda_error(e);
  }
  const RowTensor tx = matrix(x, p, p->x_stride), ty = matrix(dy, p, p->dy_stride), td = matrix(dx, p, p->y_stride);
  const RowTensor tm = flat_tensor(mean, p->rows, 4), tr = flat_tensor(rstd, p->rows, 4);
  if (!row_tensor_ok(tx, true) || !row_tensor_ok(ty, true) || !row_tensor_ok(td, true) || !row_tensor_ok(tw, false) ||
      !row_tensor_ok(tm, false) || !row_tensor_ok(tr, false))
    return MHLA_ERR_INVALID_ARG;
  if (!row_tensors_same(tx, td) && !row_tensors_apart(tx, td)) return MHLA_ERR_INVALID_ARG;
  if (!row_tensors_same(ty, td) && !row_tensors_apart(ty, td)) return MHLA_ERR_INVALID_ARG;
  const RowTensor* written[3] = {&td, &tdw, &tdb};
  for (const RowTensor* o : written)
    if (!row_tensors_apart(*o, tm) || !row_tensors_apart(*o, tr)) return MHLA_ERR_INVALID_ARG;
  for (int i = 1; i < 3; ++i)
    if (!row_tensors_apart(*written[i], tx) || !row_tensors_apart(*written[i], ty) ||
        !row_tensors_apart(*written[i], td))
      return MHLA_ERR_INVALID_ARG;
  if (!row_tensors_apart(td, tw)) return MHLA_ERR_INVALID_ARG;
  NormArgs a = args_of(p);
  a.x = x;
  a.dy = dy;
  a.w = weight;
  a.y = dx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.sx = p->x_stride;
  a.sy = p->y_stride;
  a.sdy = p->dy_stride;
  const bool sums = dweight || dbias;
  size_t need = 0;
  Scratch scratch;
  if (sums) {
    if ((st = mhla_layernorm_backward_workspace_bytes(p, &need)) != MHLA_OK) return st;
    const RowTensor tws = flat_tensor(workspace, workspace ? (int64_t)need : 0, 1);
    const RowTensor* all[8] = {&tx, &ty, &td, &tw, &tm, &tr, &tdw, &tdb};
    for (const RowTensor* t : all)
      if (!row_tensors_apart(tws, *t)) return MHLA_ERR_INVALID_ARG;
    if ((st = scratch.take(workspace, workspace_bytes, need, s)) != MHLA_OK) return st;
    a.partial = reinterpret_cast<float*>(scratch.ptr());
  }
  const int w = 16 / (int)ops_elem(p->dtype);
  const bool vec = p->cols % w == 0 && row_alignment(tx, 16) == 16 && row_alignment(ty, 16) == 16 &&
                   row_alignment(td, 16) == 16 && param_aligned(weight);
  Parts parts{a};
  if (p->dtype == MHLA_DTYPE_BF16) {
    with_bwd_shape<__nv_bfloat16>(p->cols, vec, parts);
    st = with_bwd_shape<__nv_bfloat16>(p->cols, vec, Backward<__nv_bfloat16>{a, s, parts.n});
  } else {
    with_bwd_shape<float>(p->cols, vec, parts);
    st = with_bwd_shape<float>(p->cols, vec, Backward<float>{a, s, parts.n});
  }
  if (st == MHLA_OK && sums) {
    const cudaError_t e =
        (cudaError_t)launch_pdl(norm_reduce_kernel, dim3((unsigned)((2 * p->cols + 31) / 32)), dim3(1024), 0, s,
                                (const float*)a.partial, (int)parts.n, (int)p->cols, dweight, dbias);
    if (e != cudaSuccess) st = record_cuda_error(e);
  }
  return scratch.give_back(st);
}

}  // extern "C"
