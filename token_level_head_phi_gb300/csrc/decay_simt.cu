// Linear attention with a decay for each head on the CUDA cores: float32
// arithmetic for both dtypes (see decay.h for the pass).
//
// One CTA per (unit, segment, slice of at most 64 columns of z) walks its
// segment in 32-token tiles with the state in shared memory.  Per tile: the
// masked, decayed scores (2 x 2 register tiles), the output rows
// (2 tokens x DZ/16 columns) and the state (DX/16 x DZ/16 entries a thread).
#include "common.cuh"
#include "decay.h"
#include "ops.h"

namespace mhla {
namespace {

constexpr int C = 32;  // tokens of a tile
constexpr int kThreads = 256;

template <int DX, int DZS>
struct SimtSmem {
  float x[C][DX + 1];
  float y[C][DX + 1];
  float z[C][DZS];
  float s[DX][DZS];
  float w[C][C + 1];
  float pw[C + 1];  // lambda^n
};

template <typename T, int D>
__device__ __forceinline__ void load_rows(float* dst, int ld, const T* src, int64_t token_stride, const DecayPass& p,
                                          int first, int n, int length) {
  for (int i = threadIdx.x; i < C * D; i += kThreads) {
    const int r = i / D, c = i % D;
    dst[r * ld + c] = r < n ? to_f32(src[decay_token(p, first + r, length) * token_stride + c]) : 0.f;
  }
}

// OUT: the pass itself; otherwise only the segment's own final state.
template <typename T, int DX, int DZS, bool OUT>
__global__ void __launch_bounds__(kThreads) decay_simt_kernel(const DecayPass p) {
  extern __shared__ char raw[];
  SimtSmem<DX, DZS>& sm = *reinterpret_cast<SimtSmem<DX, DZS>*>(raw);
  constexpr int KC = DZS / 16, KA = DX / 16;
  const int unit = blockIdx.x, seg = blockIdx.y, z0 = blockIdx.z * DZS;
  const int b = unit / p.H, h = unit % p.H;
  const int tid = threadIdx.x, tr = tid / 16, tc = tid % 16;
  const float g = p.g[h];
  const int length = decay_length(p, b);
  const int begin = seg * p.seg_len;
  const int end = min(begin + p.seg_len, p.N);         // rows of o this CTA writes
  const int valid = max(0, min(end, length) - begin);  // tokens it takes
  const bool last = seg == (length > 0 ? (length - 1) / p.seg_len : 0);
  const T* x = static_cast<const T*>(p.x) + b * p.sx.batch + h * p.sx.head;
  const T* y = static_cast<const T*>(p.y) + b * p.sy.batch + h * p.sy.head;
  const T* z = static_cast<const T*>(p.z) + b * p.sz.batch + h * p.sz.head + z0;
  T* o = static_cast<T*>(p.o) + b * p.so.batch + h * p.so.head + z0;
  const int64_t state = (int64_t)unit * DX * p.DZ;
  const int64_t one = (int64_t)DX * p.DZ;
  float* segs = p.seg + (p.nseg > 1 ? (int64_t)unit * p.nseg * one : 0);

  if (tid <= C) {
    const float2 w = decay_power(g, tid);
    sm.pw[tid] = w.x + w.y;
  }
  // the state before the segment; s_in may be overwritten by the last
  // segment's CTA, so with several segments the second launch reads the copy
  // that the first one left in the last slot
  const bool copied = OUT && p.nseg > 1;
  for (int i = tid; i < DX * DZS; i += kThreads) {
    const int a = i / DZS, c = i % DZS;
    const int64_t at = (int64_t)a * p.s_ldx + (int64_t)(z0 + c) * p.s_ldz;
    float s = 0.f;
    if (seg == 0 && p.s_in) {
      s = copied ? segs[(p.nseg - 1) * one + at] : p.s_in[state + at];
      if (!OUT) segs[(p.nseg - 1) * one + at] = s;
    }
    if (OUT && valid > 0)
      for (int r = 0; r < seg; ++r) {
        const float2 w = decay_power(g, (seg - 1 - r) * p.seg_len);
        const float u = segs[r * one + at];
        s = fmaf(u, w.x, fmaf(u, w.y, s));
      }
    sm.s[a][c] = s;
  }

  for (int c0 = 0; c0 < valid; c0 += C) {
    const int n = min(C, valid - c0), first = begin + c0;
    __syncthreads();
    if (OUT) load_rows<T, DX>(&sm.x[0][0], DX + 1, x, p.sx.token, p, first, n, length);
    load_rows<T, DX>(&sm.y[0][0], DX + 1, y, p.sy.token, p, first, n, length);
    load_rows<T, DZS>(&sm.z[0][0], DZS, z, p.sz.token, p, first, n, length);
    __syncthreads();
    if (OUT) {
      float d[2][2] = {};
      for (int a = 0; a < DX; ++a) {
        const float x0 = sm.x[2 * tr][a], x1 = sm.x[2 * tr + 1][a];
        const float y0 = sm.y[tc][a], y1 = sm.y[tc + 16][a];
        d[0][0] = fmaf(x0, y0, d[0][0]);
        d[0][1] = fmaf(x0, y1, d[0][1]);
        d[1][0] = fmaf(x1, y0, d[1][0]);
        d[1][1] = fmaf(x1, y1, d[1][1]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int t = 2 * tr + i, u = tc + 16 * j;
          sm.w[t][u] = t >= u ? d[i][j] * (sm.pw[t - u] * p.score) : 0.f;
        }
      // the earlier tokens through the state
      float acc[2][KC] = {};
      for (int a = 0; a < DX; ++a) {
        const float x0 = sm.x[2 * tr][a], x1 = sm.x[2 * tr + 1][a];
#pragma unroll
        for (int k = 0; k < KC; ++k) {
          const float s = sm.s[a][tc + 16 * k];
          acc[0][k] = fmaf(x0, s, acc[0][k]);
          acc[1][k] = fmaf(x1, s, acc[1][k]);
        }
      }
      const float r0 = sm.pw[2 * tr + p.e] * p.read, r1 = sm.pw[2 * tr + 1 + p.e] * p.read;
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        acc[0][k] *= r0;
        acc[1][k] *= r1;
      }
      __syncthreads();
      for (int j = 0; j <= 2 * tr + 1; ++j) {
        const float w0 = sm.w[2 * tr][j], w1 = sm.w[2 * tr + 1][j];
#pragma unroll
        for (int k = 0; k < KC; ++k) {
          const float v = sm.z[j][tc + 16 * k];
          acc[0][k] = fmaf(w0, v, acc[0][k]);
          acc[1][k] = fmaf(w1, v, acc[1][k]);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * tr + i;
        if (t >= n) continue;
        T* row = o + decay_token(p, first + t, length) * p.so.token;
#pragma unroll
        for (int k = 0; k < KC; ++k) row[tc + 16 * k] = from_f32<T>(acc[i][k]);
      }
    }
    // the state behind the tile
    float u[KA][KC] = {};
    for (int j = 0; j < n; ++j) {
      const float w = sm.pw[n - j - p.e] * p.update;
      float zz[KC];
#pragma unroll
      for (int k = 0; k < KC; ++k) zz[k] = sm.z[j][tc + 16 * k];
#pragma unroll
      for (int i = 0; i < KA; ++i) {
        const float yy = sm.y[j][tr + 16 * i] * w;
#pragma unroll
        for (int k = 0; k < KC; ++k) u[i][k] = fmaf(yy, zz[k], u[i][k]);
      }
    }
    if (OUT) __syncthreads();  // every output row has read the state
    const float2 w = decay_power(g, n);
#pragma unroll
    for (int i = 0; i < KA; ++i)
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        float& s = sm.s[tr + 16 * i][tc + 16 * k];
        s = fmaf(s, w.x, fmaf(s, w.y, u[i][k]));
      }
  }
  __syncthreads();
  if (OUT) {
    for (int i = tid; i < (end - begin - valid) * DZS; i += kThreads)
      o[(int64_t)(begin + valid + i / DZS) * p.so.token + i % DZS] = from_f32<T>(0.f);
    if (!last || !p.s_out) return;
    for (int i = tid; i < DX * DZS; i += kThreads) {
      const int a = i / DZS, c = i % DZS;
      p.s_out[state + (int64_t)a * p.s_ldx + (int64_t)(z0 + c) * p.s_ldz] = sm.s[a][c];
    }
  } else if (valid > 0) {
    for (int i = tid; i < DX * DZS; i += kThreads) {
      const int a = i / DZS, c = i % DZS;
      segs[seg * one + (int64_t)a * p.s_ldx + (int64_t)(z0 + c) * p.s_ldz] = sm.s[a][c];
    }
  }
}

template <typename T, int DX, int DZS>
cudaError_t run(const DecayPass& p, cudaStream_t s) {
  constexpr int smem = (int)sizeof(SimtSmem<DX, DZS>);
  const unsigned units = (unsigned)(p.B * p.H), slices = (unsigned)(p.DZ / DZS);
  cudaError_t e;
  if (p.nseg > 1 && (p.launches & 1)) {
    auto* k = decay_simt_kernel<T, DX, DZS, false>;
    if (smem > 48 * 1024 &&
        (e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
      return e;
    k<<<dim3(units, (unsigned)(p.nseg - 1), slices), kThreads, smem, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (!(p.launches & 2)) return cudaSuccess;
  auto* k = decay_simt_kernel<T, DX, DZS, true>;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
    return e;
  k<<<dim3(units, (unsigned)p.nseg, slices), kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int DX>
cudaError_t run_z(const DecayPass& p, cudaStream_t s) {
  if (p.DZ == 16) return run<T, DX, 16>(p, s);
  if (p.DZ == 32) return run<T, DX, 32>(p, s);
  return run<T, DX, 64>(p, s);
}

template <typename T>
cudaError_t run_x(const DecayPass& p, cudaStream_t s) {
  if (p.DX == 16) return run_z<T, 16>(p, s);
  if (p.DX == 32) return run_z<T, 32>(p, s);
  if (p.DX == 64) return run_z<T, 64>(p, s);
  return run_z<T, 128>(p, s);
}

}  // namespace

cudaError_t launch_decay_simt(const DecayPass& p, int dtype, cudaStream_t s) {
  return dtype == MHLA_DTYPE_BF16 ? run_x<__nv_bfloat16>(p, s) : run_x<float>(p, s);
}

}  // namespace mhla
