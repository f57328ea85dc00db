// Linear attention with a decay for each head on the CUDA cores: float32
// arithmetic for both dtypes (see decay.h for the pass).
//
// One CTA of 256 threads per (unit, segment, slice of at most 64 columns of z)
// walks its segment in 64-token tiles with the state in shared memory.  A
// thread keeps 4 x 4 entries of the scores, 4 tokens x DZ/16 columns of the
// output and DX/16 x DZ/16 entries of the state in registers, and reads its
// operands as 16-byte vectors along the contraction: bound by the float32
// units, not by shared memory (64 products for 8 vector reads).  Measured: 32k
// tokens x 64 heads of 64, float32, 2.40 ms; 2k tokens x 60 heads of 128 0.58 ms.
#include "common.cuh"
#include "decay.h"
#include "ops.h"
#include "tc_host.h"

namespace mhla {
namespace {

constexpr int C = 64;  // tokens of a tile
constexpr int kThreads = 256;

// Rows of x and y are 4 floats longer than they need be: eight neighbouring
// rows start in eight different groups of four banks.
template <int DX, int DZS>
struct alignas(16) SimtSmem {
  float x[C][DX + 4];
  float y[C][DX + 4];
  float z[C][DZS];
  float s[DX][DZS];
  float w[C][C + 4];
  float pw[C + 4];  // lambda^n
};

// N consecutive floats of shared memory.
template <int N>
__device__ __forceinline__ void read_n(const float* p, float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 t = reinterpret_cast<const float4*>(p)[i];
      v[4 * i] = t.x, v[4 * i + 1] = t.y, v[4 * i + 2] = t.z, v[4 * i + 3] = t.w;
    }
  } else if constexpr (N == 2) {
    const float2 t = *reinterpret_cast<const float2*>(p);
    v[0] = t.x, v[1] = t.y;
  } else {
    v[0] = p[0];
  }
}

template <typename T, int D>
__device__ __forceinline__ void load_rows(float* dst, int ld, const T* src, int64_t token_stride, const DecayPass& p,
                                          int first, int n, int length) {
  if (p.vec) {
    constexpr int V = 16 / sizeof(T), kPieces = D / V;
#pragma unroll 4
    for (int i = threadIdx.x; i < C * kPieces; i += kThreads) {
      const int r = i / kPieces, c = i % kPieces * V;
      alignas(16) T v[V];
      if (r < n) *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(src + decay_token(p, first + r, length) * token_stride + c);
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n) f = make_float4(to_f32(v[j]), to_f32(v[j + 1]), to_f32(v[j + 2]), to_f32(v[j + 3]));
        *reinterpret_cast<float4*>(dst + r * ld + c + j) = f;
      }
    }
    return;
  }
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
  if (!OUT) decay_dependents();
  // the state before the segment: the first launch starts every one from zero
  if (OUT && p.nseg > 1) decay_wait();
  const float* before = !OUT ? nullptr : p.nseg > 1 ? segs + seg * one : p.s_in ? p.s_in + state : nullptr;
  for (int i = tid; i < DX * DZS; i += kThreads) {
    const int a = i / DZS, c = i % DZS;
    sm.s[a][c] = before ? before[(int64_t)a * p.s_ldx + (int64_t)(z0 + c) * p.s_ldz] : 0.f;
  }

  for (int c0 = 0; c0 < valid; c0 += C) {
    const int n = min(C, valid - c0), first = begin + c0;
    __syncthreads();
    if (OUT) load_rows<T, DX>(&sm.x[0][0], DX + 4, x, p.sx.token, p, first, n, length);
    load_rows<T, DX>(&sm.y[0][0], DX + 4, y, p.sy.token, p, first, n, length);
    load_rows<T, DZS>(&sm.z[0][0], DZS, z, p.sz.token, p, first, n, length);
    __syncthreads();
    if (OUT) {
      // scores of tokens 4 tr .. 4 tr + 3 against tokens tc, tc + 16, ...
      float d[4][4] = {};
      const int groups = min(4, tr / 4 + 1);  // later groups of 16 lie above the diagonal
#pragma unroll 2
      for (int a = 0; a < DX; a += 4) {
        float xv[4][4], yv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) read_n<4>(&sm.x[4 * tr + i][a], xv[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j >= groups) break;
          read_n<4>(&sm.y[tc + 16 * j][a], yv);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) d[i][j] = fmaf(xv[i][q], yv[q], d[i][j]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = 4 * tr + i, u = tc + 16 * j;
          sm.w[t][u] = t >= u ? d[i][j] * (sm.pw[t - u] * p.score) : 0.f;
        }
      // the earlier tokens through the state
      float acc[4][KC] = {};
#pragma unroll 2
      for (int a = 0; a < DX; a += 4) {
        float xv[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) read_n<4>(&sm.x[4 * tr + i][a], xv[i]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float sv[KC];
          read_n<KC>(&sm.s[a + q][KC * tc], sv);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < KC; ++k) acc[i][k] = fmaf(xv[i][q], sv[k], acc[i][k]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float r = sm.pw[4 * tr + i + p.e] * p.read;
#pragma unroll
        for (int k = 0; k < KC; ++k) acc[i][k] *= r;
      }
      __syncthreads();  // the scores are there, and every output row has read the state
      for (int j = 0; j < 4 * tr + 4; j += 4) {
        float wv[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) read_n<4>(&sm.w[4 * tr + i][j], wv[i]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float zv[KC];
          read_n<KC>(&sm.z[j + q][KC * tc], zv);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < KC; ++k) acc[i][k] = fmaf(wv[i][q], zv[k], acc[i][k]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * tr + i;
        if (t >= n) continue;
        T* row = o + decay_token(p, first + t, length) * p.so.token + KC * tc;
        if (sizeof(T) * KC == 16 && p.vec) {
          alignas(16) T v[KC];
#pragma unroll
          for (int k = 0; k < KC; ++k) v[k] = from_f32<T>(acc[i][k]);
          if constexpr (sizeof(T) * KC == 16) *reinterpret_cast<uint4*>(row) = *reinterpret_cast<uint4*>(v);
        } else {
#pragma unroll
          for (int k = 0; k < KC; ++k) row[k] = from_f32<T>(acc[i][k]);
        }
      }
    }
    // the state behind the tile: rows KA tr .. and columns KC tc ..
    float u[KA][KC] = {};
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const float w = sm.pw[n - j - p.e] * p.update;
      float yv[KA], zv[KC];
      read_n<KA>(&sm.y[j][KA * tr], yv);
      read_n<KC>(&sm.z[j][KC * tc], zv);
#pragma unroll
      for (int k = 0; k < KC; ++k) zv[k] *= w;
#pragma unroll
      for (int i = 0; i < KA; ++i)
#pragma unroll
        for (int k = 0; k < KC; ++k) u[i][k] = fmaf(yv[i], zv[k], u[i][k]);
    }
    const float2 w = decay_power(g, n);
#pragma unroll
    for (int i = 0; i < KA; ++i)
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        float& s = sm.s[KA * tr + i][KC * tc + k];
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
      segs[(seg + 1) * one + (int64_t)a * p.s_ldx + (int64_t)(z0 + c) * p.s_ldz] = sm.s[a][c];
    }
  }
}

template <typename T, int DX, int DZS>
cudaError_t run(const DecayPass& p, cudaStream_t s) {
  constexpr int smem = (int)sizeof(SimtSmem<DX, DZS>);
  static_assert(decay_simt_resident(DX, DZS) * (smem + 1024) <= 228 * 1024, "");
  const unsigned units = (unsigned)(p.B * p.H), slices = (unsigned)(p.DZ / DZS);
  cudaError_t e;
  if (p.nseg > 1 && (p.launches & 1)) {
    auto* k = decay_simt_kernel<T, DX, DZS, false>;
    if (smem > 48 * 1024 &&
        (e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
      return e;
    k<<<dim3(units, (unsigned)(p.nseg - 1), slices), kThreads, smem, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_decay_scan(p, s)) != cudaSuccess) return e;
  }
  if (!(p.launches & 2)) return cudaSuccess;
  auto* k = decay_simt_kernel<T, DX, DZS, true>;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
    return e;
  if (p.nseg > 1) return (cudaError_t)launch_pdl(k, dim3(units, (unsigned)p.nseg, slices), dim3(kThreads), smem, s, p);
  k<<<dim3(units, 1, slices), kThreads, smem, s>>>(p);
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
