// Linear attention with a decay for each head: what its kernels share.
//
// Every direction is one causal pass over three sequences x, y (rows of DX
// entries) and z, o (rows of DZ entries) with a carried DX x DZ state:
//   o_i = read * lambda^(i + e) S^T x_i + score * sum_{j <= i} lambda^(i - j) (x_i . y_j) z_j
//   S  <- lambda^n S + update * sum_j lambda^(n - j - e) y_j z_j^T     over n tokens
// with
//            x   y   z   o   e  score  read   update  direction
//   forward  q   k   v   out 1  scale  scale  1       first token first
//   dq       do  v   k   dq  1  scale  scale  1       first token first, S transposed
//   dk       v   do  q   dk  0  scale  1      scale   last token first, S transposed
//   dv       k   q   do  dv  0  scale  1      scale   last token first
// (e = 0: the carried gradient already holds the decay of the boundary step.)
// Only powers with exponents >= 0 are ever formed, so any decay is safe.
//
// Long sequences are cut into `nseg` segments of seg_len tokens: a first
// launch forms each segment's own final state, a small second one turns them
// into the states before each segment, and the third runs all segments at
// once.  The second and third are launched with programmatic stream
// serialization: they set up and start their loads while their predecessor
// drains, and call decay_wait before they read what it wrote.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mhla.h"

namespace mhla {

struct DecayPass {
  const void *x, *y, *z;
  void* o;
  mhla_strides sx, sy, sz, so;
  const float* g;  // [H] log decay
  const int32_t* lengths;
  const float* s_in;  // [units][DX][DZ], or its transpose (s_ldx, s_ldz); may be null
  float* s_out;       // same layout; may be null, may be s_in
  float* seg;         // [units][nseg][DX * DZ] (nseg > 1): slot i the state before segment i
  int s_ldx, s_ldz;   // element strides of a state's x and z axes, in s_in, s_out and seg
  int B, H, N, DX, DZ;
  int nseg, seg_len;
  int slice;     // columns of z that a CTA of the 128-entry tcgen05 pass takes
  int launches;  // 1: the states before the segments, 2: the pass itself, 3: both
  int reverse;  // 1: token i of the pass is the sequence's token length - 1 - i
  int e;
  float score, read, update;
  int vec;            // rows are 16-byte aligned
  unsigned int* err;  // device error word
};

#ifdef __CUDACC__
__device__ __forceinline__ void decay_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void decay_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// lambda^n = exp(n g) as high + low parts, so that a state that is multiplied
// by it thousands of times does not drift by the rounding of one float32
// factor.  Slow decays go through exp(x) = 1 + expm1(x), whose float32 value
// is off by 2^-24 |x| only; fast ones have few factors that matter.
__device__ __forceinline__ float2 decay_power(float g, int n) {
  if (n == 0) return make_float2(1.f, 0.f);  // also for g = -inf
  const float x = (float)n * g;
  float rest = fmaf((float)n, g, -x);  // what the product's rounding left
  if (!(fabsf(rest) < 1.f)) rest = 0.f;
  if (fabsf(x) < 0.5f) {
    float m = expm1f(x);
    m = fmaf(1.f + m, rest, m);
    const float hi = 1.f + m;
    return make_float2(hi, m - (hi - 1.f));
  }
  const float y = expf(x);
  return make_float2(fmaf(y, rest, y), 0.f);
}

__device__ __forceinline__ int decay_length(const DecayPass& p, int b) {
  if (!p.lengths) return p.N;
  const int n = p.lengths[b];
  return n < 0 ? 0 : n > p.N ? p.N : n;
}

// Token of the sequence that the pass takes at place i.
__device__ __forceinline__ int decay_token(const DecayPass& p, int i, int length) {
  return p.reverse && i < length ? length - 1 - i : i;
}
#endif

// Resident CTAs of an SM of the CUDA-core kernel's pass: one where its tiles
// take 131 KB of shared memory; three with short rows and 64-column slices (64
// registers a thread); two elsewhere (up to 128 registers, or more than a third
// of the shared memory).
constexpr int decay_simt_resident(int dx, int slice) {
  return dx == 128 && slice == 64 ? 1 : dx <= 32 && slice == 64 ? 3 : 2;
}

// Launches return a cudaError_t.
cudaError_t launch_decay_scan(const DecayPass& p, cudaStream_t s);
cudaError_t launch_decay_simt(const DecayPass& p, int dtype, cudaStream_t s);
cudaError_t launch_decay_mma(const DecayPass& p, cudaStream_t s);  // bf16
cudaError_t launch_decay_tc(const DecayPass& p, cudaStream_t s);   // bf16, DX = 64 or 128, DZ a multiple of 64, vec
cudaError_t launch_decay_step(const DecayPass& p, int dtype, cudaStream_t s);

}  // namespace mhla
