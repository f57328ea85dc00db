// The states before each segment of a decayed linear-attention pass, from the
// segments' own final states: P_0 = s_in, P_i = lambda^seg_len P_{i-1} + R_{i-1}.
// Slot i > 0 holds R_{i-1} before and P_i after; slot 0 takes P_0, because the
// pass may overwrite s_in.  A thread takes four entries of one unit and runs
// over its slots with eight loads in flight.  Bound by the latency of its
// launch and two dependent trips to memory: 6 to 10 us alone, 25 MB of slots or 4.
#include "decay.h"
#include "ops.h"
#include "tc_host.h"

namespace mhla {
namespace {

constexpr int kThreads = 128;

__global__ void __launch_bounds__(kThreads) decay_scan_kernel(const DecayPass p) {
  decay_dependents();
  const int unit = blockIdx.x;
  const int one = p.DX * p.DZ / 4;
  const int i = blockIdx.y * kThreads + threadIdx.x;
  if (i >= one) return;
  const float2 w = decay_power(p.g[unit % p.H], p.seg_len);
  float4* seg = reinterpret_cast<float4*>(p.seg) + (int64_t)unit * p.nseg * one + i;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.s_in) s = (reinterpret_cast<const float4*>(p.s_in) + (int64_t)unit * one)[i];
  decay_wait();
  seg[0] = s;
  for (int n = 1; n < p.nseg; n += 8) {
    float4 r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (n + k < p.nseg) r[k] = seg[(int64_t)(n + k) * one];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (n + k < p.nseg) {
        s.x = fmaf(s.x, w.x, fmaf(s.x, w.y, r[k].x));
        s.y = fmaf(s.y, w.x, fmaf(s.y, w.y, r[k].y));
        s.z = fmaf(s.z, w.x, fmaf(s.z, w.y, r[k].z));
        s.w = fmaf(s.w, w.x, fmaf(s.w, w.y, r[k].w));
        seg[(int64_t)(n + k) * one] = s;
      }
  }
}

}  // namespace

cudaError_t launch_decay_scan(const DecayPass& p, cudaStream_t s) {
  const unsigned blocks = (unsigned)((p.DX * p.DZ / 4 + kThreads - 1) / kThreads);
  return (cudaError_t)launch_pdl(decay_scan_kernel, dim3((unsigned)(p.B * p.H), blocks), dim3(kThreads), 0, s, p);
}

}  // namespace mhla
