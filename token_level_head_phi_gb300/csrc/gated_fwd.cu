// Gated recurrence: prompts, and one token of every sequence.
#include "gated.cuh"

namespace mhla {
namespace {

// c of two channels: sqrt(1 - a^2) = sqrt(gap (1 + a)), or k1 gap + k0.
template <bool NORM>
__device__ __forceinline__ uint64_t factor(uint64_t gap, uint64_t a, uint64_t k1, uint64_t k0) {
  if constexpr (!NORM) return fma2(gap, k1, k0);
  const float2 v = unpair(mul2(gap, add2(a, splat(1.f))));
  return pair(root(v.x), root(v.y));
}

template <typename T, int KIND, bool IN, bool NORM>
__global__ void __launch_bounds__(32 * kGatedWarps, gated_resident(sizeof(T) == 4, false))
    gated_fwd_kernel(const __grid_constant__ GatedArgs p) {
  __shared__ Scan<false> scan;
  const int rank = cluster_rank(), ranks = cluster_size(), unit = blockIdx.x / ranks;
  const int b = unit / p.slabs, w = threadIdx.x >> 5;
  const Lane ln(unit - b * p.slabs, p.D);
  const int len = gated_length(p, b), round = kGatedTile * ranks;  // tokens that the cluster takes at once
  const float2 lg = unpair(ln.get(KIND == MHLA_GATED_DECAY ? p.g : nullptr));
  const uint64_t g = pair(least(lg.x, 0.f), least(lg.y, 0.f));
  const uint64_t k1 = splat(p.scale == MHLA_GATED_SCALE_MEAN ? 1.f : 0.f), k0 = splat(p.scale == MHLA_GATED_SCALE_MEAN ? 0.f : 1.f);
  uint64_t carry = ln.get(p.state_in ? p.state_in + (int64_t)b * p.D : nullptr);
  const T* x = static_cast<const T*>(p.x) + b * p.sx.batch + ln.ch;
  const T* r = static_cast<const T*>(p.r) + b * p.sr.batch + ln.ch;
  const T* i = static_cast<const T*>(p.i) + b * p.si.batch + ln.ch;
  T* out = static_cast<T*>(p.out) + b * p.so.batch + ln.ch;
  // whole slabs of aligned pairs: no checks inside rounds that end before the length
  const bool vec = p.vec && ln.n == 2, whole = p.vec && (unit - b * p.slabs + 1) * kGatedSlab <= p.D;

  Two<T> rx[kGatedTok], rr[kGatedTok], ri[kGatedTok];
  auto fetch = [&](int t0, bool fast) {
    const T *px = x + t0 * p.sx.token, *pr = r + t0 * p.sr.token, *pi = i + t0 * p.si.token;
    if (fast) {
#pragma unroll
      for (int j = 0; j < kGatedTok; ++j, px += p.sx.token, pr += p.sr.token, pi += p.si.token) {
        rx[j].load(px, true);
        rr[j].load(pr, true);
        if constexpr (IN) ri[j].load(pi, true);
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < kGatedTok; ++j, px += p.sx.token, pr += p.sr.token, pi += p.si.token) {
      rx[j].zero();
      rr[j].zero();
      ri[j].zero();
      if (ln.n == 0 || t0 + j >= len) continue;
      rx[j].load(px, vec, ln.n);
      rr[j].load(pr, vec, ln.n);
      if constexpr (IN) ri[j].load(pi, vec, ln.n);
    }
  };
  int t0 = rank * kGatedTile + w * kGatedTok, turn = 0;
  if (ranks > 1) cluster_arrive();  // nobody sends before all have begun
  if (len > 0) fetch(t0, whole && round <= len);
  if (ranks > 1) cluster_wait();
  for (int base = 0; base < len; base += round, t0 += round, turn ^= 1) {  // the same turns in all of the cluster
    const bool fast = whole && base + round <= len;
    uint64_t a[kGatedTok], add[kGatedTok];
    Map map = same();
#pragma unroll
    for (int j = 0; j < kGatedTok; ++j) {
      const Gates t = gates_of<KIND, IN>(wide(rr[j]), IN ? wide(ri[j]) : 0, g);
      const uint64_t u = IN ? mul2(wide(rx[j]), t.q) : wide(rx[j]);
      a[j] = decay_of(t.gap);
      add[j] = mul2(factor<NORM>(t.gap, a[j], k1, k0), u);
    }
    if (!fast)
#pragma unroll
      for (int j = 0; j < kGatedTok; ++j)
        if (t0 + j >= len) {  // keeps the state
          a[j] = splat(1.f);
          add[j] = splat(0.f);
        }
#pragma unroll
    for (int j = 0; j < kGatedTok; ++j) map = then(map, Map{a[j], add[j]});
    if (base + round < len) fetch(t0 + round, whole && base + 2 * round <= len);
    uint64_t h = scan.run(turn, rank, ranks, map, &carry);
    if (p.marks && w == 0 && t0 < p.N) ln.put(p.marks + ((int64_t)b * p.n_marks + t0 / MHLA_GATED_MARK) * p.D, h);
    T* po = out + t0 * p.so.token;
    if (p.out && fast) {
#pragma unroll
      for (int j = 0; j < kGatedTok; ++j, po += p.so.token) {
        h = fma2(a[j], h, add[j]);
        narrow(h, T()).store(po, true);
      }
    } else if (p.out && ln.n) {
#pragma unroll
      for (int j = 0; j < kGatedTok; ++j, po += p.so.token) {
        h = fma2(a[j], h, add[j]);
        if (t0 + j < p.N) narrow(t0 + j < len ? h : splat(0.f), T()).store(po, vec, ln.n);
      }
    }
  }
  if (p.state_out && rank == 0 && w == 0) ln.put(p.state_out + (int64_t)b * p.D, carry);
  for (; t0 < p.N; t0 += round) {  // padding
    if (p.marks && w == 0) ln.put(p.marks + ((int64_t)b * p.n_marks + t0 / MHLA_GATED_MARK) * p.D, carry);
    if (!p.out || !ln.n) continue;
    for (int t = t0; t < t0 + kGatedTok && t < p.N; ++t) narrow(splat(0.f), T()).store(out + t * p.so.token, vec, ln.n);
  }
}

// One token of every sequence: a thread takes two channels.
template <typename T, int KIND, bool IN, bool NORM>
__global__ void __launch_bounds__(128) gated_step_kernel(const __grid_constant__ GatedArgs p) {
  const int pairs = (p.D + 1) / 2;
  const int64_t at = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (at >= (int64_t)p.B * pairs) return;
  const int64_t b = at / pairs;
  Lane ln(0, 0);
  ln.ch = 2 * (int)(at - b * pairs);
  ln.n = min(p.D - ln.ch, 2);
  const bool vec = p.vec && ln.n == 2;
  Two<T> x, r, i;
  x.load(static_cast<const T*>(p.x) + b * p.sx.batch + ln.ch, vec, ln.n);
  r.load(static_cast<const T*>(p.r) + b * p.sr.batch + ln.ch, vec, ln.n);
  if constexpr (IN) i.load(static_cast<const T*>(p.i) + b * p.si.batch + ln.ch, vec, ln.n);
  const float2 lg = unpair(ln.get(KIND == MHLA_GATED_DECAY ? p.g : nullptr));
  uint64_t h = ln.get(p.state_in ? p.state_in + b * p.D : nullptr);
  const Gates t = gates_of<KIND, IN>(wide(r), IN ? wide(i) : 0, pair(least(lg.x, 0.f), least(lg.y, 0.f)));
  const uint64_t a = decay_of(t.gap), u = IN ? mul2(wide(x), t.q) : wide(x);
  const float k = p.scale == MHLA_GATED_SCALE_MEAN ? 1.f : 0.f;
  h = fma2(a, h, mul2(factor<NORM>(t.gap, a, splat(k), splat(1.f - k)), u));
  narrow(h, T()).store(static_cast<T*>(p.out) + b * p.so.batch + ln.ch, vec, ln.n);
  if (p.state_out) ln.put(p.state_out + b * p.D, h);
}

struct Forward {
  const GatedArgs& a;
  cudaStream_t s;
  template <typename T, int KIND, bool IN>
  mhla_status go() {
    if (a.scale == MHLA_GATED_SCALE_NORM)
      return launch_gated_clusters(gated_fwd_kernel<T, KIND, IN, true>, a, gated_resident(sizeof(T) == 4, false), 0, s);
    return launch_gated_clusters(gated_fwd_kernel<T, KIND, IN, false>, a, gated_resident(sizeof(T) == 4, false), 0, s);
  }
};

struct Step {
  const GatedArgs& a;
  cudaStream_t s;
  template <typename T, int KIND, bool IN>
  mhla_status go() {
    const int64_t blocks = ((int64_t)a.B * ((a.D + 1) / 2) + 127) / 128;
    if (blocks > 0x7fffffff) return MHLA_ERR_UNSUPPORTED;
    if (a.scale == MHLA_GATED_SCALE_NORM)
      gated_step_kernel<T, KIND, IN, true><<<(unsigned)blocks, 128, 0, s>>>(a);
    else
      gated_step_kernel<T, KIND, IN, false><<<(unsigned)blocks, 128, 0, s>>>(a);
    return launch_status();
  }
};

}  // namespace

mhla_status launch_gated_fwd(const GatedArgs& a, int dtype, int kind, cudaStream_t s) {
  return with_gates(a, dtype, kind, Forward{a, s});
}

mhla_status launch_gated_step(const GatedArgs& a, int dtype, int kind, cudaStream_t s) {
  return with_gates(a, dtype, kind, Step{a, s});
}

}  // namespace mhla
