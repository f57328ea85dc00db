// Gated recurrence: the gradients.
//
// The tiles are taken from the last one; the states inside a tile come from
// the state before it, which the forward pass keeps in float32 for every 64th
// token (3 % of the inputs' bytes).  A thread copies its own tokens' inputs of
// the next round into shared memory while it works on this one's, and is the
// only one to read them.
#include "gated.cuh"

namespace mhla {
namespace {

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Inputs of one round: a thread's tokens of x, dout, r and i.
template <typename T, bool IN>
struct Stage {
  Two<T> v[IN ? 4 : 3][kGatedTok<sizeof(T) == 4, true>][32 * kGatedWarps];
};

template <typename T, int KIND, bool IN, bool NORM>
__global__ void __launch_bounds__(32 * kGatedWarps, gated_resident(sizeof(T) == 4, true))
    gated_bwd_kernel(const __grid_constant__ GatedArgs p) {
  constexpr int kTok = kGatedTok<sizeof(T) == 4, true>, kTile = kGatedWarps * kTok;
  extern __shared__ __align__(16) unsigned char dynamic[];
  Stage<T, IN>* stage = reinterpret_cast<Stage<T, IN>*>(dynamic);  // [2]
  __shared__ Scan<true> scan;
  __shared__ Map maps[2][kGatedWarps][32];
  const int rank = cluster_rank(), ranks = cluster_size(), unit = blockIdx.x / ranks;
  const int b = unit / p.slabs, w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const Lane ln(unit - b * p.slabs, p.D);
  const int len = gated_length(p, b), round = kTile * ranks;
  const float2 lg = (ln.get(KIND == MHLA_GATED_DECAY ? p.g : nullptr));
  const float2 g = make_float2(least(lg.x, 0.f), least(lg.y, 0.f));
  const float2 g2 = mulc(g, kLog2e);
  const float2 k1 = splat(p.scale == MHLA_GATED_SCALE_MEAN ? -1.f : 0.f), k0 = splat(p.scale == MHLA_GATED_SCALE_MEAN ? 0.f : 1.f);
  // the gradient that reaches a token's state from behind it
  float2 carry = ln.get(p.dstate_out ? p.dstate_out + (int64_t)b * p.D : nullptr);
  const T* x = static_cast<const T*>(p.x) + b * p.sx.batch + ln.ch;
  const T* r = static_cast<const T*>(p.r) + b * p.sr.batch + ln.ch;
  const T* i = static_cast<const T*>(p.i) + b * p.si.batch + ln.ch;
  const T* dout = static_cast<const T*>(p.dout) + b * p.sdo.batch + ln.ch;
  T* dx = static_cast<T*>(p.dx) + b * p.sdx.batch + ln.ch;
  T* dr = static_cast<T*>(p.dr) + b * p.sdr.batch + ln.ch;
  T* di = static_cast<T*>(p.di) + b * p.sdi.batch + ln.ch;
  const bool vec = p.vec && ln.n == 2, whole = p.vec && (unit - b * p.slabs + 1) * kGatedSlab <= p.D;
  const float2 zero = splat(0.f);
  float2 dg = zero;
  const int rounds = (len + round - 1) / round, mine = rank * kTile + w * kTok;

  auto fetch = [&](int slot, int base) {
    Stage<T, IN>& to = stage[slot];
    const int t0 = base + mine;
    const T* src[4] = {x + t0 * p.sx.token, dout + t0 * p.sdo.token, r + t0 * p.sr.token, i + t0 * p.si.token};
    const int64_t step[4] = {p.sx.token, p.sdo.token, p.sr.token, p.si.token};
    if (whole && base + round <= len) {
#pragma unroll
      for (int j = 0; j < kTok; ++j)
#pragma unroll
        for (int k = 0; k < (IN ? 4 : 3); ++k, src[k - 1] += step[k - 1])
          copy_async<2 * sizeof(T)>((uint32_t)__cvta_generic_to_shared(&to.v[k][j][threadIdx.x]), src[k]);
    } else {
#pragma unroll
      for (int j = 0; j < kTok; ++j)
#pragma unroll
        for (int k = 0; k < (IN ? 4 : 3); ++k, src[k - 1] += step[k - 1]) {
          Two<T> v;
          v.zero();
          if (ln.n && t0 + j < len) v.load(src[k], vec, ln.n);
          to.v[k][j][threadIdx.x] = v;
        }
    }
    copies_commit();
  };

  if (ranks > 1) cluster_arrive();  // nobody sends before all have begun
  if (rounds > 0) fetch(0, (rounds - 1) * round);
  for (int t0 = rounds * round + mine; t0 < p.N && ln.n; t0 += round)  // padding
    for (int t = t0; t < t0 + kTok && t < p.N; ++t) {
      narrow(zero, T()).store(dx + t * p.sdx.token, vec, ln.n);
      narrow(zero, T()).store(dr + t * p.sdr.token, vec, ln.n);
      if constexpr (IN) narrow(zero, T()).store(di + t * p.sdi.token, vec, ln.n);
    }
  if (ranks > 1) cluster_wait();
  int turn = 0;
  for (int base = (rounds - 1) * round; base >= 0; base -= round, turn ^= 1) {
    const int tile = base + rank * kTile, t0 = base + mine;
    const bool fast = whole && base + round <= len;
    if (base > 0) {
      fetch(turn ^ 1, base - round);
      copies_wait<1>();
    } else {
      copies_wait<0>();
    }
    const Stage<T, IN>& in = stage[turn];
    float2 h = tile < len ? ln.get(p.marks + ((int64_t)b * p.n_marks + tile / MHLA_GATED_MARK) * p.D) : zero;

    // From the last token: the map of the states, and what the tokens send to
    // the one before them.
    Gates gt[kTok];
    float2 inv[kTok];  // -1 / c for NORM
    float2 rest = zero;
    Map map = same();
    auto factor = [&](int j) {
      if constexpr (!NORM) return fma2(gt[j].m, k1, k0);
      return mul2(minus_v(gt[j].m), inv[j]);
    };
#pragma unroll
    for (int j = kTok - 1; j >= 0; --j) {
      gt[j] = gates_of<KIND, IN>(least_gate(in.v[2][j][threadIdx.x]), IN ? least_gate(in.v[IN ? 3 : 0][j][threadIdx.x]) : splat(0.f), g, g2);
      if (!fast && t0 + j >= len) gt[j].m = gt[j].s = gt[j].less = zero;  // keeps the state
      const float2 a = addc(gt[j].m, 1.f);
      if constexpr (NORM) {
        // v^(-1/2) as v (max(v, tiny)^(-1/2))^3, which is 0 for v = 0
        const float2 v = minus_v(gt[j].m);
        const float2 f = (v);
        const float2 q = make_float2(rsq(fmaxf(-f.x, 1e-36f)), rsq(fmaxf(-f.y, 1e-36f)));
        inv[j] = mul2(mul2(v, q), mul2(q, q));
      }
      const float2 xv = wide(in.v[0][j][threadIdx.x]), u = IN ? mul2(xv, gt[j].q) : xv;
      map.H = fma2(map.A, mul2(factor(j), u), map.H);
      map.A = mul2(map.A, a);
      rest = mul2(a, add2(rest, wide(in.v[1][j][threadIdx.x])));
    }
    store_map(&maps[turn][w][l], map);
    float2 e = scan.run(turn, rank, ranks, Map{map.A, rest}, &carry);
#pragma unroll
    for (int v = 0; v < kGatedWarps - 1; ++v)
      if (v < w) h = through(load_map(&maps[turn][v][l]), h);
    float2 before[kTok];
    T *px = dx + (t0 + kTok - 1) * p.sdx.token, *pr = dr + (t0 + kTok - 1) * p.sdr.token;
    T* pi = di + (t0 + kTok - 1) * p.sdi.token;
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      before[j] = h;
      const float2 xv = wide(in.v[0][j][threadIdx.x]), u = IN ? mul2(xv, gt[j].q) : xv, a = addc(gt[j].m, 1.f);
      h = fma2(a, h, mul2(factor(j), u));
    }
#pragma unroll
    for (int j = kTok - 1; j >= 0; --j) {
      const float2 xv = wide(in.v[0][j][threadIdx.x]), u = IN ? mul2(xv, gt[j].q) : xv;
      const float2 a = addc(gt[j].m, 1.f), c = factor(j);
      const float2 G = add2(e, wide(in.v[1][j][threadIdx.x]));
      // a h + u dc / dlog a = a (h - u a / c), or a (h + u k1)
      const float2 sum = NORM ? fma2(mul2(u, inv[j]), a, before[j]) : fma2(u, k1, before[j]);
      // sigma itself where a is one: 1 + m has lost a small one's last bits
      const float2 dlog = mul2(G, mul2(KIND == MHLA_GATED_DECAY ? a : gt[j].s, sum));
      float2 o_r = mul2(dlog, gt[j].less);
      if constexpr (KIND == MHLA_GATED_DECAY) {
        const float2 ds = mul2(dlog, gt[j].s);
        dg = add2(dg, ds);
        o_r = mul2(mul2(ds, g), gt[j].less);
      }
      const float2 du = mul2(G, c), o_x = IN ? mul2(du, gt[j].q) : du;
      const float2 o_xx = IN ? mul2(o_x, xv) : zero, o_i = IN ? fma2(mulc(o_xx, -1.f), gt[j].q, o_xx) : zero;
      e = mul2(a, G);
      const int t = t0 + j;
      if (fast) {
        narrow(o_x, T()).store(px, true);
        narrow(o_r, T()).store(pr, true);
        if constexpr (IN) narrow(o_i, T()).store(pi, true);
      } else if (ln.n && t < p.N) {
        const bool live = t < len;
        narrow(live ? o_x : zero, T()).store(px, vec, ln.n);
        narrow(live ? o_r : zero, T()).store(pr, vec, ln.n);
        if constexpr (IN) narrow(live ? o_i : zero, T()).store(pi, vec, ln.n);
      }
      px -= p.sdx.token;
      pr -= p.sdr.token;
      pi -= p.sdi.token;
    }
  }
  if (p.dstate_in && rank == 0 && w == 0) ln.put(p.dstate_in + (int64_t)b * p.D, carry);
  if (KIND == MHLA_GATED_DECAY && p.partial) {
    __syncthreads();  // the last reads of maps
    maps[0][w][l].A = dg;
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int v = 1; v < kGatedWarps; ++v) dg = add2(dg, maps[0][v][l].A);
      ln.put(p.partial + ((int64_t)b * ranks + rank) * p.D, dg);
    }
  }
}

struct Backward {
  const GatedArgs& a;
  cudaStream_t s;
  template <typename T, int KIND, bool IN, bool NORM>
  mhla_status run() {
    return launch_gated_clusters(gated_bwd_kernel<T, KIND, IN, NORM>, a, sizeof(T) == 4, true, 2 * sizeof(Stage<T, IN>), s);
  }
  template <typename T, int KIND, bool IN>
  mhla_status go() {
    return a.scale == MHLA_GATED_SCALE_NORM ? run<T, KIND, IN, true>() : run<T, KIND, IN, false>();
  }
};

}  // namespace

mhla_status launch_gated_bwd(const GatedArgs& a, int dtype, int kind, cudaStream_t s) {
  return with_gates(a, dtype, kind, Backward{a, s});
}

}  // namespace mhla
