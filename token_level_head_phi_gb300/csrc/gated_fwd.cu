// Gated recurrence: prompts, and one token of every sequence.
//
// Bound: memory where there are many sequences (bf16 with an input gate 8 bytes
// an element): 64 x 512 tokens of 4096 channels take 173 us, 6.2 TB/s.  With few
// it is the latency of the clusters' rounds: 2 x 32k tokens of 1024 channels take
// 134 us in 32 rounds (79 us at the rate of a copy); an SM issues 46 % of the time,
// 72 instructions to a pair of channels, half of them for the gates.
#include "gated.cuh"

namespace mhla {
namespace {

// A warp's inputs of two rounds; the results take x's place.
template <typename T, bool IN>
struct Stage {
  static constexpr int kTok = kGatedTok<sizeof(T) == 4, false>;
  Rows<T, kTok> x[2], r[2], i[IN ? 2 : 0];
};

// The warps of a CTA alone hand their states from one to the next, without a
// barrier for all of them.  In a cluster all wait for the others' tiles anyway:
// each shows the map of its tokens to the warps behind it (2 x 8k tokens of 1024
// channels 40 us, handed on from warp to warp 41; backward 80 and 78).
template <typename T, int KIND, bool IN, bool NORM, int VEC>
__global__ void __launch_bounds__(32 * kGatedWarps, gated_resident(sizeof(T) == 4))
    gated_fwd_kernel(const __grid_constant__ GatedArgs p) {
  constexpr int kTok = kGatedTok<sizeof(T) == 4, false>, kTile = kGatedWarps * kTok;
  extern __shared__ __align__(16) unsigned char dynamic[];
  __shared__ Map mail[2][kGatedWarps][32];  // alone the first half, for the states
  __shared__ Map tiles[2][kGatedCluster][32];
  const int rank = cluster_rank(), ranks = cluster_size(), unit = blockIdx.x / ranks;
  const int w = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), l = threadIdx.x & 31;
  const int b = unit / p.slabs, slab = unit - b * p.slabs, first = slab * kGatedSlab, cols = p.D - first;
  Stage<T, IN>& my = reinterpret_cast<Stage<T, IN>*>(dynamic)[w];
  const Lane ln(slab, p.D);
  const int vec = VEC == kGatedNarrow ? p.vec != 0 : VEC;
  const int len = gated_length(p, b), round = kTile * ranks;  // tokens that the cluster takes at once
  const float2 lg = ln.get(KIND == MHLA_GATED_DECAY ? p.g : nullptr);
  const float2 g2 = mulc(make_float2(least(lg.x, 0.f), least(lg.y, 0.f)), kLog2e);
  const bool mean = p.scale == MHLA_GATED_SCALE_MEAN;
  const float2 k1 = splat(mean ? -1.f : 0.f), k0 = splat(mean ? 0.f : 1.f);  // c = k0 + k1 m
  float2 carry = ln.get(p.state_in ? p.state_in + (int64_t)b * p.D : nullptr);
  using In = Walk<T, const T>;
  const In x(static_cast<const T*>(p.x) + b * p.sx.batch + first, p.sx.token, vec);
  const In r(static_cast<const T*>(p.r) + b * p.sr.batch + first, p.sr.token, vec);
  const In i(static_cast<const T*>(p.i) + b * p.si.batch + first, p.si.token, vec);
  const Walk<T, T> out(static_cast<T*>(p.out) + b * p.so.batch + first, p.so.token, vec);
  const bool whole = VEC == 2 && cols >= kGatedSlab;

  auto fetch = [&](int slot, int t0) {
    if (t0 < len) {
      const bool fast = whole && t0 + kTok <= len;
      x.fetch(my.x[slot], t0, fast, len - t0, cols, vec);
      r.fetch(my.r[slot], t0, fast, len - t0, cols, vec);
      if constexpr (IN) i.fetch(my.i[slot], t0, fast, len - t0, cols, vec);
    }
    copies_commit();
  };
  auto write = [&](int slot, int t0) {
    if (t0 < p.N) out.write(my.x[slot], t0, whole && t0 + kTok <= p.N, p.N - t0, cols, vec);
  };
  auto mark = [&](int t0, float2 h) {
    if (p.marks && t0 % MHLA_GATED_MARK == 0 && t0 < p.N)
      ln.put(p.marks + ((int64_t)b * p.n_marks + t0 / MHLA_GATED_MARK) * p.D, h);
  };
  const int mine = rank * kTile + w * kTok;
  int t0 = mine, turn = 0;
  if (ranks > 1) cluster_arrive();  // nobody sends before all have begun
  fetch(0, t0);
  __syncwarp();
  if (ranks > 1) cluster_wait();
  for (int base = 0; base < len; base += round, t0 += round, turn ^= 1) {  // the same turns in all of the cluster
    fetch(turn ^ 1, t0 + round);
    copies_wait<1>();
    __syncwarp();
    float2 a[kTok], add[kTok];
    Map map = same();
    if (t0 < len) {
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        const float2 rv = least_gate(my.r[turn].v[j][l]), iv = IN ? least_gate(my.i[turn].v[j][l]) : splat(0.f);
        const Gates t = gates_of<KIND, IN>(rv, iv, g2);
        const float2 xv = wide(my.x[turn].v[j][l]), u = IN ? mul2(xv, t.q) : xv;
        a[j] = t.a;
        add[j] = mul2(factor<NORM>(t.m, k1, k0), u);
      }
      if (t0 + kTok > len)
#pragma unroll
        for (int j = 0; j < kTok; ++j)
          if (t0 + j >= len) a[j] = splat(1.f), add[j] = splat(0.f);  // keeps the state
      map = Map{a[0], add[0]};
#pragma unroll
      for (int j = 1; j < kTok; ++j) map = then(map, Map{a[j], add[j]});
    }
    float2 h;
    if (ranks == 1) {
      h = carry;
      if (w > 0 || base > 0) {
        take_over(1 + w);
        h = mail[0][w][l].H;
      }
      carry = through(map, h);
      if (w < kGatedWarps - 1 || base + round < len) {
        const int to = (w + 1) % kGatedWarps;
        mail[0][to][l].H = carry;
        hand_over(1 + to);
      }
    } else {
      store_map(&mail[turn][w][l], map);
      __syncthreads();
      Map before = same();
      auto compose = [&] {
        for (int v = 0; v < w; ++v) before = then(before, load_map(&mail[turn][v][l]));
      };
      if (w == kGatedWarps - 1) {
        compose();
        const Map all = then(before, map);
        for (int v = 0; v < ranks; ++v) send(&tiles[turn][rank][l], v, all);
      }
      cluster_arrive();
      if (w < kGatedWarps - 1) compose();
      cluster_wait();
      h = carry;
      for (int v = 0; v < rank; ++v) h = through(load_map(&tiles[turn][v][l]), h);
      carry = h;
      for (int v = rank; v < ranks; ++v) carry = through(load_map(&tiles[turn][v][l]), carry);
      h = through(before, h);
    }
    mark(t0, h);
    if (p.out) {
      if (t0 < len)
#pragma unroll
        for (int j = 0; j < kTok; ++j) {
          h = fma2(a[j], h, add[j]);
          my.x[turn].v[j][l] = narrow(h, T());
        }
      if (t0 + kTok > len)
#pragma unroll
        for (int j = 0; j < kTok; ++j)
          if (t0 + j >= len) my.x[turn].v[j][l].zero();
      write(turn, t0);
    }
    __syncwarp();  // other lanes' copies arrive where this one has read
  }
  // alone, the last warp has the final state, and marks past the length need it
  if (ranks == 1 && len > 0 && p.marks) {
    __syncthreads();
    if (w == kGatedWarps - 1) mail[0][0][l].H = carry;
    __syncthreads();
    carry = mail[0][0][l].H;
  }
  if (p.state_out && rank == 0 && w == kGatedWarps - 1) ln.put(p.state_out + (int64_t)b * p.D, carry);
  if (t0 >= p.N) return;
#pragma unroll
  for (int j = 0; j < kTok; ++j) my.x[0].v[j][l].zero();
  for (; t0 < p.N; t0 += round) {  // padding
    mark(t0, carry);
    if (p.out) write(0, t0);
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
  const bool vec = p.vec > 0 && ln.n == 2;
  Two<T> x, r, i;
  x.load(static_cast<const T*>(p.x) + b * p.sx.batch + ln.ch, vec, ln.n);
  r.load(static_cast<const T*>(p.r) + b * p.sr.batch + ln.ch, vec, ln.n);
  if constexpr (IN) i.load(static_cast<const T*>(p.i) + b * p.si.batch + ln.ch, vec, ln.n);
  const float2 lg = ln.get(KIND == MHLA_GATED_DECAY ? p.g : nullptr);
  float2 h = ln.get(p.state_in ? p.state_in + b * p.D : nullptr);
  const float2 g2 = mulc(make_float2(least(lg.x, 0.f), least(lg.y, 0.f)), kLog2e);
  const Gates t = gates_of<KIND, IN>(least_gate(r), IN ? least_gate(i) : splat(0.f), g2);
  const float2 u = IN ? mul2(wide(x), t.q) : wide(x);
  const float k = p.scale == MHLA_GATED_SCALE_MEAN ? 1.f : 0.f;
  h = fma2(t.a, h, mul2(factor<NORM>(t.m, splat(-k), splat(1.f - k)), u));
  narrow(h, T()).store(static_cast<T*>(p.out) + b * p.so.batch + ln.ch, vec, ln.n);
  if (p.state_out) ln.put(p.state_out + b * p.D, h);
}

struct Forward {
  const GatedArgs& a;
  cudaStream_t s;
  template <typename T, int KIND, bool IN, bool NORM>
  mhla_status run() {
    constexpr bool kApart = sizeof(T) == 4;  // see kGatedNarrow
    auto kernel = a.vec == 2   ? gated_fwd_kernel<T, KIND, IN, NORM, 2>
                  : a.vec == 1 ? gated_fwd_kernel<T, KIND, IN, NORM, kApart ? 1 : kGatedNarrow>
                               : gated_fwd_kernel<T, KIND, IN, NORM, kApart ? 0 : kGatedNarrow>;
    return launch_gated_clusters(kernel, a, sizeof(T) == 4, false, kGatedWarps * sizeof(Stage<T, IN>), s);
  }
  template <typename T, int KIND, bool IN>
  mhla_status go() {
    return a.scale == MHLA_GATED_SCALE_NORM ? run<T, KIND, IN, true>() : run<T, KIND, IN, false>();
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
