// Gated recurrence: the gradients.
//
// The tiles are taken from the last one.  A warp's tokens start from a state
// that the forward pass has kept in float32 (before every 16th token, 1 / 32 of
// the inputs' bytes), or from its neighbour's; the gradient of the state behind
// them comes from the warp behind.
//
// Bound: instructions and the rounds' latency, not memory (bf16 with an input
// gate 14 bytes an element): 64 x 512 tokens of 4096 channels take 384 us, 4.9
// TB/s; 2 x 8k tokens of 1024 channels 78 us in 16 rounds of clusters of 8 (35 us at
// the rate of a copy), an SM issuing 49 % of the time, 155 instructions to a pair
// of channels.
#include "gated.cuh"

namespace mhla {
namespace {

// A warp's inputs of two rounds; dx, dgate and dinput_gate take the places of
// x, the gate and the input gate.
template <typename T, bool IN>
struct Stage {
  static constexpr int kTok = kGatedTok<sizeof(T) == 4, true>;
  Rows<T, kTok> x, d, r, i[IN ? 1 : 0];
};
static_assert(MHLA_GATED_MARK == 2 * 8, "every second warp starts at a mark");

// -1 / c, 0 for c = 0, which else is 1e-19 at least (the root of float32's smallest
// normal number): -c (1 / max(c, tiny))^2.
__device__ __forceinline__ float2 minus_inverse(float2 c) {
  const float2 i = make_float2(rcp(fmaxf(c.x, 1e-19f)), rcp(fmaxf(c.y, 1e-19f)));
  return mul2(mul2(i, make_float2(-i.x, -i.y)), c);
}

template <typename T, int KIND, bool IN, bool NORM, int VEC>
__global__ void __launch_bounds__(32 * kGatedWarps, gated_resident(sizeof(T) == 4))
    gated_bwd_kernel(const __grid_constant__ GatedArgs p) {
  constexpr int kTok = kGatedTok<sizeof(T) == 4, true>, kTile = kGatedWarps * kTok;
  extern __shared__ __align__(16) unsigned char dynamic[];
  __shared__ Map mail[kGatedWarps][32];          // from the warp behind
  __shared__ Map tiles[2][kGatedCluster][32];
  __shared__ float2 states[kGatedWarps / 2][32];  // from the warp before
  const int rank = cluster_rank(), ranks = cluster_size(), unit = blockIdx.x / ranks;
  const int w = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), l = threadIdx.x & 31;
  const int b = unit / p.slabs, slab = unit - b * p.slabs, first = slab * kGatedSlab, cols = p.D - first;
  Stage<T, IN>* stage = reinterpret_cast<Stage<T, IN>*>(dynamic) + 2 * w;
  const Lane ln(slab, p.D);
  const int vec = VEC == kGatedNarrow ? p.vec != 0 : VEC;
  const int len = gated_length(p, b), round = kTile * ranks;
  const float2 lg = ln.get(KIND == MHLA_GATED_DECAY ? p.g : nullptr);
  const float2 g = make_float2(least(lg.x, 0.f), least(lg.y, 0.f)), g2 = mulc(g, kLog2e);
  const bool mean = p.scale == MHLA_GATED_SCALE_MEAN;
  const float2 k1 = splat(mean ? -1.f : 0.f), k0 = splat(mean ? 0.f : 1.f);  // c = k0 + k1 m
  const float2 zero = splat(0.f);
  // the gradient that reaches a token's state from behind it
  float2 carry = ln.get(p.dstate_out ? p.dstate_out + (int64_t)b * p.D : nullptr), dg = zero;
  const bool whole = VEC == 2 && cols >= kGatedSlab;
  const int rounds = (len + round - 1) / round, mine = rank * kTile + w * kTok;

  // The walks are formed anew where they are used: kept, they would take
  // registers that the tokens need.
  auto in = [&](const void* base, const mhla_strides& s) {
    return Walk<T, const T>(static_cast<const T*>(base) + b * s.batch + first, s.token, vec);
  };
  auto out = [&](void* base, const mhla_strides& s) {
    return Walk<T, T>(static_cast<T*>(base) + b * s.batch + first, s.token, vec);
  };
  auto fetch = [&](int slot, int t0) {
    if (t0 >= 0 && t0 < len) {
      const bool fast = whole && t0 + kTok <= len;
      in(p.x, p.sx).fetch(stage[slot].x, t0, fast, len - t0, cols, vec);
      in(p.dout, p.sdo).fetch(stage[slot].d, t0, fast, len - t0, cols, vec);
      in(p.r, p.sr).fetch(stage[slot].r, t0, fast, len - t0, cols, vec);
      if constexpr (IN) in(p.i, p.si).fetch(stage[slot].i[0], t0, fast, len - t0, cols, vec);
    }
    copies_commit();
  };
  auto write = [&](const Stage<T, IN>& from, int t0) {
    if (t0 >= p.N) return;
    const bool fast = whole && t0 + kTok <= p.N;
    out(p.dx, p.sdx).write(from.x, t0, fast, p.N - t0, cols, vec);
    out(p.dr, p.sdr).write(from.r, t0, fast, p.N - t0, cols, vec);
    if constexpr (IN) out(p.di, p.sdi).write(from.i[0], t0, fast, p.N - t0, cols, vec);
  };
  auto blank = [&](Stage<T, IN>& to, int j) {
    to.x.v[j][l].zero();
    to.r.v[j][l].zero();
    if constexpr (IN) to.i[0].v[j][l].zero();
  };

  if (ranks > 1) cluster_arrive();  // nobody sends before all have begun
  if (rounds * round + mine < p.N) {  // padding
    for (int j = 0; j < kTok; ++j) blank(stage[0], j);
    for (int t0 = rounds * round + mine; t0 < p.N; t0 += round) write(stage[0], t0);
    __syncwarp();
  }
  fetch(0, (rounds - 1) * round + mine);
  __syncwarp();
  if (ranks > 1) cluster_wait();
  int turn = 0;
  for (int base = (rounds - 1) * round; base >= 0; base -= round, turn ^= 1) {
    const int t0 = base + mine;
    const bool live = t0 < len, fast = t0 + kTok <= len;  // of a whole warp
    fetch(turn ^ 1, base > 0 ? t0 - round : -1);
    float2 h = zero;  // before the first token; its load runs under the gates
    if (w % 2 == 0 && live) h = ln.get(p.marks + ((int64_t)b * p.n_marks + t0 / MHLA_GATED_MARK) * p.D);
    copies_wait<1>();
    __syncwarp();
    Stage<T, IN>& at = stage[turn];

    // From the last token: the gates, and what the tokens send to the one before
    // them.
    Gates gt[kTok];  // without m, from which c is formed
    float2 c[kTok];
    Map map = same();
    if (live) {
#pragma unroll
      for (int j = kTok - 1; j >= 0; --j) {
        gt[j] = gates_of<KIND, IN>(least_gate(at.r.v[j][l]), IN ? least_gate(at.i[0].v[j][l]) : zero, g2);
        c[j] = factor<NORM>(gt[j].m, k1, k0);
      }
      if (!fast)
#pragma unroll
        for (int j = 0; j < kTok; ++j)
          if (t0 + j >= len) gt[j].a = splat(1.f), gt[j].s = gt[j].less = c[j] = zero;  // keeps the state
#pragma unroll
      for (int j = kTok - 1; j >= 0; --j) map = then(map, Map{gt[j].a, mul2(gt[j].a, wide(at.d.v[j][l]))});
    }
    float2 e = carry;
    Map behind = same();
    if (ranks == 1) {
      if (w < kGatedWarps - 1 || base + round < rounds * round) {
        take_over(1 + w);
        e = mail[w][l].H;
      }
      carry = through(map, e);
      if (w > 0 || base > 0) {
        const int to = (w + kGatedWarps - 1) % kGatedWarps;
        mail[to][l].H = carry;
        hand_over(1 + to);
      }
    } else {
      if (w < kGatedWarps - 1) {
        take_over(1 + w);
        behind = load_map(&mail[w][l]);
      }
      const Map all = then(behind, map);
      if (w > 0) {
        store_map(&mail[w - 1][l], all);
        hand_over(w);
      } else {
        for (int v = 0; v < ranks; ++v) send(&tiles[turn][rank][l], v, all);
      }
      cluster_arrive();  // the tokens' states are formed meanwhile
    }
    if (w % 2) {
      take_over(9 + w / 2);
      h = states[w / 2][l];
    }
    float2 before[kTok];
    if (live)
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        before[j] = h;
        const float2 xv = wide(at.x.v[j][l]), u = IN ? mul2(xv, gt[j].q) : xv;
        h = fma2(gt[j].a, h, mul2(c[j], u));
      }
    if (w % 2 == 0) {
      states[w / 2][l] = h;
      hand_over(9 + w / 2);
    }
    if (ranks > 1) {
      cluster_wait();
      for (int v = ranks - 1; v > rank; --v) e = through(load_map(&tiles[turn][v][l]), e);
      carry = e;
      for (int v = rank; v >= 0; --v) carry = through(load_map(&tiles[turn][v][l]), carry);
      e = through(behind, e);
    }
    if (live)
#pragma unroll
      for (int j = kTok - 1; j >= 0; --j) {
        const float2 xv = wide(at.x.v[j][l]), u = IN ? mul2(xv, gt[j].q) : xv;
        const float2 a = gt[j].a, G = add2(e, wide(at.d.v[j][l]));
        // a h + u dc / dlog a = a (h - u a / c), or a (h + u k1)
        const float2 sum = NORM ? fma2(mul2(u, minus_inverse(c[j])), a, before[j]) : fma2(u, k1, before[j]);
        const float2 dlog = mul2(G, mul2(a, sum));
        float2 o_r = mul2(dlog, gt[j].less);
        if constexpr (KIND == MHLA_GATED_DECAY) {
          const float2 ds = mul2(dlog, gt[j].s);
          dg = add2(dg, ds);
          o_r = mul2(mul2(ds, g), gt[j].less);
        }
        const float2 du = mul2(G, c[j]), o_x = IN ? mul2(du, gt[j].q) : du;
        at.x.v[j][l] = narrow(o_x, T());
        at.r.v[j][l] = narrow(o_r, T());
        if constexpr (IN) {
          // 1 - sigma(i) as e^-i sigma(i); the power again, for it has no register
          const float2 k = mulc(least_gate(at.i[0].v[j][l]), -kLog2e), k1 = make_float2(ex2(k.x), ex2(k.y));
          at.i[0].v[j][l] = narrow(mul2(mul2(o_x, xv), mul2(gt[j].q, k1)), T());
        }
        e = mul2(a, G);
      }
    if (!fast)
      for (int j = 0; j < kTok; ++j)
        if (t0 + j >= len) blank(at, j);
    write(at, t0);
    __syncwarp();  // other lanes' copies arrive where this one has read and written
  }
  // alone, the first warp has the gradient of the first state
  if (p.dstate_in && rank == 0 && w == 0) ln.put(p.dstate_in + (int64_t)b * p.D, carry);
  if (KIND == MHLA_GATED_DECAY && p.partial) {
    start_successor();
    __syncthreads();  // the last reads of the mail
    mail[w][l].A = dg;
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int v = 1; v < kGatedWarps; ++v) dg = add2(dg, mail[v][l].A);
      ln.put(p.partial + ((int64_t)b * ranks + rank) * p.D, dg);
    }
  }
}

struct Backward {
  const GatedArgs& a;
  cudaStream_t s;
  template <typename T, int KIND, bool IN, bool NORM>
  mhla_status run() {
    constexpr bool kApart = sizeof(T) == 4;  // see kGatedNarrow
    auto kernel = a.vec == 2   ? gated_bwd_kernel<T, KIND, IN, NORM, 2>
                  : a.vec == 1 ? gated_bwd_kernel<T, KIND, IN, NORM, kApart ? 1 : kGatedNarrow>
                               : gated_bwd_kernel<T, KIND, IN, NORM, kApart ? 0 : kGatedNarrow>;
    return launch_gated_clusters(kernel, a, sizeof(T) == 4, true, 2 * kGatedWarps * sizeof(Stage<T, IN>), s);
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
