// Short causal convolution of each channel, y_t = f(sum_j w_j x_{t-K+1+j} + b),
// and its gradients: with dz_t = dout_t f'(z_t),
//   dx_s = sum_j w_j dz_{s+K-1-j},  dw_j = sum_t dz_t x_{t-K+1+j},  db = sum_t dz_t.
//
// A thread takes a few neighbouring channels and walks over a segment of the
// tokens with the last K rows in registers; the K - 1 rows before a segment
// (and, backwards, behind it) are read again by its neighbour.
//
// Bound: forward memory: 2 x 32k tokens of 1024 channels (bf16, 4 taps, SILU) take
// 51 us, 5.2 TB/s.  Backward bf16 by instructions, 58 to a pair of channels (the
// convolution and its activation are formed again): 4 x 8k tokens of 1024 channels
// take 52 us, 3.9 TB/s, of float32 68 us, 5.9 TB/s.
#include <algorithm>

#include "common.cuh"
#include "ops.h"
#include "pack.cuh"
#include "tc_host.h"

namespace mhla {
namespace {

constexpr int kThreads = 256;
// Rows of a step: a multiple of K - 1, so that the windows end it where they began
// and no register is copied.  Forward the next step's rows are on their way to
// registers, backward those of kAhead steps to shared memory.
constexpr int kFwdRows = 6, kAhead = 2;
template <int K>
constexpr int kBwdRows = K == 3 ? 2 : 3;

enum { kForward, kBackward, kStep };

// CTAs that an SM holds: their registers.
constexpr int resident(int what, int elem) { return what == kForward && elem == 2 ? 3 : 2; }

struct ConvArgs {
  const void *x, *dout, *w, *bias, *state_in, *dstate_out;
  void *out, *state_out, *dx, *dstate_in;
  mhla_strides sx, so, sdo, sdx;
  const int32_t* lengths;
  float* partial;  // [rows][K + 1][D]
  int B, N, D;
  int w_f32, silu;
  int width;           // channels of a thread
  int vecs;            // of a row
  int across, down;    // of a CTA: vectors and segments, powers of two
  int across_shift;
  int columns;         // CTAs to the channels of a segment; neighbours in the grid
  int segments, seg;   // segments of a sequence, tokens of one
  int whole;           // vectors in one access
};

__device__ __forceinline__ int length_of(const ConvArgs& p, int b) {
  if (!p.lengths) return p.N;
  const int n = p.lengths[b];
  return n < 0 ? 0 : n > p.N ? p.N : n;
}

// A thread's channels, sequence and segment.
struct Place {
  int ch, n, b, first;
  int down, first_vec;  // of the CTA
  bool live;
  __device__ __forceinline__ Place(const ConvArgs& p) {
    down = blockIdx.x / p.columns;
    first_vec = (blockIdx.x - down * p.columns) * p.across;
    const int vec = first_vec + (threadIdx.x & (p.across - 1));
    const int64_t at = (int64_t)down * p.down + (threadIdx.x >> p.across_shift);
    b = (int)(at / p.segments);
    first = (int)(at - (int64_t)b * p.segments) * p.seg;
    ch = vec * p.width;
    n = min(p.width, p.D - ch);
    live = vec < p.vecs && b < p.B;
  }
};

// Channel pairs of a thread's weights and bias.
template <int V, typename W, int K>
__device__ __forceinline__ void load_weights_as(const ConvArgs& p, const Place& at, float (&w)[V][K],
                                                float (&bias)[V]) {
  const W *pw = static_cast<const W*>(p.w) + (int64_t)at.ch * K, *pb = static_cast<const W*>(p.bias) + at.ch;
  if (at.n == V) {
#pragma unroll
    for (int i = 0; i < V * K; ++i) w[i / K][i % K] = to_f32(pw[i]);
#pragma unroll
    for (int c = 0; c < V; ++c) bias[c] = p.bias ? to_f32(pb[c]) : 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < V * K; ++i) w[i / K][i % K] = i < at.n * K ? to_f32(pw[i]) : 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) bias[c] = p.bias && c < at.n ? to_f32(pb[c]) : 0.f;
  }
}
template <int V, int K>
__device__ __forceinline__ void load_weights(const ConvArgs& p, const Place& at, float2 (&w)[K][V / 2],
                                             float2 (&bias)[V / 2]) {
  float f[V][K], g[V];
  if (p.w_f32)
    load_weights_as<V, float, K>(p, at, f, g);
  else
    load_weights_as<V, __nv_bfloat16, K>(p, at, f, g);
#pragma unroll
  for (int c = 0; c < V / 2; ++c) {
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][c] = make_float2(f[2 * c][j], f[2 * c + 1][j]);
    bias[c] = make_float2(g[2 * c], g[2 * c + 1]);
  }
}

// 1 / (1 + e^-z)
__device__ __forceinline__ float2 logistic(float2 z) {
  const float2 y = mul2(z, splat(-kLog2e));
  const float2 d = add2(make_float2(ex2(y.x), ex2(y.y)), splat(1.f));
  return make_float2(rcp(d.x), rcp(d.y));
}

// Row t of x, rows before the first token from the incoming state, zeros past
// the length.
template <int V, typename T, int K>
__device__ __forceinline__ void load_row(const ConvArgs& p, const Place& at, int t, int len, Pack<T, V>* r) {
  if (t >= len || !at.live) {
    r->zero();
  } else if (t >= 0) {
    r->load(static_cast<const T*>(p.x) + at.b * p.sx.batch + t * p.sx.token + at.ch, p.whole && at.n == V, at.n);
  } else if (p.state_in) {
    r->load(static_cast<const T*>(p.state_in) + ((int64_t)at.b * (K - 1) + t + K - 1) * p.D + at.ch, false, at.n);
  } else {
    r->zero();
  }
}

// A thread's V elements of a row, by asynchronous copies into a place of its own.
// SINGLE: rows start at single elements, and `n` of the V are there.  bf16 then
// comes in words, the first and last of which may hold a neighbour's element (of
// the same tensor, which lies between lo and hi), and is shifted when it is used.
template <typename T, int V, bool SINGLE>
struct Slot {
  static constexpr bool kWords = SINGLE && sizeof(T) == 2;
  static_assert(!kWords || V == 4, "three words");
  alignas(kWords ? 16 : V * sizeof(T)) unsigned char v[kWords ? 16 : V * sizeof(T)];
  __device__ __forceinline__ void start(const T* from, int n, const T* lo, const T* hi) {
    if constexpr (kWords) {
      const int odd = (int)((uintptr_t)from >> 1) & 1, words = (n + odd + 1) >> 1;
      const T* first = from - odd;
      if (first >= lo && first + 2 * words <= hi) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (i < words) copy_async<4>(v + 4 * i, first + 2 * i, 4);
      } else {  // the tensor's first or last element
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < n) reinterpret_cast<T*>(v)[odd + i] = from[i];
      }
    } else if constexpr (SINGLE) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) copy_async<sizeof(T)>(v + sizeof(T) * i, from + i, sizeof(T));
    } else {
      copy_async<V * (int)sizeof(T)>(v, from, V * (int)sizeof(T));
    }
  }
  __device__ __forceinline__ Pack<T, V> take(const T* from) const {
    if constexpr (kWords) {
      const uint4 w = *reinterpret_cast<const uint4*>(v);
      const int shift = (int)((uintptr_t)from >> 1 & 1) * 16;
      Pack<T, V> r;
      reinterpret_cast<uint32_t*>(r.v)[0] = __funnelshift_r(w.x, w.y, shift);
      reinterpret_cast<uint32_t*>(r.v)[1] = __funnelshift_r(w.y, w.z, shift);
      return r;
    } else {
      return *reinterpret_cast<const Pack<T, V>*>(v);
    }
  }
  // Writes a row's elements.
  __device__ __forceinline__ static void store(T* to, const Pack<T, V>& r, int n) {
    if (SINGLE && n < V) {
      r.store(to, false, n);
    } else if constexpr (kWords) {
      const uint32_t a = reinterpret_cast<const uint32_t*>(r.v)[0], b = reinterpret_cast<const uint32_t*>(r.v)[1];
      if ((uintptr_t)to & 2) {
        to[0] = r.v[0];
        *reinterpret_cast<uint32_t*>(to + 1) = __funnelshift_r(a, b, 16);
        to[3] = r.v[3];
      } else {
        reinterpret_cast<uint32_t*>(to)[0] = a;
        reinterpret_cast<uint32_t*>(to)[1] = b;
      }
    } else {
      r.store(to, !SINGLE);
    }
  }
};

// One behind the last element of a tensor.
template <typename T>
__device__ __forceinline__ const T* end_of(const ConvArgs& p, const void* t, const mhla_strides& s) {
  return static_cast<const T*>(t) + (p.B - 1) * s.batch + (p.N - 1) * s.token + p.D;
}

template <typename T, int K, int V, bool SINGLE>
__global__ void __launch_bounds__(kThreads, resident(kForward, sizeof(T)))
    conv_fwd_kernel(const __grid_constant__ ConvArgs p) {
  constexpr int H = V / 2;
  using Row = Slot<T, V, SINGLE>;
  extern __shared__ __align__(16) unsigned char dynamic[];  // SINGLE: rows on their way
  const Place at(p);
  if (!at.live) return;
  const int len = length_of(p, at.b), last = min(at.first + p.seg, p.N);
  float2 w[K][H], bias[H];
  load_weights<V, K>(p, at, w, bias);
  float2 win[K - 1][H];  // rows t - K + 1 .. t - 1
  Pack<T, V> r;
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    load_row<V, T, K>(p, at, at.first - (K - 1) + j, len, &r);
#pragma unroll
    for (int c = 0; c < H; ++c) win[j][c] = pair_of(r, c);
  }
  const T* x = static_cast<const T*>(p.x) + at.b * p.sx.batch + at.ch;
  T* out = static_cast<T*>(p.out) + at.b * p.so.batch + at.ch;
  const bool whole = !SINGLE && p.whole && at.n == V;
  const int inside = SINGLE || whole ? min(last, len) : at.first;  // steps up to here need no checks
  constexpr int R = SINGLE ? kBwdRows<K> : kFwdRows;
  auto fetch = [&](Pack<T, V>(&to)[R], int t0) {
    if (t0 + R <= inside) {
      const T* from = x + t0 * p.sx.token;
#pragma unroll
      for (int u = 0; u < R; ++u, from += p.sx.token) to[u].load(from, true);
    } else if (t0 < last) {
#pragma unroll
      for (int u = 0; u < R; ++u) load_row<V, T, K>(p, at, t0 + u, len, &to[u]);
    }
  };
  auto step = [&](const Pack<T, V>(&row)[R], int t0) {
    T* to = out + t0 * p.so.token;
#pragma unroll
    for (int u = 0; u < R; ++u, to += p.so.token) {
      const int t = t0 + u;
      Pack<T, V> o;
#pragma unroll
      for (int c = 0; c < H; ++c) {
        const float2 xv = pair_of(row[u], c);
        float2 z = fma2(w[K - 1][c], xv, bias[c]);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) z = fma2(w[j][c], win[j][c], z);
#pragma unroll
        for (int j = 0; j + 1 < K - 1; ++j) win[j][c] = win[j + 1][c];
        win[K - 2][c] = xv;
        if (p.silu) z = mul2(z, logistic(z));
        put_pair(&o, c, z);
      }
      if (t0 + R <= inside) {
        Row::store(to, o, at.n);
      } else if (t < last) {
        if (t >= len) o.zero();
        o.store(to, whole, at.n);
      }
    }
  };
  auto pad = [&](int t0) {
    r.zero();
    for (int t = t0; t < last; ++t) r.store(out + t * p.so.token, whole, at.n);
  };
  if constexpr (SINGLE) {
    const T* x_end = end_of<T>(p, p.x, p.sx);
    Row* places = reinterpret_cast<Row*>(dynamic) + threadIdx.x;
    int put = 0, got = 0;
    auto start = [&](int t0) {
      const T* from = x + t0 * p.sx.token;
#pragma unroll
      for (int u = 0; u < R; ++u, from += p.sx.token)
        if (t0 + u < inside) places[(put * R + u) * kThreads].start(from, at.n, static_cast<const T*>(p.x), x_end);
      copies_commit();
      put = put < kAhead ? put + 1 : 0;
    };
    for (int i = 0; i < kAhead; ++i) start(at.first + i * R);
    for (int t0 = at.first; t0 < last; t0 += R) {
      if (t0 >= len) {
        pad(t0);
        break;
      }
      start(t0 + kAhead * R);
      copies_wait<kAhead>();
      Pack<T, V> row[R];
#pragma unroll
      for (int u = 0; u < R; ++u) {
        row[u].zero();
        if (t0 + u < inside) row[u] = places[(got * R + u) * kThreads].take(x + (t0 + u) * p.sx.token);
      }
      got = got < kAhead ? got + 1 : 0;
      step(row, t0);
    }
  } else {
    Pack<T, V> rows[2][R];
    fetch(rows[0], at.first);
    for (int t0 = at.first; t0 < last; t0 += 2 * R) {
      if (t0 >= len) {
        pad(t0);
        break;
      }
      fetch(rows[1], t0 + R);
      step(rows[0], t0);
      if (t0 + R >= last) break;
      fetch(rows[0], t0 + 2 * R);
      step(rows[1], t0 + R);
    }
  }
  if (p.state_out && at.first == 0) {
    // the same thread that read state_in, which this may be
    Pack<T, V> keep[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) load_row<V, T, K>(p, at, len - (K - 1) + j, len, &keep[j]);
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
      keep[j].store(static_cast<T*>(p.state_out) + ((int64_t)at.b * (K - 1) + j) * p.D + at.ch, false, at.n);
  }
}

template <typename T, int K, int V, bool SINGLE>
__global__ void __launch_bounds__(kThreads, resident(kBackward, sizeof(T)))
    conv_bwd_kernel(const __grid_constant__ ConvArgs p) {
  constexpr int H = V / 2, R = kBwdRows<K>;
  using Row = Slot<T, V, SINGLE>;
  extern __shared__ __align__(16) float sums[];  // rows on their way; then [down][(K + 1) * V][across]
  const Place at(p);
  float2 dw[K + 1][H];
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int c = 0; c < H; ++c) dw[j][c] = splat(0.f);
  if (at.live) {
    const int len = length_of(p, at.b), last = min(at.first + p.seg, p.N), end = last + K - 1;
    float2 w[K][H], bias[H];
    load_weights<V, K>(p, at, w, bias);
    float2 win[K - 1][H], dz[K - 1][H];  // rows t - K + 1 .. t - 1 of x and of dL/dz
    Pack<T, V> r;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      load_row<V, T, K>(p, at, at.first - (K - 1) + j, len, &r);
#pragma unroll
      for (int c = 0; c < H; ++c) {
        win[j][c] = pair_of(r, c);
        dz[j][c] = splat(0.f);
      }
    }
    const bool whole = !SINGLE && p.whole && at.n == V;
    const bool quick = SINGLE || whole;
    const T* x = static_cast<const T*>(p.x) + at.b * p.sx.batch + at.ch;
    const T* dout = static_cast<const T*>(p.dout) + at.b * p.sdo.batch + at.ch;
    T* dx = static_cast<T*>(p.dx) + at.b * p.sdx.batch + at.ch;
    const T *x_end = end_of<T>(p, p.x, p.sx), *dout_end = end_of<T>(p, p.dout, p.sdo);
    // Steps inside need no checks: their rows are before the length and the
    // segment's end, and the rows s = t - (K - 1) of dx not before its start.
    auto inside = [&](int t0) { return quick && t0 >= at.first + K - 1 && t0 + R <= min(last, len); };
    // Rows of x and dout go through shared memory of the thread's own.
    const int copied = quick ? min(end, len) : at.first;
    auto place = [&](int slot, int u, int which) {
      return reinterpret_cast<Row*>(sums) + ((slot * R + u) * 2 + which) * kThreads + threadIdx.x;
    };
    int put = 0, got = 0;
    auto fetch = [&](int t0) {
      const T *from = x + t0 * p.sx.token, *fromd = dout + t0 * p.sdo.token;
      const bool all = t0 + R <= copied;
#pragma unroll
      for (int u = 0; u < R; ++u, from += p.sx.token, fromd += p.sdo.token)
        if (all || t0 + u < copied) {
          place(put, u, 0)->start(from, at.n, static_cast<const T*>(p.x), x_end);
          place(put, u, 1)->start(fromd, at.n, static_cast<const T*>(p.dout), dout_end);
        }
      copies_commit();
      put = put < kAhead ? put + 1 : 0;
    };
    for (int i = 0; i < kAhead; ++i) fetch(at.first + i * R);
    Pack<T, V> row[R], rd[R];
    // The rows of a step, `fast` (a constant where it is called, as `silu`) inside.
    auto step = [&](bool fast, bool silu, int t0) {
      T* to = dx + (t0 - (K - 1)) * p.sdx.token;
#pragma unroll
      for (int u = 0; u < R; ++u, to += p.sdx.token) {
        const int t = t0 + u, s = t - (K - 1);
        float2 o[H];
#pragma unroll
        for (int c = 0; c < H; ++c) {
          const float2 xv = pair_of(row[u], c);
          float2 d = pair_of(rd[u], c);
          if (silu) {
            float2 z = fma2(w[K - 1][c], xv, bias[c]);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) z = fma2(w[j][c], win[j][c], z);
            // q (1 + z (1 - q))
            const float2 q = logistic(z), zq = mul2(z, q);
            d = mul2(d, fma2(zq, fma2(q, splat(-1.f), splat(1.f)), q));
          }
          if (!fast && t >= len) d = splat(0.f);
          const float2 own = fast || t < last ? d : splat(0.f);
#pragma unroll
          for (int j = 0; j < K - 1; ++j) dw[j][c] = fma2(own, win[j][c], dw[j][c]);
          dw[K - 1][c] = fma2(own, xv, dw[K - 1][c]);
          dw[K][c] = add2(dw[K][c], own);
          // dz_{s + i} meets w_{K - 1 - i}; d is dz_{s + K - 1}
          o[c] = mul2(w[0][c], d);
#pragma unroll
          for (int i = 0; i < K - 1; ++i) o[c] = fma2(w[K - 1 - i][c], dz[i][c], o[c]);
#pragma unroll
          for (int j = 0; j + 1 < K - 1; ++j) {
            win[j][c] = win[j + 1][c];
            dz[j][c] = dz[j + 1][c];
          }
          win[K - 2][c] = xv;
          dz[K - 2][c] = d;
        }
        if (fast) {
#pragma unroll
          for (int c = 0; c < H; ++c) put_pair(&r, c, o[c]);
          Row::store(to, r, at.n);
        } else {
          const int extra = s - (len - (K - 1));
          if (t >= end || s < at.first - (at.first == 0 ? K - 1 : 0)) continue;
          if (p.dstate_out && extra >= 0 && extra < K - 1) {  // the row went into the outgoing state
            r.load(static_cast<const T*>(p.dstate_out) + ((int64_t)at.b * (K - 1) + extra) * p.D + at.ch, false, at.n);
#pragma unroll
            for (int c = 0; c < H; ++c) o[c] = add2(o[c], pair_of(r, c));
          }
#pragma unroll
          for (int c = 0; c < H; ++c) put_pair(&r, c, s < len ? o[c] : splat(0.f));
          if (s >= 0)
            r.store(dx + s * p.sdx.token, whole, at.n);
          else if (p.dstate_in)
            r.store(static_cast<T*>(p.dstate_in) + ((int64_t)at.b * (K - 1) + s + K - 1) * p.D + at.ch, false, at.n);
        }
      }
    };
    // Rows s < first belong to the segment before, but the first one's are the
    // incoming state's.
    for (int t0 = at.first; t0 < end; t0 += R) {
      if (t0 - (K - 1) >= max(len, at.first)) {  // padding
        r.zero();
        for (int s = t0 - (K - 1); s < last; ++s) r.store(dx + s * p.sdx.token, whole, at.n);
        break;
      }
      fetch(t0 + kAhead * R);
      copies_wait<kAhead>();
      if (inside(t0)) {
#pragma unroll
        for (int u = 0; u < R; ++u) {
          row[u] = place(got, u, 0)->take(x + (t0 + u) * p.sx.token);
          rd[u] = place(got, u, 1)->take(dout + (t0 + u) * p.sdo.token);
        }
        if (p.silu)
          step(true, true, t0);
        else
          step(true, false, t0);
      } else {
#pragma unroll
        for (int u = 0; u < R; ++u) {
          const int t = t0 + u;
          if (t < copied) {
            row[u] = place(got, u, 0)->take(x + t * p.sx.token);
            rd[u] = place(got, u, 1)->take(dout + t * p.sdo.token);
          } else {
            load_row<V, T, K>(p, at, t, t < end ? len : 0, &row[u]);
            rd[u].zero();
            if (t < min(end, len)) rd[u].load(dout + t * p.sdo.token, whole, at.n);
          }
        }
        step(false, p.silu, t0);
      }
      got = got < kAhead ? got + 1 : 0;
    }
  }
  if (!p.partial) return;
  start_successor();
  __syncthreads();  // the rows' places are free
  const int a = threadIdx.x & (p.across - 1), d = threadIdx.x >> p.across_shift;
  constexpr int kSums = (K + 1) * V;
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int c = 0; c < V; ++c)
      sums[(d * kSums + j * V + c) * p.across + a] = c % 2 ? dw[j][c / 2].y : dw[j][c / 2].x;
  __syncthreads();
  for (int i = threadIdx.x; i < kSums * p.across; i += kThreads) {
    const int vec = at.first_vec + i % p.across, j = i / p.across / V, c = i / p.across % V;
    if (vec * V + c >= p.D) continue;
    float s = 0.f;
    for (int v = 0; v < p.down; ++v) s += sums[v * kSums * p.across + i];
    p.partial[((int64_t)at.down * (K + 1) + j) * p.D + vec * V + c] = s;
  }
}

// Adds the partial rows in order: 32 channels per CTA, 32 threads to one.
__global__ void __launch_bounds__(1024) conv_reduce_kernel(const float* partial, int rows, int K, int D, float* dweight,
                                                           float* dbias) {
  __shared__ float sh[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx, j = blockIdx.y;
  float s = 0.f;
  after_predecessor();
  if (c < D)
    for (int r = ty; r < rows; r += 32) s += partial[((int64_t)r * (K + 1) + j) * D + c];
  sh[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && c < D) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += sh[i][tx];
    if (j < K) {
      if (dweight) dweight[(int64_t)c * K + j] = t;
    } else if (dbias) {
      dbias[c] = t;
    }
  }
}

// One token of every sequence.
template <typename T, int K>
__global__ void __launch_bounds__(128) conv_step_kernel(const __grid_constant__ ConvArgs p) {
  const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (i >= (int64_t)p.B * p.D) return;
  const int64_t b = i / p.D;
  const int ch = (int)(i - b * p.D);
  const T x = static_cast<const T*>(p.x)[b * p.sx.batch + ch];
  T row[K];
#pragma unroll
  for (int j = 0; j < K - 1; ++j)
    row[j] = p.state_in ? static_cast<const T*>(p.state_in)[(b * (K - 1) + j) * p.D + ch] : from_f32<T>(0.f);
  row[K - 1] = x;
  // the forward kernel's order, so that tokens give the same bits either way
  const float bias = p.bias ? param_at(p.bias, p.w_f32, ch) : 0.f;
  float z = fmaf(param_at(p.w, p.w_f32, (int64_t)ch * K + K - 1), to_f32(x), bias);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) z = fmaf(param_at(p.w, p.w_f32, (int64_t)ch * K + j), to_f32(row[j]), z);
  if (p.silu) z = z * rcp(1.f + ex2(-z * kLog2e));
  static_cast<T*>(p.out)[b * p.so.batch + ch] = from_f32<T>(z);
  if (p.state_out)
#pragma unroll
    for (int j = 0; j < K - 1; ++j) static_cast<T*>(p.state_out)[(b * (K - 1) + j) * p.D + ch] = row[j + 1];
}

// ---------------------------------------------------------------- dispatch

// Threads of a CTA across the channels and down the tokens, and the tokens of
// a segment: those with the least time, counted in rows that one thread takes
// after another -- a segment's own and about 16 for its weights and borders --
// over the waves of CTAs that the GPU holds at once.
void shape(ConvArgs* p, int what, int dtype) {
  p->vecs = (p->D + p->width - 1) / p->width;
  p->across = 1;
  p->across_shift = 0;
  while (p->across < 32 && p->across < p->vecs) {
    p->across *= 2;
    ++p->across_shift;
  }
  p->down = kThreads / p->across;
  p->columns = (p->vecs + p->across - 1) / p->across;
  const int64_t slots = (int64_t)kOpsSms * resident(what, (int)ops_elem(dtype));
  int64_t best = 0;
  for (int seg = 8; seg <= 256; seg += 4) {
    const int64_t segments = p->N > 0 ? ((int64_t)p->N + seg - 1) / seg : 1;
    const int64_t ctas = p->columns * (((int64_t)p->B * segments + p->down - 1) / p->down);
    const int64_t cost = (ctas + slots - 1) / slots * (seg + 16);
    if (seg == 8 || cost < best) {
      best = cost;
      p->seg = seg;
      p->segments = (int)segments;
    }
  }
}

int64_t grid_down(const ConvArgs& p) { return ((int64_t)p.B * p.segments + p.down - 1) / p.down; }

// Bytes of the backward pass's partial sums in this shape.
size_t sums_bytes(const ConvArgs& p, int taps) {
  return sizeof(float) * (size_t)grid_down(p) * (taps + 1) * (size_t)p.D;
}

template <typename T, int K>
mhla_status launch(const ConvArgs& a, int what, cudaStream_t s) {
  if (what == kStep) {
    const int64_t blocks = ((int64_t)a.B * a.D + 127) / 128;
    if (blocks > 0x7fffffff) return MHLA_ERR_UNSUPPORTED;
    conv_step_kernel<T, K><<<(unsigned)blocks, 128, 0, s>>>(a);
    return launch_status();
  }
  const unsigned grid = (unsigned)(a.columns * grid_down(a));
  constexpr int kBack = sizeof(T) == 4 ? 2 : 4;  // see choose_width
  if (what == kForward) {
    auto kernel = a.whole ? conv_fwd_kernel<T, K, 4, false> : conv_fwd_kernel<T, K, 4, true>;
    if constexpr (sizeof(T) == 2)
      if (a.width == 2) kernel = conv_fwd_kernel<T, K, 2, false>;
    // at most 36 KB
    const size_t smem = a.whole ? 0 : sizeof(Slot<T, 4, true>) * kBwdRows<K> * (kAhead + 1) * kThreads;
    kernel<<<grid, kThreads, smem, s>>>(a);
    return launch_status();
  }
  auto kernel = a.whole ? conv_bwd_kernel<T, K, kBack, false> : conv_bwd_kernel<T, K, kBack, true>;
  if constexpr (sizeof(T) == 2)
    if (a.width == 2) kernel = conv_bwd_kernel<T, K, 2, false>;
  // the rows on their way, then the sums
  const size_t slot = a.whole ? sizeof(T) * a.width : sizeof(Slot<T, kBack, true>);
  const size_t rows = slot * 2 * kBwdRows<K> * (kAhead + 1) * kThreads;
  const size_t sums = a.partial ? sizeof(float) * (K + 1) * a.width * kThreads : 0, smem = rows > sums ? rows : sums;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return record_cuda_error(e);
  kernel<<<grid, kThreads, smem, s>>>(a);
  return launch_status();
}

template <typename T>
mhla_status with_taps(const ConvArgs& a, int taps, int what, cudaStream_t s) {
  if (taps == 2) return launch<T, 2>(a, what, s);
  if (taps == 3) return launch<T, 3>(a, what, s);
  return launch<T, 4>(a, what, s);
}

mhla_status dispatch(const ConvArgs& a, const mhla_shortconv_params* p, int what, cudaStream_t s) {
  if (what != kStep && a.columns * grid_down(a) > 0x7fffffff) return MHLA_ERR_UNSUPPORTED;
  return p->dtype == MHLA_DTYPE_BF16 ? with_taps<__nv_bfloat16>(a, p->taps, what, s)
                                     : with_taps<float>(a, p->taps, what, s);
}

mhla_status check_params(const mhla_shortconv_params* p) {
  if (!p || p->batch < 0 || p->tokens < 0 || p->width < 0 || !ops_dtype_ok(p->dtype) || !ops_dtype_ok(p->weight_dtype))
    return MHLA_ERR_INVALID_ARG;
  if (p->activation != MHLA_ACTIVATION_NONE && p->activation != MHLA_ACTIVATION_SILU) return MHLA_ERR_INVALID_ARG;
  if (p->taps < 1) return MHLA_ERR_INVALID_ARG;
  if (p->taps < 2 || p->taps > 4 || p->tokens > 0x7fffff00 || p->width > 0x7fffff00) return MHLA_ERR_UNSUPPORTED;
  return MHLA_OK;
}

RowTensor rows(const void* ptr, const mhla_shortconv_params* p, const mhla_strides& s) {
  return row_tensor(ptr, p->batch, 1, p->tokens, s, p->width, ops_elem(p->dtype));
}
// a state, contiguous, or NULL
RowTensor state_of(const void* ptr, const mhla_shortconv_params* p) {
  return flat_tensor(ptr, ptr ? (int64_t)p->batch * (p->taps - 1) * p->width : 0, ops_elem(p->dtype));
}
RowTensor param_of(const void* ptr, int64_t n, int dtype) { return flat_tensor(ptr, ptr ? n : 0, ops_elem(dtype)); }

// Inputs may share memory, results nothing with one another or with an input
// but out[same_out] with in[same_in].
bool apart(const RowTensor* in, int n_in, const RowTensor* out, int n_out, int same_in, int same_out) {
  for (int i = 0; i < n_in; ++i)
    if (!row_tensor_ok(in[i], false)) return false;
  for (int o = 0; o < n_out; ++o) {
    if (!row_tensor_ok(out[o], true)) return false;
    for (int i = 0; i < n_in; ++i) {
      if (i == same_in && o == same_out && row_tensors_same(in[i], out[o])) continue;
      if (!row_tensors_apart(in[i], out[o])) return false;
    }
    for (int q = o + 1; q < n_out; ++q)
      if (!row_tensors_apart(out[o], out[q])) return false;
  }
  return true;
}

// Channels of a thread: four, in one access where rows allow it, but two of
// float32 in the backward pass, whose registers they fill (4 x 8k x 1024: 68 us,
// with four 74), and two of bf16 where rows start at pairs only (4 x 4k x 1030:
// forward 21 and backward 36 us; of 1001, in words of shared memory, 25 and 54,
// element by element 31 and 88).
void choose_width(ConvArgs* a, const RowTensor* t, int n, const RowTensor& last, int dtype, bool backward) {
  int align = row_alignment(last, 16);
  for (int i = 0; i < n; ++i) {
    const int x = t[i].empty() ? 16 : row_alignment(t[i], 16);
    align = x < align ? x : align;
  }
  const int elem = (int)ops_elem(dtype);
  const bool two = dtype == MHLA_DTYPE_F32 ? backward : align == 2 * elem;
  a->width = two ? 2 : 4;
  a->whole = align >= a->width * elem;
}

ConvArgs args_of(const mhla_shortconv_params* p, const void* x, const void* weight, const void* bias,
                 const int32_t* lengths, const void* state_in) {
  ConvArgs a = {};
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.lengths = lengths;
  a.state_in = state_in;
  a.sx = p->x;
  a.B = p->batch;
  a.N = p->tokens;
  a.D = p->width;
  a.w_f32 = p->weight_dtype == MHLA_DTYPE_F32;
  a.silu = p->activation == MHLA_ACTIVATION_SILU;
  return a;
}

}  // namespace
}  // namespace mhla

extern "C" {

mhla_status mhla_shortconv_forward(const void* x, const void* weight, const void* bias, const int32_t* lengths,
                                   const void* state_in, const mhla_shortconv_params* p, void* out, void* state_out,
                                   void* stream) {
  using namespace mhla;
  const mhla_status st = check_params(p);
  if (st != MHLA_OK) return st;
  if (!weight && p->width) return MHLA_ERR_INVALID_ARG;
  const RowTensor in[5] = {rows(x, p, p->x), param_of(weight, (int64_t)p->width * p->taps, p->weight_dtype),
                           param_of(bias, p->width, p->weight_dtype), flat_tensor(lengths, lengths ? p->batch : 0, 4),
                           state_of(state_in, p)};
  const RowTensor res[2] = {rows(out, p, p->out), state_of(state_out, p)};
  if (!apart(in, 5, res, 2, 4, 1)) return MHLA_ERR_INVALID_ARG;
  if (p->batch == 0 || p->width == 0) return MHLA_OK;
  ConvArgs a = args_of(p, x, weight, bias, lengths, state_in);
  a.out = out;
  a.so = p->out;
  a.state_out = state_out;
  choose_width(&a, in, 1, res[0], p->dtype, false);
  shape(&a, kForward, p->dtype);
  return dispatch(a, p, kForward, static_cast<cudaStream_t>(stream));
}

mhla_status mhla_shortconv_backward_workspace_bytes(const mhla_shortconv_params* p, size_t* bytes) {
  using namespace mhla;
  if (!bytes) return MHLA_ERR_INVALID_ARG;
  const mhla_status st = check_params(p);
  if (st != MHLA_OK) return st;
  ConvArgs a = args_of(p, nullptr, nullptr, nullptr, nullptr, nullptr);
  *bytes = 0;
  for (a.width = 2; a.width <= 4 && p->batch && p->width; a.width += 2) {  // whatever the pointers' alignment
    shape(&a, kBackward, p->dtype);
    *bytes = std::max(*bytes, sums_bytes(a, p->taps));
  }
  return MHLA_OK;
}

mhla_status mhla_shortconv_backward(const void* x, const void* weight, const void* bias, const int32_t* lengths,
                                    const void* state_in, const void* dout, const void* dstate_out,
                                    const mhla_shortconv_params* p, void* dx, float* dweight, float* dbias,
                                    void* dstate_in, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace mhla;
  mhla_status st = check_params(p);
  if (st != MHLA_OK) return st;
  if (!weight && p->width) return MHLA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool sums = dweight || dbias;
  size_t need = 0;
  if (sums && (st = mhla_shortconv_backward_workspace_bytes(p, &need)) != MHLA_OK) return st;
  const RowTensor in[7] = {rows(x, p, p->x), rows(dout, p, p->dout),
                           param_of(weight, (int64_t)p->width * p->taps, p->weight_dtype),
                           param_of(bias, p->width, p->weight_dtype), flat_tensor(lengths, lengths ? p->batch : 0, 4),
                           state_of(state_in, p), state_of(dstate_out, p)};
  const RowTensor res[5] = {rows(dx, p, p->dx), param_of(dweight, (int64_t)p->width * p->taps, MHLA_DTYPE_F32),
                            param_of(dbias, p->width, MHLA_DTYPE_F32), state_of(dstate_in, p),
                            flat_tensor(workspace, workspace ? (int64_t)need : 0, 1)};
  if (!apart(in, 7, res, 5, -1, -1)) return MHLA_ERR_INVALID_ARG;
  if (p->batch == 0 || p->width == 0) {  // empty sums
    cudaError_t e = cudaSuccess;
    if (dweight && p->width) e = cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)p->width * p->taps, s);
    if (e == cudaSuccess && dbias && p->width) e = cudaMemsetAsync(dbias, 0, sizeof(float) * (size_t)p->width, s);
    return e == cudaSuccess ? MHLA_OK : record_cuda_error(e);
  }
  ConvArgs a = args_of(p, x, weight, bias, lengths, state_in);
  choose_width(&a, in, 2, res[0], p->dtype, true);
  shape(&a, kBackward, p->dtype);
  // the launch's own shape has the last word on what its sums need
  Scratch scratch;
  if (sums && (st = scratch.take(workspace, workspace_bytes, std::max(need, sums_bytes(a, p->taps)), s)) != MHLA_OK)
    return st;
  a.dout = dout;
  a.sdo = p->dout;
  a.dstate_out = dstate_out;
  a.dx = dx;
  a.sdx = p->dx;
  a.dstate_in = dstate_in;
  a.partial = sums ? reinterpret_cast<float*>(scratch.ptr()) : nullptr;
  st = dispatch(a, p, kBackward, s);
  if (st == MHLA_OK && sums) {
    const dim3 grid((unsigned)((p->width + 31) / 32), (unsigned)(p->taps + 1));
    const int e = launch_pdl(conv_reduce_kernel, grid, dim3(1024), 0, s, (const float*)a.partial, (int)grid_down(a),
                             p->taps, p->width, dweight, dbias);
    if (e != cudaSuccess) st = record_cuda_error((cudaError_t)e);
  }
  return scratch.give_back(st);
}

mhla_status mhla_shortconv_step(const void* x, const void* weight, const void* bias, const void* state_in,
                                const mhla_shortconv_params* p, void* out, void* state_out, void* stream) {
  using namespace mhla;
  const mhla_status st = check_params(p);
  if (st != MHLA_OK) return st;
  if (p->tokens != 1 || (!weight && p->width)) return MHLA_ERR_INVALID_ARG;
  const RowTensor in[4] = {rows(x, p, p->x), param_of(weight, (int64_t)p->width * p->taps, p->weight_dtype),
                           param_of(bias, p->width, p->weight_dtype), state_of(state_in, p)};
  const RowTensor res[2] = {rows(out, p, p->out), state_of(state_out, p)};
  if (!apart(in, 4, res, 2, 3, 1)) return MHLA_ERR_INVALID_ARG;
  if (p->batch == 0 || p->width == 0) return MHLA_OK;
  ConvArgs a = args_of(p, x, weight, bias, nullptr, state_in);
  a.out = out;
  a.so = p->out;
  a.state_out = state_out;
  return dispatch(a, p, kStep, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
