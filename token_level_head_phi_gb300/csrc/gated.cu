// Linear recurrence with gates of each token and channel:
//   h_t = a_t h_{t-1} + c_t u_t,   u_t = x_t sigma(i_t)
//   a_t = exp(log_decay sigma(r_t)) or sigma(r_t),   c_t = sqrt(1 - a_t^2), 1 - a_t or 1
// and its gradients: with G_t = dout_t + a_{t+1} G_{t+1},
//   dlog a_t = G_t (a_t h_{t-1} + u_t dc_t / dlog a_t),   du_t = G_t c_t.
// Both recurrences are scans of the maps h -> A h + H, which compose.
//
// A CTA takes 64 channels of one sequence, tile by tile of 64 tokens: a warp 8
// tokens, a lane two channels.  Each warp forms the map of its 8 tokens in
// registers, the maps meet in shared memory behind one barrier, and a second
// walk over the same registers writes the results from the state that each
// warp starts with.  Every input is read once.  The backward pass walks the
// tiles from the last one; the states inside a tile come from the state before
// it, which the forward pass keeps in float32 for every 64th token (3 % of
// the inputs' bytes).
//
// a is formed as 1 + expm1(log a): its rounding (2^-25 next to 1) is multiplied
// with itself over all the tokens that a slow channel remembers, so a float32
// exponential's last bit, which errs to one side, would show (the final state
// of 32k tokens 4.5e-6 off instead of 3e-7).
#include <cmath>

#include "common.cuh"
#include "ops.h"
#include "pack.cuh"

namespace mhla {
namespace {

constexpr int kWarps = 8, kTok = 8, kTile = kWarps * kTok;  // tokens of a tile
constexpr int kSlab = 64;                                   // channels of a CTA
constexpr int kThreads = 32 * kWarps;
static_assert(kTile == MHLA_GATED_MARK, "a tile starts at a mark");

struct GatedArgs {
  const void *x, *r, *i, *dout;
  void *out, *dx, *dr, *di;
  mhla_strides sx, sr, si, so, sdo, sdx, sdr, sdi;
  const float* g;  // log_decay [D]
  const int32_t* lengths;
  const float *state_in, *dstate_out;
  float *state_out, *dstate_in;
  float* marks;    // [B][tiles][D]
  float* partial;  // [B][D], the units' sums for log_decay's gradient
  int B, N, D, tiles, slabs;
  int scale;
  int vec;  // both channels of a lane in one access
};

// expm1(x) and exp(x): the Taylor series for |x| < 1/4 (the first term left
// out is x^7 / 5040, 5e-8 of the sum), 2^(x log2 e) elsewhere.
__device__ __forceinline__ void exp_and_less(float x, float* e, float* m) {
  float p = fmaf(x, 1.f / 720.f, 1.f / 120.f);
  p = fmaf(x, p, 1.f / 24.f);
  p = fmaf(x, p, 1.f / 6.f);
  p = fmaf(x, p, 0.5f);
  p = fmaf(x * x, p, x);
  const float y = ex2(x * kLog2e);
  const bool small = fabsf(x) < 0.25f;
  *m = small ? p : y - 1.f;
  *e = small ? 1.f + p : y;
}

// What one token and channel contributes.
struct Gate {
  float a;      // decay
  float c;      // factor of u
  float q;      // sigma(i), 1 without an input gate
  float s;      // sigma(r)
  float less;   // 1 - s
  float turn;   // dc / dlog a
};

template <int KIND, bool IN>
__device__ __forceinline__ Gate gate_of(float r, float i, float g, int scale) {
  Gate o;
  const float e = ex2(-fabsf(r) * kLog2e);  // in (0, 1]: no overflow on either side
  const bool up = r >= 0.f;
  if constexpr (IN) {
    const float f = ex2(-fabsf(i) * kLog2e);
    const float both = rcp((1.f + e) * (1.f + f));  // one reciprocal for two
    const float inv = both * (1.f + f);
    o.s = up ? inv : e * inv;
    o.less = up ? e * inv : inv;
    o.q = both * (1.f + e) * (i >= 0.f ? 1.f : f);
  } else {
    const float inv = rcp(1.f + e);
    o.s = up ? inv : e * inv;
    o.less = up ? e * inv : inv;
    o.q = 1.f;
  }
  float gap;  // 1 - a
  if constexpr (KIND == MHLA_GATED_DECAY) {
    float m;
    exp_and_less(g * o.s, &o.a, &m);
    gap = -m;
  } else {
    o.a = o.s;
    gap = o.less;
  }
  if (scale == MHLA_GATED_SCALE_NORM) {
    const float v = fmaxf(gap * (1.f + o.a), 0.f);
    const float root = rsq(fmaxf(v, 1e-36f));
    o.c = v * root;
    o.turn = v > 0.f ? -o.a * o.a * root : 0.f;
  } else {
    o.c = scale == MHLA_GATED_SCALE_MEAN ? gap : 1.f;
    o.turn = scale == MHLA_GATED_SCALE_MEAN ? -o.a : 0.f;
  }
  return o;
}

__device__ __forceinline__ int length_of(const GatedArgs& p, int b) {
  if (!p.lengths) return p.N;
  const int n = p.lengths[b];
  return n < 0 ? 0 : n > p.N ? p.N : n;
}

// A lane's two channels.
struct Lane {
  int ch, n;  // n: of them inside the row
  bool one, two;
  __device__ Lane(int slab, int D) {
    ch = slab * kSlab + 2 * (threadIdx.x & 31);
    one = ch < D;
    two = ch + 1 < D;
    n = two ? 2 : 1;
  }
  __device__ __forceinline__ float2 get(const float* p, float fill) const {
    return make_float2(p && one ? p[ch] : fill, p && two ? p[ch + 1] : fill);
  }
  __device__ __forceinline__ void put(float* p, float2 v) const {
    if (one) p[ch] = v.x;
    if (two) p[ch + 1] = v.y;
  }
};

template <typename T>
__device__ __forceinline__ float2 both(const Pack<T, 2>& x) {
  return make_float2(x.f(0), x.f(1));
}
template <typename T>
__device__ __forceinline__ void put_two(T* p, float2 x, bool vec, int n) {
  Pack<T, 2> y;
  y.v[0] = from_f32<T>(x.x);
  y.v[1] = from_f32<T>(x.y);
  y.store(p, vec, n);
}

template <typename T, int KIND, bool IN>
__global__ void __launch_bounds__(kThreads) gated_fwd_kernel(const __grid_constant__ GatedArgs p) {
  __shared__ float4 maps[2][kWarps][32];
  const int unit = blockIdx.x, b = unit / p.slabs, w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const Lane ln(unit - b * p.slabs, p.D);
  const int len = length_of(p, b), active = (len + kTile - 1) / kTile;
  const float2 g = KIND == MHLA_GATED_DECAY ? ln.get(p.g, 0.f) : make_float2(0.f, 0.f);
  float2 carry = ln.get(p.state_in ? p.state_in + (int64_t)b * p.D : nullptr, 0.f);
  const T* x = static_cast<const T*>(p.x) + b * p.sx.batch + ln.ch;
  const T* r = static_cast<const T*>(p.r) + b * p.sr.batch + ln.ch;
  const T* i = static_cast<const T*>(p.i) + b * p.si.batch + ln.ch;
  T* out = static_cast<T*>(p.out) + b * p.so.batch + ln.ch;
  const bool vec = p.vec && ln.two;

  Pack<T, 2> rx[kTok], rr[kTok], ri[kTok];
  auto fetch = [&](int tile) {
    const int t0 = tile * kTile + w * kTok;
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      if (!ln.one || t0 + j >= len) continue;
      rx[j].load(x + (t0 + j) * p.sx.token, vec, ln.n);
      rr[j].load(r + (t0 + j) * p.sr.token, vec, ln.n);
      if constexpr (IN) ri[j].load(i + (t0 + j) * p.si.token, vec, ln.n);
    }
  };
  if (active > 0) fetch(0);
  for (int tile = 0; tile < active; ++tile) {
    const int t0 = tile * kTile + w * kTok;
    float2 a[kTok], add[kTok];
    float4 map = make_float4(1.f, 1.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      if (ln.one && t0 + j < len) {
        const float2 xv = both(rx[j]), rv = both(rr[j]), iv = IN ? both(ri[j]) : make_float2(0.f, 0.f);
        const Gate u = gate_of<KIND, IN>(rv.x, iv.x, g.x, p.scale), v = gate_of<KIND, IN>(rv.y, iv.y, g.y, p.scale);
        a[j] = make_float2(u.a, v.a);
        add[j] = make_float2(u.c * (xv.x * u.q), v.c * (xv.y * v.q));
      } else {  // keeps the state
        a[j] = make_float2(1.f, 1.f);
        add[j] = make_float2(0.f, 0.f);
      }
      map.x *= a[j].x;
      map.y *= a[j].y;
      map.z = fmaf(a[j].x, map.z, add[j].x);
      map.w = fmaf(a[j].y, map.w, add[j].y);
    }
    if (tile + 1 < active) fetch(tile + 1);
    maps[tile & 1][w][l] = map;
    __syncthreads();
    float2 h = carry;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) {
      if (v == w) h = carry;
      const float4 m = maps[tile & 1][v][l];
      carry.x = fmaf(m.x, carry.x, m.z);
      carry.y = fmaf(m.y, carry.y, m.w);
    }
    if (p.marks && w == 0) ln.put(p.marks + ((int64_t)b * p.tiles + tile) * p.D, h);
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      h.x = fmaf(a[j].x, h.x, add[j].x);
      h.y = fmaf(a[j].y, h.y, add[j].y);
      if (p.out && ln.one && t0 + j < p.N)
        put_two<T>(out + (t0 + j) * p.so.token, t0 + j < len ? h : make_float2(0.f, 0.f), vec, ln.n);
    }
  }
  if (p.state_out && w == 0) ln.put(p.state_out + (int64_t)b * p.D, carry);
  for (int tile = active; tile < p.tiles; ++tile) {  // padding
    if (p.marks && w == 0) ln.put(p.marks + ((int64_t)b * p.tiles + tile) * p.D, carry);
    if (!p.out || !ln.one) continue;
    for (int t = tile * kTile + w * kTok, j = 0; j < kTok && t < p.N; ++j, ++t)
      put_two<T>(out + t * p.so.token, make_float2(0.f, 0.f), vec, ln.n);
  }
}

template <typename T, int KIND, bool IN>
__global__ void __launch_bounds__(kThreads) gated_bwd_kernel(const __grid_constant__ GatedArgs p) {
  __shared__ float4 maps[2][kWarps][32];
  __shared__ float2 back[2][kWarps][32];
  const int unit = blockIdx.x, b = unit / p.slabs, w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const Lane ln(unit - b * p.slabs, p.D);
  const int len = length_of(p, b), active = (len + kTile - 1) / kTile;
  const float2 g = KIND == MHLA_GATED_DECAY ? ln.get(p.g, 0.f) : make_float2(0.f, 0.f);
  // the gradient that reaches a token's state from behind it
  float2 carry = ln.get(p.dstate_out ? p.dstate_out + (int64_t)b * p.D : nullptr, 0.f);
  const T* x = static_cast<const T*>(p.x) + b * p.sx.batch + ln.ch;
  const T* r = static_cast<const T*>(p.r) + b * p.sr.batch + ln.ch;
  const T* i = static_cast<const T*>(p.i) + b * p.si.batch + ln.ch;
  const T* dout = static_cast<const T*>(p.dout) + b * p.sdo.batch + ln.ch;
  T* dx = static_cast<T*>(p.dx) + b * p.sdx.batch + ln.ch;
  T* dr = static_cast<T*>(p.dr) + b * p.sdr.batch + ln.ch;
  T* di = static_cast<T*>(p.di) + b * p.sdi.batch + ln.ch;
  const bool vec = p.vec && ln.two;
  const float2 zero = make_float2(0.f, 0.f);
  float2 dg = zero;

  for (int tile = p.tiles - 1; tile >= active; --tile) {  // padding
    if (!ln.one) break;
    for (int t = tile * kTile + w * kTok, j = 0; j < kTok && t < p.N; ++j, ++t) {
      put_two<T>(dx + t * p.sdx.token, zero, vec, ln.n);
      put_two<T>(dr + t * p.sdr.token, zero, vec, ln.n);
      if constexpr (IN) put_two<T>(di + t * p.sdi.token, zero, vec, ln.n);
    }
  }
  for (int tile = active - 1; tile >= 0; --tile) {
    const int t0 = tile * kTile + w * kTok;
    Gate gt[kTok][2];
    Pack<T, 2> rx[kTok], rd[kTok];
    float4 map = make_float4(1.f, 1.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      if (ln.one && t0 + j < len) {
        Pack<T, 2> rr, ri;
        rx[j].load(x + (t0 + j) * p.sx.token, vec, ln.n);
        rd[j].load(dout + (t0 + j) * p.sdo.token, vec, ln.n);
        rr.load(r + (t0 + j) * p.sr.token, vec, ln.n);
        if constexpr (IN) ri.load(i + (t0 + j) * p.si.token, vec, ln.n);
        const float2 xv = both(rx[j]), rv = both(rr), iv = IN ? both(ri) : zero;
        gt[j][0] = gate_of<KIND, IN>(rv.x, iv.x, g.x, p.scale);
        gt[j][1] = gate_of<KIND, IN>(rv.y, iv.y, g.y, p.scale);
        const Gate &u = gt[j][0], &v = gt[j][1];
        map.x *= u.a;
        map.y *= v.a;
        map.z = fmaf(u.a, map.z, u.c * (xv.x * u.q));
        map.w = fmaf(v.a, map.w, v.c * (xv.y * v.q));
      }
    }
    float2 rest = zero;  // what the 8 tokens themselves send to the token before them
#pragma unroll
    for (int j = kTok - 1; j >= 0; --j)
      if (ln.one && t0 + j < len) {
        const float2 d = both(rd[j]);
        rest.x = gt[j][0].a * (rest.x + d.x);
        rest.y = gt[j][1].a * (rest.y + d.y);
      }
    maps[tile & 1][w][l] = map;
    back[tile & 1][w][l] = rest;
    __syncthreads();
    float2 h = ln.get(p.marks + ((int64_t)b * p.tiles + tile) * p.D, 0.f), e = carry;
#pragma unroll
    for (int v = 0; v < kWarps - 1; ++v)
      if (v < w) {
        const float4 m = maps[tile & 1][v][l];
        h.x = fmaf(m.x, h.x, m.z);
        h.y = fmaf(m.y, h.y, m.w);
      }
#pragma unroll
    for (int v = kWarps - 1; v >= 0; --v) {
      if (v == w) e = carry;
      const float4 m = maps[tile & 1][v][l];
      const float2 n = back[tile & 1][v][l];
      carry.x = fmaf(m.x, carry.x, n.x);
      carry.y = fmaf(m.y, carry.y, n.y);
    }
    float2 before[kTok];
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      before[j] = h;
      if (ln.one && t0 + j < len) {
        const float2 xv = both(rx[j]);
        h.x = fmaf(gt[j][0].a, h.x, gt[j][0].c * (xv.x * gt[j][0].q));
        h.y = fmaf(gt[j][1].a, h.y, gt[j][1].c * (xv.y * gt[j][1].q));
      }
    }
#pragma unroll
    for (int j = kTok - 1; j >= 0; --j) {
      if (!ln.one || t0 + j >= p.N) continue;
      const bool live = t0 + j < len;
      float2 ox = zero, orr = zero, oi = zero;
      if (live) {
        const float2 xv = both(rx[j]), d = both(rd[j]);
        auto token = [&](const Gate& u, float xx, float G, float hb, float gg, float* o_x, float* o_r, float* o_i) {
          const float dlog = G * fmaf(u.a, hb, xx * u.q * u.turn);
          *o_r = KIND == MHLA_GATED_DECAY ? dlog * (gg * u.s * u.less) : dlog * u.less;
          const float du = G * u.c;
          *o_x = du * u.q;
          *o_i = du * xx * u.q * (1.f - u.q);
          return dlog * u.s;
        };
        e.x += d.x;
        e.y += d.y;
        dg.x += token(gt[j][0], xv.x, e.x, before[j].x, g.x, &ox.x, &orr.x, &oi.x);
        dg.y += token(gt[j][1], xv.y, e.y, before[j].y, g.y, &ox.y, &orr.y, &oi.y);
        e.x *= gt[j][0].a;
        e.y *= gt[j][1].a;
      }
      put_two<T>(dx + (t0 + j) * p.sdx.token, ox, vec, ln.n);
      put_two<T>(dr + (t0 + j) * p.sdr.token, orr, vec, ln.n);
      if constexpr (IN) put_two<T>(di + (t0 + j) * p.sdi.token, oi, vec, ln.n);
    }
  }
  if (p.dstate_in && w == 0) ln.put(p.dstate_in + (int64_t)b * p.D, carry);
  if (KIND == MHLA_GATED_DECAY && p.partial) {
    __syncthreads();
    back[0][w][l] = dg;
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int v = 1; v < kWarps; ++v) {
        dg.x += back[0][v][l].x;
        dg.y += back[0][v][l].y;
      }
      ln.put(p.partial + (int64_t)b * p.D, dg);
    }
  }
}

// Adds the units' rows in order.
__global__ void __launch_bounds__(128) gated_reduce_kernel(const float* partial, int rows, int D, float* out) {
  const int c = blockIdx.x * 128 + threadIdx.x;
  if (c >= D) return;
  float s = 0.f;
  for (int i = 0; i < rows; ++i) s += partial[(int64_t)i * D + c];
  out[c] = s;
}

// One token of every sequence.
template <typename T, int KIND, bool IN>
__global__ void __launch_bounds__(128) gated_step_kernel(const __grid_constant__ GatedArgs p) {
  const int64_t at = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (at >= (int64_t)p.B * p.D) return;
  const int64_t b = at / p.D;
  const int ch = (int)(at - b * p.D);
  const float x = to_f32(static_cast<const T*>(p.x)[b * p.sx.batch + ch]);
  const float r = to_f32(static_cast<const T*>(p.r)[b * p.sr.batch + ch]);
  const float i = IN ? to_f32(static_cast<const T*>(p.i)[b * p.si.batch + ch]) : 0.f;
  const Gate u = gate_of<KIND, IN>(r, i, KIND == MHLA_GATED_DECAY ? p.g[ch] : 0.f, p.scale);
  const float h = fmaf(u.a, p.state_in ? p.state_in[at] : 0.f, u.c * (x * u.q));
  static_cast<T*>(p.out)[b * p.so.batch + ch] = from_f32<T>(h);
  if (p.state_out) p.state_out[at] = h;
}

// ---------------------------------------------------------------- dispatch

enum { kForward, kBackward, kStep };

template <typename T, int KIND, bool IN>
mhla_status launch(const GatedArgs& a, int what, cudaStream_t s) {
  const int64_t blocks = what == kStep ? ((int64_t)a.B * a.D + 127) / 128 : (int64_t)a.B * a.slabs;
  if (blocks > 0x7fffffff) return MHLA_ERR_UNSUPPORTED;
  if (what == kStep)
    gated_step_kernel<T, KIND, IN><<<(unsigned)blocks, 128, 0, s>>>(a);
  else if (what == kForward)
    gated_fwd_kernel<T, KIND, IN><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  else
    gated_bwd_kernel<T, KIND, IN><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  return launch_status();
}

template <typename T>
mhla_status with_kind(const GatedArgs& a, int kind, int what, cudaStream_t s) {
  if (kind == MHLA_GATED_DECAY)
    return a.i ? launch<T, MHLA_GATED_DECAY, true>(a, what, s) : launch<T, MHLA_GATED_DECAY, false>(a, what, s);
  return a.i ? launch<T, MHLA_GATED_SIGMOID, true>(a, what, s) : launch<T, MHLA_GATED_SIGMOID, false>(a, what, s);
}

mhla_status dispatch(const GatedArgs& a, const mhla_gated_params* p, int what, cudaStream_t s) {
  return p->dtype == MHLA_DTYPE_BF16 ? with_kind<__nv_bfloat16>(a, p->kind, what, s)
                                     : with_kind<float>(a, p->kind, what, s);
}

mhla_status check_params(const mhla_gated_params* p, const float* log_decay) {
  if (!p || p->batch < 0 || p->tokens < 0 || p->width < 0 || !ops_dtype_ok(p->dtype)) return MHLA_ERR_INVALID_ARG;
  if (p->kind != MHLA_GATED_DECAY && p->kind != MHLA_GATED_SIGMOID) return MHLA_ERR_INVALID_ARG;
  if (p->scale < MHLA_GATED_SCALE_NORM || p->scale > MHLA_GATED_SCALE_NONE) return MHLA_ERR_INVALID_ARG;
  if (p->marks != 0 && p->marks != 1) return MHLA_ERR_INVALID_ARG;
  if (p->tokens > 0x7fffff00) return MHLA_ERR_UNSUPPORTED;  // tokens are rounded up to tiles in 32 bits
  if ((p->kind == MHLA_GATED_DECAY) != (log_decay != nullptr) && p->width > 0) return MHLA_ERR_INVALID_ARG;
  return MHLA_OK;
}

int64_t tiles_of(const mhla_gated_params* p) { return ((int64_t)p->tokens + kTile - 1) / kTile; }

RowTensor rows(const void* ptr, const mhla_gated_params* p, const mhla_strides& s) {
  return row_tensor(ptr, p->batch, 1, p->tokens, s, p->width, ops_elem(p->dtype));
}
// a state or the marks: float32, contiguous
RowTensor floats(const void* ptr, int64_t n) { return flat_tensor(ptr, ptr ? n : 0, 4); }

// Inputs may share memory, results nothing with one another or with an input;
// `same` may be each other (a state updated in place).
bool apart(const RowTensor* in, int n_in, const RowTensor* out, int n_out, const RowTensor* same_in,
           const RowTensor* same_out) {
  for (int i = 0; i < n_in; ++i)
    if (!row_tensor_ok(in[i], false)) return false;
  for (int o = 0; o < n_out; ++o) {
    if (!row_tensor_ok(out[o], true)) return false;
    for (int i = 0; i < n_in; ++i) {
      if (&in[i] == same_in && &out[o] == same_out && row_tensors_same(in[i], out[o])) continue;
      if (!row_tensors_apart(in[i], out[o])) return false;
    }
    for (int q = o + 1; q < n_out; ++q)
      if (!row_tensors_apart(out[o], out[q])) return false;
  }
  return true;
}

GatedArgs args_of(const mhla_gated_params* p, const void* x, const void* gate, const void* input_gate,
                  const float* log_decay, const int32_t* lengths) {
  GatedArgs a = {};
  a.x = x;
  a.r = gate;
  a.i = input_gate;
  a.g = log_decay;
  a.lengths = lengths;
  a.sx = p->x;
  a.sr = p->gate;
  a.si = p->input_gate;
  a.B = p->batch;
  a.N = p->tokens;
  a.D = p->width;
  a.tiles = (int)tiles_of(p);
  a.slabs = (p->width + kSlab - 1) / kSlab;
  a.scale = p->scale;
  return a;
}

// Whether the two channels of a lane can be one access in all of these.
int pairs_aligned(const RowTensor* t, int n) {
  for (int i = 0; i < n; ++i)
    if (!t[i].empty() && row_alignment(t[i], 2 * (int)t[i].elem) < 2 * (int)t[i].elem) return 0;
  return 1;
}

}  // namespace
}  // namespace mhla

extern "C" {

mhla_status mhla_gated_forward(const void* x, const void* gate, const void* input_gate, const float* log_decay,
                               const int32_t* lengths, const float* state_in, const mhla_gated_params* p, void* out,
                               float* state_out, float* marks, void* stream) {
  using namespace mhla;
  mhla_status st = check_params(p, log_decay);
  if (st != MHLA_OK) return st;
  const int64_t state = (int64_t)p->batch * p->width;
  const RowTensor in[6] = {rows(x, p, p->x), rows(gate, p, p->gate),
                           input_gate ? rows(input_gate, p, p->input_gate) : floats(nullptr, 0),
                           floats(log_decay, p->width), floats(lengths, p->batch), floats(state_in, state)};
  const RowTensor res[3] = {rows(out, p, p->out), floats(state_out, state),
                            floats(marks, tiles_of(p) * state)};
  if (!apart(in, 6, res, 3, &in[5], &res[1])) return MHLA_ERR_INVALID_ARG;
  if (state == 0) return MHLA_OK;
  GatedArgs a = args_of(p, x, gate, input_gate, log_decay, lengths);
  a.state_in = state_in;
  a.out = out;
  a.so = p->out;
  a.state_out = state_out;
  a.marks = marks;
  a.vec = pairs_aligned(in, 3) && pairs_aligned(res, 1);
  return dispatch(a, p, kForward, static_cast<cudaStream_t>(stream));
}

mhla_status mhla_gated_backward_workspace_bytes(const mhla_gated_params* p, size_t* bytes) {
  using namespace mhla;
  static const float some = 0.f;
  if (!bytes || !p) return MHLA_ERR_INVALID_ARG;
  const mhla_status st = check_params(p, p->kind == MHLA_GATED_DECAY ? &some : nullptr);
  if (st != MHLA_OK) return st;
  const size_t state = sizeof(float) * (size_t)p->batch * (size_t)p->width;
  *bytes = (p->kind == MHLA_GATED_DECAY ? state : 0) + (p->marks ? 0 : state * (size_t)tiles_of(p));
  return MHLA_OK;
}

mhla_status mhla_gated_backward(const void* x, const void* gate, const void* input_gate, const float* log_decay,
                                const int32_t* lengths, const float* state_in, const float* marks, const void* dout,
                                const float* dstate_out, const mhla_gated_params* p, void* dx, void* dgate,
                                void* dinput_gate, float* dlog_decay, float* dstate_in, void* workspace,
                                size_t workspace_bytes, void* stream) {
  using namespace mhla;
  mhla_status st = check_params(p, log_decay);
  if (st != MHLA_OK) return st;
  if ((marks != nullptr) != (p->marks != 0) && p->batch && p->tokens && p->width) return MHLA_ERR_INVALID_ARG;
  if ((input_gate == nullptr) != (dinput_gate == nullptr) && p->batch && p->tokens && p->width)
    return MHLA_ERR_INVALID_ARG;
  if (dlog_decay && p->kind != MHLA_GATED_DECAY) return MHLA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t state = (int64_t)p->batch * p->width;
  size_t need = 0;
  if ((st = mhla_gated_backward_workspace_bytes(p, &need)) != MHLA_OK) return st;
  const RowTensor none = floats(nullptr, 0);
  const RowTensor in[9] = {rows(x, p, p->x), rows(gate, p, p->gate),
                           input_gate ? rows(input_gate, p, p->input_gate) : none, rows(dout, p, p->dout),
                           floats(log_decay, p->width), floats(lengths, p->batch), floats(state_in, state),
                           floats(marks, tiles_of(p) * state), floats(dstate_out, state)};
  const RowTensor res[6] = {rows(dx, p, p->dx), rows(dgate, p, p->dgate),
                            dinput_gate ? rows(dinput_gate, p, p->dinput_gate) : none,
                            floats(dlog_decay, p->width), floats(dstate_in, state),
                            flat_tensor(workspace, workspace ? (int64_t)need : 0, 1)};
  if (!apart(in, 9, res, 6, &in[8], &res[4])) return MHLA_ERR_INVALID_ARG;
  if (state == 0) {
    if (dlog_decay && p->width) {  // an empty sum
      const cudaError_t e = cudaMemsetAsync(dlog_decay, 0, sizeof(float) * (size_t)p->width, s);
      if (e != cudaSuccess) return record_cuda_error(e);
    }
    return MHLA_OK;
  }
  Scratch scratch;
  if ((st = scratch.take(workspace, workspace_bytes, need, s)) != MHLA_OK) return st;
  GatedArgs a = args_of(p, x, gate, input_gate, log_decay, lengths);
  float* at = reinterpret_cast<float*>(scratch.ptr());
  if (p->kind == MHLA_GATED_DECAY) {
    if (dlog_decay) a.partial = at;
    at += state;
  }
  a.state_in = state_in;
  a.vec = pairs_aligned(in, 4) && pairs_aligned(res, 3);
  a.marks = const_cast<float*>(marks);
  if (!marks && a.tiles > 0) {
    a.marks = at;
    st = dispatch(a, p, kForward, s);  // the states alone
  }
  a.dout = dout;
  a.sdo = p->dout;
  a.dstate_out = dstate_out;
  a.dx = dx;
  a.dr = dgate;
  a.di = dinput_gate;
  a.sdx = p->dx;
  a.sdr = p->dgate;
  a.sdi = p->dinput_gate;
  a.dstate_in = dstate_in;
  if (st == MHLA_OK) st = dispatch(a, p, kBackward, s);
  if (st == MHLA_OK && dlog_decay) {
    gated_reduce_kernel<<<(unsigned)((p->width + 127) / 128), 128, 0, s>>>(a.partial, p->batch, p->width, dlog_decay);
    st = launch_status();
  }
  return scratch.give_back(st);
}

mhla_status mhla_gated_step(const void* x, const void* gate, const void* input_gate, const float* log_decay,
                            const float* state_in, const mhla_gated_params* p, void* out, float* state_out,
                            void* stream) {
  using namespace mhla;
  mhla_status st = check_params(p, log_decay);
  if (st != MHLA_OK) return st;
  if (p->tokens != 1) return MHLA_ERR_INVALID_ARG;
  const int64_t state = (int64_t)p->batch * p->width;
  const RowTensor in[5] = {rows(x, p, p->x), rows(gate, p, p->gate),
                           input_gate ? rows(input_gate, p, p->input_gate) : floats(nullptr, 0),
                           floats(log_decay, p->width), floats(state_in, state)};
  const RowTensor res[2] = {rows(out, p, p->out), floats(state_out, state)};
  if (!apart(in, 5, res, 2, &in[4], &res[1])) return MHLA_ERR_INVALID_ARG;
  if (state == 0) return MHLA_OK;
  GatedArgs a = args_of(p, x, gate, input_gate, log_decay, nullptr);
  a.state_in = state_in;
  a.out = out;
  a.so = p->out;
  a.state_out = state_out;
  return dispatch(a, p, kStep, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
