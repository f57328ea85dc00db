// Norm of queries and keys over each head and their rotation, in one pass:
//   y = R(position) (x rstd w),  rstd = 1 / sqrt(mean(x^2) + eps),
// and the gradients: with t = R^T dy and g = w t,
//   dx = rstd (g - xh mean(g xh)),  dw = sum t xh,  xh = x rstd.
//
// A row is held by a group of G threads, so that both entries of a rotated
// pair are one thread's, and is read once; its sums meet through shuffles.  A
// group forms the sines of its token once and walks over the heads.  Phases
// are the 64-bit fractions of a turn of mhla_rotary_table.
// Bound: memory (each row read once and written once; the backward pass reads
// two rows and writes one), with the latency of a row's sums where heads are
// wide: 16 + 4 heads of 64 over 4 x 32k tokens (bf16) take 116 us forward, 5.8 TB/s,
// and 173 us backward; of 128 over 2 x 8k tokens 32 us (25 at the rate of a copy)
// and 49 us (37), of which 3 us add the weights' gradients.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "ops.h"
#include "pack.cuh"
#include "qknorm_heads.h"
#include "tc_host.h"

namespace mhla {
namespace {

constexpr int kMaxDim = 256;

struct QkArgs {
  const void* x[2];
  const void* dy[2];  // backward
  void* y[2];         // results; dq and dk in the backward pass
  mhla_strides sx[2], sdy[2], sy[2];
  const void* w[2];
  int w_f32;
  const void* positions;
  int64_t pos_offset, pos_sb, pos_st;
  int pos64;
  int heads[2];
  int batch, tokens, dim;
  int half;      // rotated pairs
  int adjacent;  // pairs (2i, 2i + 1) taken apart into two single entries
  int slots;     // of a row, two vectors each
  int group, lanes_shift;  // threads of a row, a power of two, and its logarithm
  int heads_per_thread;
  int ctas[2];     // backward: CTAs that take q's and k's rows
  float eps, inv_dim, amp;
  float* partial;  // backward: [CTAs][dim]
  mhla_rotary_table table;
};

// Columns of a slot's two vectors.  ACROSS pairs entry i of the first with
// entry i of the second; otherwise neighbours inside a vector are paired.  Only
// single entries of adjacent pairs are next to one another: neighbouring threads
// read neighbouring vectors.
template <int VEC, bool ACROSS>
__device__ __forceinline__ void columns(const QkArgs& a, int slot, int* lo, int* hi) {
  if (ACROSS && a.adjacent) {
    *lo = 2 * slot;
    *hi = 2 * slot + 1;
    return;
  }
  const int rot = ACROSS ? a.half / VEC : 0;  // slots that are rotated across
  if (slot < rot) {
    *lo = slot * VEC;
    *hi = a.half + slot * VEC;
  } else {
    *lo = 2 * rot * VEC + (slot - rot) * VEC;
    *hi = *lo + (a.slots - rot) * VEC;
  }
}

// A slot's 2 VEC values, as pairs of neighbours where there are any.
template <int VEC, bool ACROSS>
struct Values {
  static constexpr bool kPairs = ACROSS && VEC > 1;
  float2 p[kPairs ? VEC : 1];    // the first vector's pairs, then the second's
  float f[kPairs ? 1 : 2 * VEC];

  template <typename T>
  __device__ __forceinline__ void read(const Pack<T, VEC> (&x)[2]) {
    if constexpr (kPairs) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = pair_of(x[i >= VEC / 2], i % (VEC / 2));
    } else {
#pragma unroll
      for (int i = 0; i < 2 * VEC; ++i) f[i] = x[i / VEC].f(i % VEC);
    }
  }
  template <typename T>
  __device__ __forceinline__ void write(Pack<T, VEC> (&x)[2]) const {
    if constexpr (kPairs) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) put_pair(&x[i >= VEC / 2], i % (VEC / 2), p[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 2 * VEC; ++i) x[i / VEC].v[i % VEC] = from_f32<T>(f[i]);
    }
  }
  // entries of the first, then of the second vector
  __device__ __forceinline__ void set(const float (&v)[2 * VEC]) {
    if constexpr (kPairs) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = make_float2(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 2 * VEC; ++i) f[i] = v[i];
    }
  }
  __device__ __forceinline__ void get(float (&v)[2 * VEC]) const {
#pragma unroll
    for (int i = 0; i < 2 * VEC; ++i) {
      if constexpr (kPairs)
        v[i] = i % 2 ? p[i / 2].y : p[i / 2].x;
      else
        v[i] = f[i];
    }
  }
  __device__ __forceinline__ void fill(float v) {
    if constexpr (kPairs) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = splat(v);
    } else {
#pragma unroll
      for (int i = 0; i < 2 * VEC; ++i) f[i] = v;
    }
  }
  // this = x y, x y + this, this s
  __device__ __forceinline__ void product(const Values& x, const Values& y) {
    if constexpr (kPairs) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = mul2(x.p[i], y.p[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 2 * VEC; ++i) f[i] = x.f[i] * y.f[i];
    }
  }
  __device__ __forceinline__ void add_product(const Values& x, const Values& y) {
    if constexpr (kPairs) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = fma2(x.p[i], y.p[i], p[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 2 * VEC; ++i) f[i] = fmaf(x.f[i], y.f[i], f[i]);
    }
  }
  __device__ __forceinline__ void scale(float s) {
    if constexpr (kPairs) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = mul2(p[i], splat(s));
    } else {
#pragma unroll
      for (int i = 0; i < 2 * VEC; ++i) f[i] *= s;
    }
  }
  // this = a this + b x
  __device__ __forceinline__ void combine(float a, float b, const Values& x) {
    if constexpr (kPairs) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = fma2(x.p[i], splat(b), mul2(p[i], splat(a)));
    } else {
#pragma unroll
      for (int i = 0; i < 2 * VEC; ++i) f[i] = fmaf(x.f[i], b, f[i] * a);
    }
  }
  __device__ __forceinline__ float dot(const Values& x) const {
    if constexpr (kPairs) {
      float2 s = mul2(p[0], x.p[0]);
#pragma unroll
      for (int i = 1; i < VEC; ++i) s = fma2(p[i], x.p[i], s);
      return s.x + s.y;
    } else {
      float s = f[0] * x.f[0];
#pragma unroll
      for (int i = 1; i < 2 * VEC; ++i) s = fmaf(f[i], x.f[i], s);
      return s;
    }
  }
  // Rotates the pairs: (a, b) -> (c_a a + s_b b, s_a a + c_b b), `c` and `s` laid
  // out as the values that they multiply.
  __device__ __forceinline__ void turn(const Values& c, const Values& s) {
    if constexpr (kPairs) {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const float2 a = p[i], b = p[i + VEC / 2];
        p[i] = fma2(a, c.p[i], mul2(b, s.p[i + VEC / 2]));
        p[i + VEC / 2] = fma2(b, c.p[i + VEC / 2], mul2(a, s.p[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int j = ACROSS ? i : 2 * i, k = ACROSS ? i + VEC : 2 * i + 1;
        const float a = f[j], b = f[k];
        f[j] = fmaf(a, c.f[j], b * s.f[k]);
        f[k] = fmaf(b, c.f[k], a * s.f[j]);
      }
    }
  }
};

// What a slot's values are multiplied with by Values::turn: cosines (in `c`) and
// sines (in `s`, the second one's with the sign turned, so that turn adds them)
// times the values' weights; 1 and 0 where nothing is rotated, which are those of
// no turn.  Two angles at a time, without a branch (16 + 4 heads of 128, bf16, over 2
// x 8k tokens 32 us, with one 36).
template <int VEC, bool ACROSS>
__device__ __forceinline__ void turns_of(const QkArgs& a, const uint64_t* turns, int64_t pos, const int (&col)[2],
                                         float sign, Values<VEC, ACROSS>* c, Values<VEC, ACROSS>* s) {
  float fc[2 * VEC], fs[2 * VEC];
#pragma unroll
  for (int first = 0; first < VEC; first += 2) {
    float cs[2], sn[2];
    bool rotated[2] = {false, false};
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int i = first + n, j = ACROSS ? i : 2 * i;            // the pair's first entry
      const int entry = j < VEC ? col[0] + j : col[1] + j - VEC;  // its column
      const int pair = ACROSS && !a.adjacent ? entry : entry / 2;
      rotated[n] = i < VEC && pair < a.half && (!ACROSS || a.adjacent || col[0] < a.half);
      const uint64_t phase = rotated[n] ? (uint64_t)pos * turns[pair] : 0;
      sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &sn[n], &cs[n]);  // half turns in [-1, 1)
    }
    const float2 cosines = mulc(make_float2(cs[0], cs[1]), a.amp);
    const float2 sines = mulc(make_float2(sn[0], sn[1]), a.amp * sign);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int i = first + n, j = ACROSS ? i : 2 * i, k = ACROSS ? i + VEC : 2 * i + 1;
      if (i >= VEC) break;
      fc[j] = fc[k] = !rotated[n] ? 1.f : n ? cosines.y : cosines.x;
      fs[j] = n ? sines.y : sines.x;
      fs[k] = -fs[j];
    }
  }
  c->set(fc);
  s->set(fs);
}

__device__ __forceinline__ int64_t position_of(const QkArgs& a, int64_t b, int t) {
  if (!a.positions) return a.pos_offset + t;
  const int64_t at = b * a.pos_sb + t * a.pos_st;
  return a.pos64 ? static_cast<const int64_t*>(a.positions)[at] : static_cast<const int32_t*>(a.positions)[at];
}

template <int VEC, bool ACROSS>
__device__ __forceinline__ void weights_of(const QkArgs& a, int which, const int (&col)[2], const bool (&in)[2],
                                           Values<VEC, ACROSS>* w) {
  float f[2 * VEC];
#pragma unroll
  for (int i = 0; i < 2 * VEC; ++i)
    f[i] = a.w[which] && in[i / VEC] ? param_at(a.w[which], a.w_f32, col[i / VEC] + i % VEC) : 1.f;
  w->set(f);
}

// CTAs that an SM holds.
constexpr int kResident = 2;

// A thread's vectors of the next rows: asynchronous copies into places of its own
// in shared memory, STEPS - 1 steps of ROWS rows ahead; elements of 2 bytes, which
// cannot be copied so, are read a row ahead into registers.
template <typename T, int VEC, int E, int ROWS, int STEPS>
struct Ring {
  static constexpr int kBytes = VEC * (int)sizeof(T);
  static constexpr bool kAsync = kBytes >= 4;
  static constexpr size_t kSmem = kAsync ? (size_t)STEPS * ROWS * E * 2 * kBytes * 256 : 0;
  static_assert(kSmem <= 100 * 1024, "two CTAs on an SM");
  unsigned char* base;

  __device__ __forceinline__ explicit Ring(unsigned char* smem) : base(smem) {}
  __device__ __forceinline__ unsigned char* place(int step, int row, int i) const {
    return base + ((((step * ROWS + row) * 2 * E) + i) * 256 + threadIdx.x) * kBytes;
  }
  // Starts vector i of a row; zeros where it does not exist.
  __device__ __forceinline__ void start(int step, int row, int i, const T* from, bool exists, const T* any) {
    if constexpr (kAsync)
      copy_async<kBytes>(place(step, row, i), exists ? from : any, exists ? kBytes : 0);
  }
  __device__ __forceinline__ void take(int step, int row, int i, Pack<T, VEC>* to) const {
    if constexpr (kBytes == 16)
      *reinterpret_cast<uint4*>(to->v) = *reinterpret_cast<const uint4*>(place(step, row, i));
    else if constexpr (kBytes == 8)
      *reinterpret_cast<uint2*>(to->v) = *reinterpret_cast<const uint2*>(place(step, row, i));
    else
      *reinterpret_cast<uint32_t*>(to->v) = *reinterpret_cast<const uint32_t*>(place(step, row, i));
  }
};

constexpr int kFwdRows = 4, kFwdSteps = 2, kBwdSteps = 3;
template <typename T, int VEC, int E>
using FwdRing = Ring<T, VEC, E, kFwdRows, kFwdSteps>;

template <typename T, int VEC, bool ACROSS, int E>
__global__ void __launch_bounds__(256, kResident) qknorm_fwd_kernel(const __grid_constant__ QkArgs a) {
  constexpr int R = kFwdRows, kSteps = kFwdSteps;
  using V = Values<VEC, ACROSS>;
  using Rows = FwdRing<T, VEC, E>;
  extern __shared__ __align__(16) unsigned char dynamic[];
  __shared__ uint64_t turns[MHLA_ROTARY_MAX_PAIRS];
  for (int i = threadIdx.x; i < a.half; i += blockDim.x) turns[i] = a.table.turns[i];
  __syncthreads();
  Rows ring(dynamic);
  const int lane = threadIdx.x & (a.group - 1), per = blockDim.x >> a.lanes_shift;
  int col[E][2];
  bool in[E][2];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int slot = lane + e * a.group;
    columns<VEC, ACROSS>(a, slot, &col[e][0], &col[e][1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) in[e][k] = slot < a.slots && col[e][k] < a.dim;
  }
  const int64_t all = (int64_t)a.batch * a.tokens, stride = (int64_t)gridDim.x * per;
  const HeadShare share(blockIdx.y, a.heads_per_thread, a.heads[0], a.heads[0] + a.heads[1]);
  const int first = share.first, split = share.split, last = share.last;

  // a token's rows: those that are computed, and those that are fetched ahead
  struct Place {
    int64_t base, b;
    int t, h;
    bool live;
  };
  auto locate = [&](Place& p, int64_t base) {
    const int64_t token = base + (threadIdx.x >> a.lanes_shift);
    p.base = base;
    p.h = first;
    p.live = token < all;
    p.b = p.live ? token / a.tokens : 0;
    p.t = p.live ? (int)(token - p.b * a.tokens) : 0;
  };
  auto row_of = [&](const Place& p, int h) {
    const int which = h >= a.heads[0];
    return static_cast<const T*>(a.x[which]) + p.b * a.sx[which].batch + p.t * a.sx[which].token +
           (h - (which ? a.heads[0] : 0)) * a.sx[which].head;
  };
  Place ahead, now;
  locate(ahead, (int64_t)blockIdx.x * per);
  int put = 0, got = 0;
  auto fetch = [&] {
    if (Rows::kAsync && ahead.base < all) {
      const int end = share.step_end(ahead.h, R);  // rows behind it do not exist
      const T* any = row_of(ahead, ahead.h);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool exists = ahead.live && ahead.h + r < end;
        const T* from = row_of(ahead, exists ? ahead.h + r : ahead.h);
#pragma unroll
        for (int i = 0; i < 2 * E; ++i)
          ring.start(put, r, i, from + col[i / 2][i % 2], exists && in[i / 2][i % 2], any);
      }
      ahead.h = end;
      if (end >= last) locate(ahead, ahead.base + stride);
    }
    copies_commit();
    put = put + 1 < kSteps ? put + 1 : 0;
  };
  if (Rows::kAsync)
    for (int i = 0; i < kSteps - 1; ++i) fetch();

  locate(now, (int64_t)blockIdx.x * per);
  int64_t pos = position_of(a, now.b, now.t);
  for (int64_t base = (int64_t)blockIdx.x * per; base < all; base += stride) {
    V cs[E], sn[E];
#pragma unroll
    for (int e = 0; e < E; ++e) turns_of<VEC, ACROSS>(a, turns, pos, col[e], 1.f, &cs[e], &sn[e]);
    Place then;
    locate(then, base + stride);
    pos = position_of(a, then.b, then.t);  // a token ahead
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const int end = which ? last : split;
      int h = which ? split : first;
      if (h >= end) continue;  // the same for the whole grid row
      V c[E], s[E];  // with the weights
#pragma unroll
      for (int e = 0; e < E; ++e) {
        V w;
        weights_of(a, which, col[e], in[e], &w);
        c[e].product(cs[e], w);
        s[e].product(sn[e], w);
      }
      const int64_t yh = a.sy[which].head;
      T* dst = static_cast<T*>(a.y[which]) + now.b * a.sy[which].batch + now.t * a.sy[which].token +
               (h - (which ? a.heads[0] : 0)) * yh;
      for (; h < end; h += R, dst += R * yh) {
        Pack<T, VEC> raw[R][E][2];
        if constexpr (Rows::kAsync) {
          fetch();
          copies_wait<kSteps - 1>();
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 2 * E; ++i) ring.take(got, r, i, &raw[r][i / 2][i % 2]);
          got = got + 1 < kSteps ? got + 1 : 0;
        } else {
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 2 * E; ++i) {
              raw[r][i / 2][i % 2].zero();
              if (in[i / 2][i % 2] && now.live && h + r < end)
                raw[r][i / 2][i % 2].load(row_of(now, h + r) + col[i / 2][i % 2], true);
            }
        }
        float sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          sum[r] = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            V v;
            v.read(raw[r][e]);
            sum[r] += v.dot(v);
          }
        }
        for (int o = a.group / 2; o > 0; o >>= 1)
#pragma unroll
          for (int r = 0; r < R; ++r) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], o);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (h + r >= end) break;  // the same for all lanes
          const float rstd = rsqrtf(fmaf(sum[r], a.inv_dim, a.eps));
#pragma unroll
          for (int e = 0; e < E; ++e) {
            V v;
            v.read(raw[r][e]);
            v.scale(rstd);
            v.turn(c[e], s[e]);
            Pack<T, VEC> o[2];
            v.write(o);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (in[e][k] && now.live) o[k].store(dst + r * yh + col[e][k], true);
          }
        }
      }
    }
    now = then;
  }
}

// CTAs take the tokens in turn, those below ctas[0] q's rows and the others
// k's, and keep the sums of dw of their columns in registers.
template <typename T, int VEC, int E>
using BwdRing = Ring<T, VEC, 2 * E, 1, kBwdSteps>;  // x's vectors, then dy's

template <typename T, int VEC, bool ACROSS, int E>
__global__ void __launch_bounds__(256, kResident) qknorm_bwd_kernel(const __grid_constant__ QkArgs a) {
  constexpr int kSteps = kBwdSteps;
  using V = Values<VEC, ACROSS>;
  using Rows = BwdRing<T, VEC, E>;
  extern __shared__ __align__(16) unsigned char dynamic[];
  __shared__ uint64_t turns[MHLA_ROTARY_MAX_PAIRS];
  __shared__ float sums[8][kMaxDim];
  for (int i = threadIdx.x; i < a.half; i += blockDim.x) turns[i] = a.table.turns[i];
  __syncthreads();
  Rows ring(dynamic);
  const int which = (int)blockIdx.x >= a.ctas[0];
  const int cta = blockIdx.x - (which ? a.ctas[0] : 0), heads = a.heads[which];
  const int lane = threadIdx.x & (a.group - 1), per = blockDim.x >> a.lanes_shift;
  int col[E][2];
  bool in[E][2];
  V w[E], dw[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int slot = lane + e * a.group;
    columns<VEC, ACROSS>(a, slot, &col[e][0], &col[e][1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) in[e][k] = slot < a.slots && col[e][k] < a.dim;
    weights_of(a, which, col[e], in[e], &w[e]);
    dw[e].fill(0.f);
  }
  const int64_t all = (int64_t)a.batch * a.tokens, stride = (int64_t)a.ctas[which] * per, start = (int64_t)cta * per;
  const int64_t xh = a.sx[which].head, dyh = a.sdy[which].head, dxh = a.sy[which].head;

  // the token whose rows are fetched ahead
  int64_t ahead = start;
  const T *ax = nullptr, *ady = nullptr;
  bool alive = false;
  int ah = 0, put = 0, got = 0;
  auto point = [&](int64_t base, const T** x, const T** dy) {
    const int64_t token = base + (threadIdx.x >> a.lanes_shift);
    const bool live = token < all;
    const int64_t b = live ? token / a.tokens : 0, t = live ? token - b * a.tokens : 0;
    *x = static_cast<const T*>(a.x[which]) + b * a.sx[which].batch + t * a.sx[which].token;
    *dy = static_cast<const T*>(a.dy[which]) + b * a.sdy[which].batch + t * a.sdy[which].token;
    return live;
  };
  auto fetch = [&] {
    if (Rows::kAsync && ahead < all) {
      if (ah == 0) alive = point(ahead, &ax, &ady);
#pragma unroll
      for (int i = 0; i < 2 * E; ++i) {
        const bool exists = alive && in[i / 2][i % 2];
        ring.start(put, 0, i, ax + col[i / 2][i % 2], exists, ax);
        ring.start(put, 0, 2 * E + i, ady + col[i / 2][i % 2], exists, ady);
      }
      ax += xh;
      ady += dyh;
      if (++ah == heads) {
        ah = 0;
        ahead += stride;
      }
    }
    copies_commit();
    put = put + 1 < kSteps ? put + 1 : 0;
  };
  if (Rows::kAsync)
    for (int i = 0; i < kSteps - 1; ++i) fetch();

  // every thread of the CTA makes the same number of turns
  for (int64_t base = start; base < all; base += stride) {
    const T *x, *dy;
    const bool live = point(base, &x, &dy);
    const int64_t token = live ? base + (threadIdx.x >> a.lanes_shift) : 0;
    const int64_t b = token / a.tokens, t = token - b * a.tokens;
    T* dx = static_cast<T*>(a.y[which]) + b * a.sy[which].batch + t * a.sy[which].token;
    const int64_t pos = position_of(a, b, (int)t);
    V cs[E], sn[E];
#pragma unroll
    for (int e = 0; e < E; ++e) turns_of<VEC, ACROSS>(a, turns, pos, col[e], -1.f, &cs[e], &sn[e]);
    Pack<T, VEC> nx[Rows::kAsync ? 1 : E][2], nd[Rows::kAsync ? 1 : E][2];
    auto read = [&](int h) {
      if constexpr (!Rows::kAsync) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            nx[e][k].zero();
            nd[e][k].zero();
            if (in[e][k] && live && h < heads) {
              nx[e][k].load(x + h * xh + col[e][k], true);
              nd[e][k].load(dy + h * dyh + col[e][k], true);
            }
          }
        }
      }
    };
    read(0);
    for (int h = 0; h < heads; ++h, dx += dxh) {
      Pack<T, VEC> rx[E][2];
      V v[E];
      float sum = 0.f, along = 0.f;
      if constexpr (Rows::kAsync) {
        fetch();
        copies_wait<kSteps - 1>();
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        Pack<T, VEC> rd[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if constexpr (Rows::kAsync) {
            ring.take(got, 0, 2 * e + k, &rx[e][k]);
            ring.take(got, 0, 2 * E + 2 * e + k, &rd[k]);
          } else {
            rx[e][k] = nx[e][k];
            rd[k] = nd[e][k];
          }
        }
        v[e].read(rd);
        v[e].turn(cs[e], sn[e]);  // t
        V xv, g;
        xv.read(rx[e]);
        g.product(v[e], w[e]);
        sum += xv.dot(xv);
        along += g.dot(xv);
      }
      got = got + 1 < kSteps ? got + 1 : 0;
      read(h + 1);
      for (int o = a.group / 2; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        along += __shfl_xor_sync(0xffffffffu, along, o);
      }
      // a row that is not there adds nothing, although its rstd may be infinite
      const float rstd = live ? rsqrtf(fmaf(sum, a.inv_dim, a.eps)) : 0.f;
      const float mean = along * rstd * a.inv_dim;  // of g xh
#pragma unroll
      for (int e = 0; e < E; ++e) {
        V xv;
        xv.read(rx[e]);
        xv.scale(rstd);  // xh
        dw[e].add_product(v[e], xv);
        v[e].product(v[e], w[e]);
        v[e].combine(rstd, -mean * rstd, xv);
        Pack<T, VEC> o[2];
        v[e].write(o);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (in[e][k] && live) o[k].store(dx + col[e][k], true);
      }
    }
  }
  if (!a.partial) return;
  start_successor();
  // groups of a warp hold the same columns; then the warps in order
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float f[2 * VEC];
    dw[e].get(f);
    for (int o = a.group; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 2 * VEC; ++i) f[i] += __shfl_xor_sync(0xffffffffu, f[i], o);
    if ((threadIdx.x & 31) < a.group)
#pragma unroll
      for (int i = 0; i < 2 * VEC; ++i)
        if (in[e][i / VEC]) sums[threadIdx.x >> 5][col[e][i / VEC] + i % VEC] = f[i];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.dim; c += blockDim.x) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < 8; ++v) s += sums[v][c];
    a.partial[(int64_t)blockIdx.x * a.dim + c] = s;
  }
}

// Adds the CTAs' rows: a CTA takes 32 columns of q's or k's, 32 threads a column.
__global__ void __launch_bounds__(1024) qknorm_reduce_kernel(const float* partial, int ctas_q, int ctas_k, int dim,
                                                             float* dq_weight, float* dk_weight) {
  __shared__ float sh[32][33];
  const int which = blockIdx.y, tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
  const int first = which ? ctas_q : 0, last = which ? ctas_q + ctas_k : ctas_q;
  float s = 0.f;
  after_predecessor();
  if (c < dim)
    for (int p = first + ty; p < last; p += 32) s += partial[(int64_t)p * dim + c];
  sh[ty][tx] = s;
  __syncthreads();
  float* out = which ? dk_weight : dq_weight;
  if (ty == 0 && c < dim && out) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += sh[i][tx];
    out[c] = t;
  }
}

// ---------------------------------------------------------------- dispatch

// CTAs of the backward pass: those that are resident at once, shared out by
// the number of heads, none for nothing.
void share_ctas(QkArgs* a) {
  const int64_t per = 256 / a->group, all = (int64_t)a->batch * a->tokens;
  const int64_t most = (all + per - 1) / per;  // one turn each
  const int total = a->heads[0] + a->heads[1];
  for (int i = 0; i < 2; ++i) {
    // a token's sines and positions count about two rows
    const int64_t weight[2] = {a->heads[0] ? a->heads[0] + 2 : 0, a->heads[1] ? a->heads[1] + 2 : 0};
    int64_t n = total ? (int64_t)kResident * kOpsSms * weight[i] / (weight[0] + weight[1]) : 0;
    if (n < 1) n = 1;
    if (n > most) n = most;
    a->ctas[i] = a->heads[i] && all ? (int)n : 0;
  }
}

template <typename T, int VEC, bool ACROSS, int E>
mhla_status launch(QkArgs& a, bool backward, cudaStream_t s) {
  if (backward) {
    auto kernel = qknorm_bwd_kernel<T, VEC, ACROSS, E>;
    constexpr size_t smem = BwdRing<T, VEC, E>::kSmem;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return record_cuda_error(e);
    kernel<<<a.ctas[0] + a.ctas[1], 256, smem, s>>>(a);
    return launch_status();
  }
  // Heads are shared out over threads only where there are too few tokens to
  // fill the GPU, as each share forms the sines again.
  auto kernel = qknorm_fwd_kernel<T, VEC, ACROSS, E>;
  constexpr size_t smem = FwdRing<T, VEC, E>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return record_cuda_error(e);
  const int64_t slots = (int64_t)kOpsSms * kResident, per = 256 / a.group;
  int64_t blocks = ((int64_t)a.batch * a.tokens + per - 1) / per;
  const int total = a.heads[0] + a.heads[1];
  int64_t parts = slots / blocks;
  parts = parts < 1 ? 1 : parts > total ? total : parts;
  a.heads_per_thread = (int)((total + parts - 1) / parts);
  parts = (total + a.heads_per_thread - 1) / a.heads_per_thread;
  if (blocks > slots) blocks = slots;
  kernel<<<dim3((unsigned)blocks, (unsigned)parts), 256, smem, s>>>(a);
  return launch_status();
}

// Elements of the widest vector that divides the row, every row start and, for
// HALF, each half of the rotated part (INTERLEAVED, the rotated part may end inside
// a vector: 4 x 8k tokens x 16 + 4 heads of 64, 50 rotated, 31 us; in vectors of 2, 51).
int vector_of(int dim, int pairs, int style, int elem, int align) {
  for (int v = 16 / elem; v > 1; v /= 2)
    if ((style != MHLA_ROTARY_HALF || pairs % v == 0) && dim % v == 0 && align >= v * elem) return v;
  return 1;
}

// Slots and the threads of a row for vectors of `vec` elements.
void shape_rows(QkArgs* a, int vec, int style) {
  a->adjacent = vec == 1 && style == MHLA_ROTARY_INTERLEAVED;
  a->slots = style == MHLA_ROTARY_HALF ? a->half / vec + (a->dim - 2 * a->half + 2 * vec - 1) / (2 * vec)
                                       : (a->dim + 2 * vec - 1) / (2 * vec);
  a->group = 1;
  a->lanes_shift = 0;
  while (a->group < 32 && a->group < a->slots) {
    a->group *= 2;
    ++a->lanes_shift;
  }
}

template <typename T, int VEC>
mhla_status with_style(QkArgs& a, int style, bool backward, cudaStream_t s) {
  const bool half = style == MHLA_ROTARY_HALF;
  if constexpr (VEC >= 4) {  // at most 32 slots
    return half ? launch<T, VEC, true, 1>(a, backward, s) : launch<T, VEC, false, 1>(a, backward, s);
  } else if constexpr (VEC == 2) {
    if (a.slots <= 32) return half ? launch<T, 2, true, 1>(a, backward, s) : launch<T, 2, false, 1>(a, backward, s);
    return half ? launch<T, 2, true, 2>(a, backward, s) : launch<T, 2, false, 2>(a, backward, s);
  } else {
    if (a.slots <= 32) return launch<T, 1, true, 1>(a, backward, s);
    if (a.slots <= 64) return launch<T, 1, true, 2>(a, backward, s);
    return launch<T, 1, true, 4>(a, backward, s);
  }
}

template <typename T>
mhla_status dispatch(QkArgs& a, int style, int vec, bool backward, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (vec == 8) return with_style<T, 8>(a, style, backward, s);
  if (vec == 4) return with_style<T, 4>(a, style, backward, s);
  if (vec == 2) return with_style<T, 2>(a, style, backward, s);
  return with_style<T, 1>(a, style, backward, s);
}

mhla_status check_params(const mhla_qknorm_params* p, const mhla_rotary_table* table) {
  if (!p || p->batch < 0 || p->tokens < 0 || p->heads < 0 || p->kv_heads < 0) return MHLA_ERR_INVALID_ARG;
  if (!ops_dtype_ok(p->dtype) || !ops_dtype_ok(p->weight_dtype)) return MHLA_ERR_INVALID_ARG;
  if (p->style != MHLA_ROTARY_HALF && p->style != MHLA_ROTARY_INTERLEAVED) return MHLA_ERR_INVALID_ARG;
  if (p->position_dtype != MHLA_POSITIONS_I32 && p->position_dtype != MHLA_POSITIONS_I64) return MHLA_ERR_INVALID_ARG;
  if (!std::isfinite(p->eps) || p->eps < 0.f || p->head_dim < 1) return MHLA_ERR_INVALID_ARG;
  if (p->style == MHLA_ROTARY_INTERLEAVED && p->head_dim % 2 != 0) return MHLA_ERR_INVALID_ARG;
  if (table && (table->pairs < 1 || table->pairs > MHLA_ROTARY_MAX_PAIRS || p->head_dim < 2 * table->pairs))
    return MHLA_ERR_INVALID_ARG;
  if (p->head_dim > kMaxDim || p->heads > 32768 || p->kv_heads > 32768) return MHLA_ERR_UNSUPPORTED;
  return MHLA_OK;
}

QkArgs args_of(const mhla_qknorm_params* p, const mhla_rotary_table* table, bool k, const void* positions) {
  QkArgs a = {};
  a.heads[0] = p->heads;
  a.heads[1] = k ? p->kv_heads : 0;
  a.batch = p->batch;
  a.tokens = p->tokens;
  a.dim = p->head_dim;
  a.inv_dim = 1.f / (float)p->head_dim;
  a.eps = p->eps;
  a.w_f32 = p->weight_dtype == MHLA_DTYPE_F32;
  a.sx[0] = p->q;
  a.sx[1] = p->k;
  a.sdy[0] = p->dq_out;
  a.sdy[1] = p->dk_out;
  a.sy[0] = p->q_out;
  a.sy[1] = p->k_out;
  a.positions = positions;
  a.pos_offset = p->position_offset;
  a.pos_sb = p->position_batch_stride;
  a.pos_st = p->position_token_stride;
  a.pos64 = p->position_dtype == MHLA_POSITIONS_I64;
  a.amp = 1.f;
  if (table) {
    a.half = table->pairs;
    a.amp = table->amplitude;
    a.table = *table;
  }
  return a;
}

RowTensor rows(const void* ptr, const mhla_qknorm_params* p, int heads, const mhla_strides& s) {
  return row_tensor(ptr, p->batch, heads, p->tokens, s, p->head_dim, ops_elem(p->dtype));
}

// Tensors without rows may have no address.
bool any_rows(const mhla_qknorm_params* p, int heads) { return p->batch > 0 && p->tokens > 0 && heads > 0; }

RowTensor positions_of(const void* ptr, const mhla_qknorm_params* p) {
  const mhla_strides s = {p->position_batch_stride, 0, p->position_token_stride};
  return row_tensor(ptr, ptr ? p->batch : 0, 1, p->tokens, s, 1, p->position_dtype == MHLA_POSITIONS_I64 ? 8 : 4);
}

int least_alignment(const RowTensor* t, int n) {
  int align = 16;
  for (int i = 0; i < n; ++i)
    if (!t[i].empty()) {
      const int x = row_alignment(t[i], 16);
      align = x < align ? x : align;
    }
  return align;
}

// At least the CTAs of the backward pass, whatever the table, the pointers'
// alignment and the presence of k: rows by 32 threads take the most turns, and
// rounding up the smaller share adds one.
int64_t most_ctas(const mhla_qknorm_params* p) {
  const int64_t all = (int64_t)p->batch * p->tokens, turns = 2 * ((all + 8 - 1) / (8));
  const int64_t most = kResident * kOpsSms + 1;
  return turns < most ? turns : most;
}

}  // namespace
}  // namespace mhla

extern "C" {

mhla_status mhla_qknorm_forward(const void* q, const void* k, const void* q_weight, const void* k_weight,
                                const void* positions, const mhla_rotary_table* table, const mhla_qknorm_params* p,
                                void* q_out, void* k_out, void* stream) {
  using namespace mhla;
  const mhla_status st = check_params(p, table);
  if (st != MHLA_OK) return st;
  if (!k && any_rows(p, p->kv_heads) && (k_out || k_weight)) return MHLA_ERR_INVALID_ARG;
  const int kv = k ? p->kv_heads : 0;
  const RowTensor t[4] = {rows(q, p, p->heads, p->q), rows(k, p, kv, p->k), rows(q_out, p, p->heads, p->q_out),
                          rows(k_out, p, kv, p->k_out)};
  const size_t we = ops_elem(p->weight_dtype);
  const RowTensor side[3] = {flat_tensor(q_weight, q_weight ? p->head_dim : 0, we),
                             flat_tensor(k_weight, k_weight ? p->head_dim : 0, we), positions_of(positions, p)};
  for (int i = 0; i < 4; ++i)
    if (!row_tensor_ok(t[i], i >= 2)) return MHLA_ERR_INVALID_ARG;
  for (const RowTensor& x : side)
    if (!row_tensor_ok(x, false) || !row_tensors_apart(x, t[2]) || !row_tensors_apart(x, t[3]))
      return MHLA_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i) {
    if (!row_tensors_same(t[i], t[2 + i]) && !row_tensors_apart(t[i], t[2 + i])) return MHLA_ERR_INVALID_ARG;
    if (!row_tensors_apart(t[1 - i], t[2 + i])) return MHLA_ERR_INVALID_ARG;
  }
  if (!row_tensors_apart(t[2], t[3])) return MHLA_ERR_INVALID_ARG;
  if (p->batch == 0 || p->tokens == 0 || p->heads + kv == 0) return MHLA_OK;
  QkArgs a = args_of(p, table, k != nullptr, positions);
  a.x[0] = q;
  a.x[1] = k;
  a.y[0] = q_out;
  a.y[1] = k_out;
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  const int vec = vector_of(a.dim, a.half, p->style, (int)ops_elem(p->dtype), least_alignment(t, 4));
  shape_rows(&a, vec, p->style);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return p->dtype == MHLA_DTYPE_BF16 ? dispatch<__nv_bfloat16>(a, p->style, vec, false, s)
                                     : dispatch<float>(a, p->style, vec, false, s);
}

mhla_status mhla_qknorm_backward_workspace_bytes(const mhla_qknorm_params* p, size_t* bytes) {
  using namespace mhla;
  if (!bytes) return MHLA_ERR_INVALID_ARG;
  const mhla_status st = check_params(p, nullptr);
  if (st != MHLA_OK) return st;
  *bytes = sizeof(float) * (size_t)most_ctas(p) * (size_t)p->head_dim;
  return MHLA_OK;
}

mhla_status mhla_qknorm_backward(const void* dq_out, const void* dk_out, const void* q, const void* k,
                                 const void* q_weight, const void* k_weight, const void* positions,
                                 const mhla_rotary_table* table, const mhla_qknorm_params* p, void* dq, void* dk,
                                 float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  using namespace mhla;
  mhla_status st = check_params(p, table);
  if (st != MHLA_OK) return st;
  if (!k && any_rows(p, p->kv_heads) && (dk_out || dk || k_weight || dk_weight)) return MHLA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int kv = k ? p->kv_heads : 0;
  const RowTensor x[2] = {rows(q, p, p->heads, p->q), rows(k, p, kv, p->k)};
  const RowTensor dy[2] = {rows(dq_out, p, p->heads, p->dq_out), rows(dk_out, p, kv, p->dk_out)};
  const RowTensor dx[2] = {rows(dq, p, p->heads, p->q_out), rows(dk, p, kv, p->k_out)};
  const bool sums = dq_weight || dk_weight;
  size_t need = 0;
  if (sums && (st = mhla_qknorm_backward_workspace_bytes(p, &need)) != MHLA_OK) return st;
  const size_t we = ops_elem(p->weight_dtype);
  const RowTensor side[3] = {flat_tensor(q_weight, q_weight ? p->head_dim : 0, we),
                             flat_tensor(k_weight, k_weight ? p->head_dim : 0, we), positions_of(positions, p)};
  const RowTensor more[3] = {flat_tensor(dq_weight, dq_weight ? p->head_dim : 0, 4),
                             flat_tensor(dk_weight, dk_weight ? p->head_dim : 0, 4),
                             flat_tensor(workspace, workspace ? (int64_t)need : 0, 1)};
  const RowTensor* inputs[7] = {&x[0], &x[1], &dy[0], &dy[1], &side[0], &side[1], &side[2]};
  const RowTensor* results[5] = {&dx[0], &dx[1], &more[0], &more[1], &more[2]};
  for (const RowTensor* i : inputs)
    if (!row_tensor_ok(*i, false)) return MHLA_ERR_INVALID_ARG;
  for (int o = 0; o < 5; ++o) {
    if (!row_tensor_ok(*results[o], true)) return MHLA_ERR_INVALID_ARG;
    for (int i = 0; i < 7; ++i) {
      const bool own = o < 2 && i < 4 && i % 2 == o;  // dq over dq_out or q
      if (own && row_tensors_same(*inputs[i], *results[o])) continue;
      if (!row_tensors_apart(*inputs[i], *results[o])) return MHLA_ERR_INVALID_ARG;
    }
    for (int i = o + 1; i < 5; ++i)
      if (!row_tensors_apart(*results[i], *results[o])) return MHLA_ERR_INVALID_ARG;
  }
  QkArgs a = args_of(p, table, k != nullptr, positions);
  const RowTensor all[6] = {x[0], x[1], dy[0], dy[1], dx[0], dx[1]};
  const int vec = vector_of(a.dim, a.half, p->style, (int)ops_elem(p->dtype), least_alignment(all, 6));
  shape_rows(&a, vec, p->style);
  share_ctas(&a);
  Scratch scratch;
  // the launch's own CTAs have the last word on what their sums need
  need = std::max(need, sizeof(float) * (size_t)(a.ctas[0] + a.ctas[1]) * (size_t)a.dim);
  if (sums && (st = scratch.take(workspace, workspace_bytes, need, s)) != MHLA_OK) return st;
  a.x[0] = q;
  a.x[1] = k;
  a.dy[0] = dq_out;
  a.dy[1] = dk_out;
  a.y[0] = dq;
  a.y[1] = dk;
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  a.partial = sums ? reinterpret_cast<float*>(scratch.ptr()) : nullptr;
  if (a.ctas[0] + a.ctas[1] > 0)
    st = p->dtype == MHLA_DTYPE_BF16 ? dispatch<__nv_bfloat16>(a, p->style, vec, true, s)
                                     : dispatch<float>(a, p->style, vec, true, s);
  if (st == MHLA_OK && sums) {
    const int e = launch_pdl(qknorm_reduce_kernel, dim3((unsigned)((a.dim + 31) / 32), 2), dim3(1024), 0, s,
                             (const float*)a.partial, a.ctas[0], a.ctas[1], a.dim, dq_weight, dk_weight);
    if (e != cudaSuccess) st = record_cuda_error((cudaError_t)e);
  }
  return scratch.give_back(st);
}

}  // extern "C"
