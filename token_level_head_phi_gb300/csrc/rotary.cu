// Rotary positions: every pair (a, b) of a row becomes
// m (a cos x - b sin x, a sin x + b cos x) with x = position * f_i ("RoFormer:
// Enhanced Transformer with Rotary Position Embedding", section 3.2.2).
//
// f_i is kept as a 64-bit fraction of a turn, so that position * f_i modulo 2^64
// takes the phase of that fraction without a rounding (integer wrap-around
// drops whole turns), and its top 32 bits feed sincospif.  The fraction comes
// of doubles: it is off by less than 2^-51 of a turn for f_i <= 1 (2^-53 without
// a scaling), so the phase by less than position * 2^-51 turns, and by another
// 2^-26 from its float32 value.  At position 2^20 that is 1e-7 radians, where a
// float32 angle is off by up to 0.03.
//
// Bound: memory.  A thread takes one vector of pairs of one token, forms its
// sines once and walks over the heads of q and k with four heads' loads in
// flight.  Measured: q and k of 4 x 32k tokens x 16 heads of 64, bf16, 162 us =
// 6.6 TB/s, 98 % of a copy; calls of a few tokens are the host's 10 to 17 us.
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "ops.h"

namespace mhla {
namespace {

struct RotaryArgs {
  const void* x[2];
  void* y[2];
  mhla_strides sx[2], sy[2];
  const void* positions;
  int64_t pos_offset, pos_sb, pos_st;
  int pos64;
  int heads[2];
  int tokens;
  int64_t items;    // batch * tokens * vectors
  int vectors;      // vectors per row that are touched
  int rot_vectors;  // of which rotated
  int half;         // rot_dim / 2
  int heads_per_thread;
  float amp;
  float sin_sign;
  mhla_rotary_table table;
};

// VEC elements of a row; SCALAR loads them one by one (rows that are aligned
// to their elements only).
template <typename T, int VEC, bool SCALAR>
struct Vec {
  alignas(sizeof(T) * VEC) T v[VEC];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (SCALAR || VEC == 1) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = p[i];
    } else if constexpr (sizeof(T) * VEC == 16) {
      *reinterpret_cast<uint4*>(v) = __ldcs(reinterpret_cast<const uint4*>(p));
    } else {
      static_assert(sizeof(T) * VEC == 8, "");
      *reinterpret_cast<uint2*>(v) = __ldcs(reinterpret_cast<const uint2*>(p));
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (SCALAR || VEC == 1) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = v[i];
    } else if constexpr (sizeof(T) * VEC == 16) {
      __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(v));
    } else {
      __stcs(reinterpret_cast<uint2*>(p), *reinterpret_cast<const uint2*>(v));
    }
  }
};

// HALF: a vector is VEC pairs, entries [VEC v, VEC v + VEC) and the same
// rot_dim / 2 further on.  Otherwise it is VEC consecutive entries = VEC / 2
// pairs.  Vectors from rot_vectors on are copied.
template <typename T, int VEC, bool HALF, bool SCALAR>
__global__ void __launch_bounds__(256) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int PAIRS = HALF ? VEC : VEC / 2;
  constexpr int UNROLL = 4;
  __shared__ uint64_t turns[MHLA_ROTARY_MAX_PAIRS];
  for (int i = threadIdx.x; i < a.half; i += blockDim.x) turns[i] = a.table.turns[i];
  __syncthreads();
  const int64_t item = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= a.items) return;
  int v, t;
  int64_t b;
  if (a.items <= 0x7fffffff) {
    const uint32_t i32 = (uint32_t)item, tok = i32 / (uint32_t)a.vectors;
    v = (int)(i32 - tok * (uint32_t)a.vectors);
    b = tok / (uint32_t)a.tokens;
    t = (int)(tok - (uint32_t)b * (uint32_t)a.tokens);
  } else {
    const int64_t tok = item / a.vectors;
    v = (int)(item - tok * a.vectors);
    b = tok / a.tokens;
    t = (int)(tok - b * a.tokens);
  }
  const bool rotate = v < a.rot_vectors;
  float cs[PAIRS], sn[PAIRS];
  if (rotate) {
    int64_t pos = a.pos_offset + t;
    if (a.positions) {
      const int64_t at = b * a.pos_sb + t * a.pos_st;
      pos = a.pos64 ? static_cast<const int64_t*>(a.positions)[at] : static_cast<const int32_t*>(a.positions)[at];
    }
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      const uint64_t phase = (uint64_t)pos * turns[v * PAIRS + i];
      // signed half turns in [-1, 1)
      sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &sn[i], &cs[i]);
      cs[i] *= a.amp;
      sn[i] *= a.amp * a.sin_sign;
    }
  }
  // entry of the first element; copied vectors follow the rotated entries
  const int col = HALF ? (rotate ? v * VEC : 2 * a.half + (v - a.rot_vectors) * VEC) : v * VEC;
  const int total = a.heads[0] + a.heads[1];
  int h = blockIdx.y * a.heads_per_thread;
  const int h_end = min(h + a.heads_per_thread, total);

  auto where = [&](int hh, const T** src, T** dst) {
    const int w = hh >= a.heads[0];
    const int64_t head = w ? hh - a.heads[0] : hh;
    *src = static_cast<const T*>(a.x[w]) + b * a.sx[w].batch + head * a.sx[w].head + t * a.sx[w].token + col;
    *dst = static_cast<T*>(a.y[w]) + b * a.sy[w].batch + head * a.sy[w].head + t * a.sy[w].token + col;
  };
  auto turn = [&](Vec<T, VEC, SCALAR>& lo, Vec<T, VEC, SCALAR>& hi) {
    if constexpr (HALF) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float x = to_f32(lo.v[i]), y = to_f32(hi.v[i]);
        lo.v[i] = from_f32<T>(x * cs[i] - y * sn[i]);
        hi.v[i] = from_f32<T>(x * sn[i] + y * cs[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        const float x = to_f32(lo.v[2 * i]), y = to_f32(lo.v[2 * i + 1]);
        lo.v[2 * i] = from_f32<T>(x * cs[i] - y * sn[i]);
        lo.v[2 * i + 1] = from_f32<T>(x * sn[i] + y * cs[i]);
      }
    }
  };

  if (HALF && rotate) {
    for (; h < h_end; h += UNROLL) {
      Vec<T, VEC, SCALAR> lo[UNROLL], hi[UNROLL];
      const T* src;
      T* dst[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u)
        if (h + u < h_end) {
          where(h + u, &src, &dst[u]);
          lo[u].load(src);
          hi[u].load(src + a.half);
        }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u)
        if (h + u < h_end) {
          turn(lo[u], hi[u]);
          lo[u].store(dst[u]);
          hi[u].store(dst[u] + a.half);
        }
    }
    return;
  }
  for (; h < h_end; h += UNROLL) {
    Vec<T, VEC, SCALAR> x[UNROLL];
    const T* src;
    T* dst[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (h + u < h_end) {
        where(h + u, &src, &dst[u]);
        x[u].load(src);
      }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (h + u < h_end) {
        if (!HALF && rotate) turn(x[u], x[u]);
        x[u].store(dst[u]);
      }
  }
}

template <typename T, int VEC, bool HALF, bool SCALAR>
mhla_status launch(RotaryArgs& a, int head_dim, bool in_place, int64_t tokens, cudaStream_t s) {
  a.rot_vectors = HALF ? a.half / VEC : 2 * a.half / VEC;
  a.vectors = a.rot_vectors + (in_place ? 0 : (head_dim - 2 * a.half) / VEC);
  a.items = tokens * a.vectors;
  const int total = a.heads[0] + a.heads[1];
  // Sines are formed once for all heads that a thread walks over; heads are
  // shared out over threads only where there are too few items to fill the GPU
  // (one token of 16 sequences: 64 items).
  const int64_t want = (int64_t)kOpsSms * 2048;
  int64_t groups = (want + a.items - 1) / a.items;
  if (groups > total) groups = total;
  a.heads_per_thread = (int)((total + groups - 1) / groups);
  groups = (total + a.heads_per_thread - 1) / a.heads_per_thread;
  const int threads = a.items * groups < want ? 64 : 256;
  const int64_t blocks = (a.items + threads - 1) / threads;
  if (blocks > 0x7fffffff || groups > 65535) return MHLA_ERR_UNSUPPORTED;
  rotary_kernel<T, VEC, HALF, SCALAR><<<dim3((unsigned)blocks, (unsigned)groups), threads, 0, s>>>(a);
  return launch_status();
}

// The widest vector that divides the rotated part (each half of it for HALF),
// the rest of the row and every row start.
template <typename T>
mhla_status dispatch(RotaryArgs& a, int style, int head_dim, bool in_place, int align, int64_t tokens,
                     cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const bool half = style == MHLA_ROTARY_HALF;
  const int unit = half ? a.half : 2 * a.half;
  const int rest = head_dim - 2 * a.half;
  auto fits = [&](int vec) {
    return unit % vec == 0 && (in_place || rest % vec == 0) && align >= vec * (int)sizeof(T);
  };
  if (fits(W))
    return half ? launch<T, W, true, false>(a, head_dim, in_place, tokens, s)
                : launch<T, W, false, false>(a, head_dim, in_place, tokens, s);
  if (fits(W / 2))
    return half ? launch<T, W / 2, true, false>(a, head_dim, in_place, tokens, s)
                : launch<T, W / 2, false, false>(a, head_dim, in_place, tokens, s);
  // single pairs
  return half ? launch<T, 1, true, false>(a, head_dim, in_place, tokens, s)
              : launch<T, 2, false, true>(a, head_dim, in_place, tokens, s);
}

}  // namespace
}  // namespace mhla

extern "C" {

mhla_status mhla_rotary_table_init(int rot_dim, double base, int scaling, double factor, double original_length,
                                   mhla_rotary_table* table) {
  if (!table || rot_dim < 2 || rot_dim % 2 != 0 || rot_dim / 2 > MHLA_ROTARY_MAX_PAIRS) return MHLA_ERR_INVALID_ARG;
  if (!std::isfinite(base) || base <= 0.0) return MHLA_ERR_INVALID_ARG;
  if (scaling < MHLA_ROTARY_SCALE_NONE || scaling > MHLA_ROTARY_SCALE_PARTS) return MHLA_ERR_INVALID_ARG;
  const bool parts = scaling == MHLA_ROTARY_SCALE_PARTS;
  if (scaling != MHLA_ROTARY_SCALE_NONE && (!std::isfinite(factor) || factor <= 0.0 || (parts && factor < 1.0)))
    return MHLA_ERR_INVALID_ARG;
  if (parts && (!std::isfinite(original_length) || original_length <= 0.0)) return MHLA_ERR_INVALID_ARG;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  std::memset(table, 0, sizeof(*table));
  table->pairs = rot_dim / 2;
  table->amplitude = parts ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  if (scaling == MHLA_ROTARY_SCALE_BASE && rot_dim > 2) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  for (int i = 0; i < table->pairs; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == MHLA_ROTARY_SCALE_LINEAR) f /= factor;
    if (parts) {
      double keep = (original_length * f / kTwoPi - 1.0) / 31.0;
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f = f * (keep + (1.0 - keep) / factor);
    }
    if (!std::isfinite(f)) return MHLA_ERR_INVALID_ARG;
    double turn = f / kTwoPi;
    turn -= std::floor(turn);  // whole turns drop out
    turn = std::ldexp(turn, 64);
    table->turns[i] = turn >= 18446744073709551616.0 ? 0 : (uint64_t)turn;
  }
  return MHLA_OK;
}

mhla_status mhla_rotary(const void* q, const void* k, const void* positions, const mhla_rotary_table* table,
                        const mhla_rotary_params* p, void* q_out, void* k_out, void* stream) {
  using namespace mhla;
  if (!p || !table) return MHLA_ERR_INVALID_ARG;
  if (p->batch < 0 || p->tokens < 0 || p->heads < 0 || p->kv_heads < 0) return MHLA_ERR_INVALID_ARG;
  if (!ops_dtype_ok(p->dtype)) return MHLA_ERR_INVALID_ARG;
  if (p->style != MHLA_ROTARY_HALF && p->style != MHLA_ROTARY_INTERLEAVED) return MHLA_ERR_INVALID_ARG;
  if (p->transpose != 0 && p->transpose != 1) return MHLA_ERR_INVALID_ARG;
  if (p->position_dtype != MHLA_POSITIONS_I32 && p->position_dtype != MHLA_POSITIONS_I64) return MHLA_ERR_INVALID_ARG;
  if (table->pairs < 1 || table->pairs > MHLA_ROTARY_MAX_PAIRS) return MHLA_ERR_INVALID_ARG;
  if (p->head_dim < 2 * table->pairs || p->head_dim > 1024) return MHLA_ERR_INVALID_ARG;
  // neighbours are paired: no entry may be left over
  if (p->style == MHLA_ROTARY_INTERLEAVED && p->head_dim % 2 != 0) return MHLA_ERR_INVALID_ARG;
  const size_t e = ops_elem(p->dtype);
  const int kv = k ? p->kv_heads : 0;
  if (!k && k_out) return MHLA_ERR_INVALID_ARG;
  if (p->heads > 32768 || kv > 32768) return MHLA_ERR_UNSUPPORTED;
  const RowTensor in[2] = {row_tensor(q, p->batch, p->heads, p->tokens, p->q, p->head_dim, e),
                           row_tensor(k, p->batch, kv, p->tokens, p->k, p->head_dim, e)};
  const RowTensor out[2] = {row_tensor(q_out, p->batch, p->heads, p->tokens, p->q_out, p->head_dim, e),
                            row_tensor(k_out, p->batch, kv, p->tokens, p->k_out, p->head_dim, e)};
  bool in_place = true;
  for (int i = 0; i < 2; ++i)
    if (!row_tensor_ok(in[i], false) || !row_tensor_ok(out[i], true)) return MHLA_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i) {
    if (out[i].empty()) continue;
    const bool same = row_tensors_same(in[i], out[i]);
    if (!same && !row_tensors_apart(in[i], out[i])) return MHLA_ERR_INVALID_ARG;
    if (!row_tensors_apart(in[1 - i], out[i])) return MHLA_ERR_INVALID_ARG;
    in_place = in_place && same;
  }
  if (!row_tensors_apart(out[0], out[1])) return MHLA_ERR_INVALID_ARG;
  const int64_t tokens = (int64_t)p->batch * p->tokens;
  if (tokens == 0 || p->heads + kv == 0) return MHLA_OK;
  if (positions) {
    const size_t pe = p->position_dtype == MHLA_POSITIONS_I64 ? 8 : 4;
    const mhla_strides ps = {p->position_batch_stride, 0, p->position_token_stride};
    const RowTensor pt = row_tensor(positions, p->batch, 1, p->tokens, ps, 1, pe);
    if (!row_tensor_ok(pt, false)) return MHLA_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i)
      if (!row_tensors_apart(pt, out[i])) return MHLA_ERR_INVALID_ARG;
  }
  RotaryArgs a = {};
  int align = 16;
  for (int i = 0; i < 2; ++i) {
    a.x[i] = in[i].ptr;
    a.y[i] = const_cast<void*>(out[i].ptr);
    a.heads[i] = (int)in[i].n[1];
    if (in[i].empty()) continue;
    const int ai = row_alignment(in[i], 16), ao = row_alignment(out[i], 16);
    align = ai < align ? ai : align;
    align = ao < align ? ao : align;
  }
  a.sx[0] = p->q;
  a.sx[1] = p->k;
  a.sy[0] = p->q_out;
  a.sy[1] = p->k_out;
  a.positions = positions;
  a.pos_offset = p->position_offset;
  a.pos_sb = p->position_batch_stride;
  a.pos_st = p->position_token_stride;
  a.pos64 = p->position_dtype == MHLA_POSITIONS_I64;
  a.tokens = p->tokens;
  a.half = table->pairs;
  a.amp = table->amplitude;
  a.sin_sign = p->transpose ? -1.f : 1.f;
  a.table = *table;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return p->dtype == MHLA_DTYPE_BF16 ? dispatch<__nv_bfloat16>(a, p->style, p->head_dim, in_place, align, tokens, s)
                                     : dispatch<float>(a, p->style, p->head_dim, in_place, align, tokens, s);
}

}  // extern "C"
