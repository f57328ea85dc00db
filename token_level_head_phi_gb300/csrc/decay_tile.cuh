// Shared-memory tiles of bf16 rows for the tensor-core kernels of the decayed
// linear attention: layout, asynchronous loading, and the split of weighted
// values into bf16 parts.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace mhla {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Byte offset of 16-byte piece `piece` of row `row` in a tile of D-entry bf16
// rows: pieces are permuted so that eight rows' pieces of one column fall into
// different banks.
template <int D>
__device__ __forceinline__ uint32_t tile_off(int row, int piece) {
  constexpr int kPieces = D / 8;
  if constexpr (kPieces >= 8)
    return (uint32_t)(row * (D * 2) + ((piece ^ (row & 7)) << 4));
  else
    return (uint32_t)(row * (D * 2) + ((piece ^ ((row / (8 / kPieces)) & (kPieces - 1))) << 4));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Pairs of float32 in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
  const float2 f = unpair(v);
  return pack2(f.x, f.y);
}

// Two bf16 values times their common weight, as sums of PARTS bf16 parts.
template <int PARTS>
__device__ __forceinline__ void scale_split2(uint32_t v, uint64_t w, uint32_t (&o)[PARTS]) {
  const uint64_t minus = pair(-1.f, -1.f);
  uint64_t a = mul2(pair(lo_f(v), hi_f(v)), w);
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    o[i] = pack2(a);
    if (i + 1 < PARTS) a = fma2(pair(lo_f(o[i]), hi_f(o[i])), minus, a);
  }
}

// Two bf16 values times their weights, as sums of PARTS bf16 parts (8 bits each).
template <int PARTS>
__device__ __forceinline__ void scale_split(uint32_t v, float w0, float w1, uint32_t (&o)[PARTS]) {
  float a = lo_f(v) * w0, b = hi_f(v) * w1;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    o[i] = pack2(a, b);
    a -= lo_f(o[i]), b -= hi_f(o[i]);
  }
}

// Copies ROWS rows of C-token chunk after chunk of one tensor into tiles, by
// THREADS threads; rows from n on are zeros.  A thread takes the same 16-byte piece of
// every STEP-th row.
template <int D, int C, int ROWS, int THREADS>
struct RowLoader {
  static constexpr int kPieces = D / 8;
  static constexpr int kStep = THREADS / kPieces;  // rows taken at a time
  static constexpr int kTurns = ROWS / kStep;
  static_assert(THREADS % kPieces == 0 && ROWS % kStep == 0, "");
  const __nv_bfloat16* src;  // this thread's piece of its first row
  int64_t step;              // elements from token to token of the pass
  int row, piece;

  __device__ __forceinline__ void init(const __nv_bfloat16* first, int64_t token_step, int r0, int thread) {
    row = r0 + thread / kPieces;
    piece = thread % kPieces;
    step = token_step;
    src = first + row * token_step + piece * 8;
  }
  __device__ __forceinline__ void load(__nv_bfloat16* tile, int n, bool vec) {
    const __nv_bfloat16* at = src;
    if (vec && n == C) {
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        const uint32_t dst = smem_addr(tile) + tile_off<D>(row + i * kStep, piece);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(at) : "memory");
        at += kStep * step;
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < kTurns; ++i) {
        const int r = row + i * kStep;
        const bool live = r < n;
        alignas(16) __nv_bfloat16 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __float2bfloat16_rn(0.f);
        if (live && vec) {
          *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(at);
        } else if (live) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = at[j];
        }
        *reinterpret_cast<uint4*>(reinterpret_cast<char*>(tile) + tile_off<D>(r, piece)) = *reinterpret_cast<uint4*>(v);
        at += kStep * step;
      }
    }
    src += C * step;
  }
};

}  // namespace mhla
