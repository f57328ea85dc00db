// What the tcgen05 kernels of the decayed linear attention share: row maps,
// TMA and tensor-memory helpers.
#pragma once

#include "decay.h"
#include "tc_common.cuh"
#include "tc_host.h"

namespace mhla {

using namespace tc;

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}

// True in one lane of a converged warp.  Work under this predicate, in a warp
// whose index comes from a shuffle, keeps its addresses and descriptors in
// uniform registers: a product issues in 40 cycles instead of 100 under
// `lane == 0`.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0u;
}

// A map of rows and the places of its token, head and batch axes (1 to 3,
// ordered by stride).
struct RowMap {
  CUtensorMap map;
  int token, head, batch;
};
struct TcArgs {
  RowMap x, y, z, o;
  RowMap y64, z64;  // in boxes of 64 rows
  DecayPass p;
};

__device__ __forceinline__ int coordinate(const RowMap& m, int axis, int token, int head, int batch) {
  return m.token == axis ? token : m.head == axis ? head : batch;
}
__device__ __forceinline__ void load_rows(uint32_t dst, const RowMap& m, uint32_t bar, int col, int token, int head,
                                          int batch) {
  tma_load_4d(dst, &m.map, bar, col, coordinate(m, 1, token, head, batch), coordinate(m, 2, token, head, batch),
              coordinate(m, 3, token, head, batch), policy_evict_first());
}

// E entries of a state along x, ldx apart, from a 16-byte boundary.
template <int E>
__device__ __forceinline__ void read_state(float (&s)[E], const float* from, int ldx) {
  if (ldx == 1) {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(from + i);
      s[i] = v.x, s[i + 1] = v.y, s[i + 2] = v.z, s[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) s[i] = from[(int64_t)i * ldx];
  }
}
template <int E>
__device__ __forceinline__ void write_state(const float (&s)[E], float* to, int ldx) {
  if (ldx == 1) {
#pragma unroll
    for (int i = 0; i < E; i += 4)
      *reinterpret_cast<float4*>(to + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) to[(int64_t)i * ldx] = s[i];
  }
}

// Axes ordered by stride, as nested as they are in memory.
inline bool make_map(RowMap* m, const void* base, const mhla_strides& st, int64_t cols, const DecayPass& p, int box_cols,
              int box_rows, int swizzle) {
  struct Axis {
    int64_t n, stride;
    int* place;
    uint32_t box;
  } ax[3] = {{p.N, st.token, &m->token, (uint32_t)box_rows}, {p.H, st.head, &m->head, 1u}, {p.B, st.batch, &m->batch, 1u}};
  for (Axis& x : ax) {
    if (x.n > 1 && x.stride <= 0) return false;  // a broadcast axis
    if (x.n <= 1) x.stride = (int64_t)1 << 34;   // never stepped along
  }
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (ax[j].stride < ax[i].stride) {
        const Axis t = ax[i];
        ax[i] = ax[j];
        ax[j] = t;
      }
  uint64_t dims[4] = {(uint64_t)cols}, strides[3];
  uint32_t box[4] = {(uint32_t)box_cols};
  for (int i = 0; i < 3; ++i) {
    *ax[i].place = i + 1;
    dims[i + 1] = (uint64_t)ax[i].n;
    strides[i] = 2ull * (uint64_t)ax[i].stride;
    if (strides[i] >= (1ull << 40)) return false;
    box[i + 1] = ax[i].box;
  }
  return encode_tmap_rows(&m->map, base, dims, strides, box, swizzle);
}

template <class K>
cudaError_t room(K* kernel, size_t smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

// The pass over rows of 128 entries (decay_tc_wide.cu).
cudaError_t launch_decay_tc_wide(const TcArgs& a, cudaStream_t s);

}  // namespace mhla
