// What the strided operators (rotary positions, layer norm, decayed linear
// attention) share on the host: checks of strided tensors, scratch memory and
// error reporting.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mhla.h"

namespace mhla {

// Keeps the text of a CUDA error for mhla_last_error_string.
mhla_status record_cuda_error(cudaError_t e);

// The device error word that kernels with bounded waits write.
mhla_status ops_error_ptr(unsigned int** out);

constexpr int kOpsSms = 152;  // SMs of a GB300: grids are sized in multiples of it

inline size_t ops_elem(int dtype) { return dtype == MHLA_DTYPE_BF16 ? 2 : 4; }
inline bool ops_dtype_ok(int dtype) { return dtype == MHLA_DTYPE_BF16 || dtype == MHLA_DTYPE_F32; }

// A tensor of contiguous rows [batch, head, token] for the checks below.
struct RowTensor {
  const void* ptr;
  int64_t n[3];       // batch, heads, tokens
  int64_t stride[3];  // elements
  int64_t row;        // elements of a row
  size_t elem;        // bytes of an element

  bool empty() const { return n[0] == 0 || n[1] == 0 || n[2] == 0 || row == 0; }
  // bytes from the first to behind the last element
  int64_t extent() const {
    int64_t e = row;
    for (int i = 0; i < 3; ++i) e += (n[i] - 1) * stride[i];
    return e * (int64_t)elem;
  }
};

inline RowTensor row_tensor(const void* ptr, int64_t b, int64_t h, int64_t t, const mhla_strides& s, int64_t row,
                            size_t elem) {
  return RowTensor{ptr, {b, h, t}, {s.batch, s.head, s.token}, row, elem};
}

// A flat buffer as one row.
inline RowTensor flat_tensor(const void* ptr, int64_t n, size_t elem) {
  return RowTensor{ptr, {1, 1, 1}, {0, 0, 0}, n, elem};
}

// Pointer, alignment and stride checks; an output's rows must not overlap.
inline bool row_tensor_ok(const RowTensor& t, bool output) {
  if (t.empty()) return true;
  if (!t.ptr || (uintptr_t)t.ptr % t.elem != 0) return false;
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 3; ++i) {
    // strides and extents far below 2^62 elements, so sums cannot wrap
    if (t.n[i] > 1 && (t.stride[i] < 0 || t.stride[i] > ((int64_t)1 << 56) / t.n[i])) return false;
  }
  if (!output) return true;
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (t.stride[order[j]] < t.stride[order[i]]) {
        const int x = order[i];
        order[i] = order[j];
        order[j] = x;
      }
  int64_t inner = t.row;  // elements one step of the next axis has to clear
  for (int i = 0; i < 3; ++i) {
    const int a = order[i];
    if (t.n[a] <= 1) continue;
    if (t.stride[a] < inner) return false;
    inner += t.stride[a] * (t.n[a] - 1);
  }
  return true;
}

// The same memory with adjacent rows joined (the heads of a token-major
// tensor) and axes that do not move (one entry, stride 0) dropped.
inline RowTensor joined_rows(RowTensor t) {
  for (int i = 0; i < 3; ++i)
    if (t.n[i] <= 1 || t.stride[i] == 0) t.n[i] = 1, t.stride[i] = 0;
  for (int pass = 0; pass < 3; ++pass)
    for (int i = 0; i < 3; ++i)
      if (t.n[i] > 1 && t.stride[i] == t.row) {
        t.row *= t.n[i];
        t.n[i] = 1;
        t.stride[i] = 0;
      }
  return t;
}

// Whether two tensors certainly share no byte: their extents are apart, or
// all their rows lie at residues of one common stride that are apart (slices
// of one fused buffer, such as the q, k and v parts of a projection).
inline bool row_tensors_apart(const RowTensor& first, const RowTensor& second) {
  if (first.empty() || second.empty() || !first.ptr || !second.ptr) return true;
  const RowTensor a = joined_rows(first), b = joined_rows(second);
  const uintptr_t pa = (uintptr_t)a.ptr, pb = (uintptr_t)b.ptr;
  if (pa + (uintptr_t)a.extent() <= pb || pb + (uintptr_t)b.extent() <= pa) return true;
  int64_t g = 0;  // of all strides, in bytes
  const RowTensor* both[2] = {&a, &b};
  for (const RowTensor* t : both)
    for (int i = 0; i < 3; ++i) {
      int64_t x = t->stride[i] * (int64_t)t->elem;
      while (x) {
        const int64_t r = g % x;
        g = x;
        x = r;
      }
    }
  if (g == 0) return false;
  const int64_t ra = a.row * (int64_t)a.elem, rb = b.row * (int64_t)b.elem;
  // where b's rows start, counted from a's, modulo g
  int64_t d = (int64_t)(pb - pa) % g;
  if (d < 0) d += g;
  return d >= ra && d + rb <= g;
}

// Exactly the same rows (an operation in place).
inline bool row_tensors_same(const RowTensor& a, const RowTensor& b) {
  if (a.ptr != b.ptr || a.elem != b.elem || a.row != b.row) return false;
  for (int i = 0; i < 3; ++i)
    if (a.n[i] != b.n[i] || (a.n[i] > 1 && a.stride[i] != b.stride[i])) return false;
  return true;
}

// Largest power of two, at most `most` bytes, that divides every row start.
inline int row_alignment(const RowTensor& t, int most) {
  uintptr_t bits = (uintptr_t)t.ptr | (uintptr_t)most;
  for (int i = 0; i < 3; ++i)
    if (t.n[i] > 1) bits |= (uintptr_t)(t.stride[i] * (int64_t)t.elem);
  return (int)(bits & (~bits + 1));
}

// Scratch memory of a call: the caller's workspace, or stream-ordered memory
// that give_back returns.
class Scratch {
 public:
  mhla_status take(void* workspace, size_t have, size_t need, cudaStream_t s) {
    stream_ = s;
    if (!workspace) {
      if (have != 0) return MHLA_ERR_INVALID_ARG;
      if (need == 0) return MHLA_OK;
      const cudaError_t e = cudaMallocAsync(&ptr_, need, s);
      if (e != cudaSuccess) {
        ptr_ = nullptr;
        return record_cuda_error(e);
      }
      owned_ = true;
      return MHLA_OK;
    }
    if (have < need) return MHLA_ERR_WORKSPACE;
    if (need && (uintptr_t)workspace % 256 != 0) return MHLA_ERR_INVALID_ARG;
    ptr_ = workspace;
    return MHLA_OK;
  }
  char* ptr() const { return static_cast<char*>(ptr_); }
  mhla_status give_back(mhla_status st) {
    if (owned_) {
      owned_ = false;
      const cudaError_t e = cudaFreeAsync(ptr_, stream_);
      if (st == MHLA_OK && e != cudaSuccess) return record_cuda_error(e);
    }
    return st;
  }

 private:
  void* ptr_ = nullptr;
  cudaStream_t stream_ = nullptr;
  bool owned_ = false;
};

inline mhla_status launch_status() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MHLA_OK : record_cuda_error(e);
}

}  // namespace mhla
