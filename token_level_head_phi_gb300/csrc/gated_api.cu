// C entries of the gated recurrence: checks, scratch, launches.
#include <algorithm>

#include "gated.cuh"
#include "tc_host.h"

namespace mhla {
namespace {

// Adds the CTAs' rows in order: 32 channels per CTA, 32 threads to one.
__global__ void __launch_bounds__(1024) gated_reduce_kernel(const float* partial, int rows, int D, float* out) {
  __shared__ float sh[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
  float s = 0.f;
  after_predecessor();
  if (c < D)
    for (int r = ty; r < rows; r += 32) s += partial[(int64_t)r * D + c];
  sh[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && c < D) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += sh[i][tx];
    out[c] = t;
  }
}

mhla_status check_params(const mhla_gated_params* p, const float* log_decay) {
  if (!p || p->batch < 0 || p->tokens < 0 || p->width < 0 || !ops_dtype_ok(p->dtype)) return MHLA_ERR_INVALID_ARG;
  if (p->kind != MHLA_GATED_DECAY && p->kind != MHLA_GATED_SIGMOID) return MHLA_ERR_INVALID_ARG;
  if (p->scale < MHLA_GATED_SCALE_NORM || p->scale > MHLA_GATED_SCALE_NONE) return MHLA_ERR_INVALID_ARG;
  if (p->marks != 0 && p->marks != 1) return MHLA_ERR_INVALID_ARG;
  // tokens and channels are counted in 32 bits, tokens up to three rounds of a
  // cluster's tiles past the end
  static_assert(3 * kGatedCluster * kGatedWarps * 16 < 0x1000, "room behind the last token");
  if (p->tokens > 0x7ffff000 || p->width > 0x7ffff000) return MHLA_ERR_UNSUPPORTED;
  if ((p->kind == MHLA_GATED_DECAY) != (log_decay != nullptr) && p->width > 0) return MHLA_ERR_INVALID_ARG;
  return MHLA_OK;
}

int64_t marks_of(const mhla_gated_params* p) { return ((int64_t)p->tokens + MHLA_GATED_MARK - 1) / MHLA_GATED_MARK; }

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
  a.n_marks = (int)marks_of(p);
  a.slabs = (p->width + kGatedSlab - 1) / kGatedSlab;
  a.scale = p->scale;
  return a;
}

// Rows of the sums for log_decay's gradient.
int64_t partial_rows(const mhla_gated_params* p) {
  const int64_t units = (int64_t)p->batch * ((p->width + kGatedSlab - 1) / kGatedSlab);
  return (int64_t)p->batch * gated_cluster(units, p->tokens, p->dtype == MHLA_DTYPE_F32, true);
}

// Bytes of the backward pass's scratch: those sums, and the marks that it forms.
size_t scratch_bytes(const mhla_gated_params* p, bool sums) {
  const size_t state = sizeof(float) * (size_t)p->batch * (size_t)p->width;
  return (sums ? partial_rows(p) * sizeof(float) * (size_t)p->width : 0) + (p->marks ? 0 : state * (size_t)marks_of(p));
}

// 2, 1 or 0: rows of all of these start at multiples of 16 bytes, of a pair of
// elements, or of one.
int alignment_of(const RowTensor* t, int n) {
  int level = 2;
  for (int i = 0; i < n; ++i) {
    if (t[i].empty()) continue;
    const int a = row_alignment(t[i], 16), mine = a == 16 ? 2 : a >= 2 * (int)t[i].elem ? 1 : 0;
    level = mine < level ? mine : level;
  }
  return level;
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
                            floats(marks, marks_of(p) * state)};
  if (!apart(in, 6, res, 3, &in[5], &res[1])) return MHLA_ERR_INVALID_ARG;
  if (state == 0) return MHLA_OK;
  GatedArgs a = args_of(p, x, gate, input_gate, log_decay, lengths);
  a.state_in = state_in;
  a.out = out;
  a.so = p->out;
  a.state_out = state_out;
  a.marks = marks;
  a.vec = std::min(alignment_of(in, 3), alignment_of(res, 1));
  return launch_gated_fwd(a, p->dtype, p->kind, static_cast<cudaStream_t>(stream));
}

mhla_status mhla_gated_backward_workspace_bytes(const mhla_gated_params* p, size_t* bytes) {
  using namespace mhla;
  static const float some = 0.f;
  if (!bytes || !p) return MHLA_ERR_INVALID_ARG;
  const mhla_status st = check_params(p, p->kind == MHLA_GATED_DECAY ? &some : nullptr);
  if (st != MHLA_OK) return st;
  *bytes = scratch_bytes(p, p->kind == MHLA_GATED_DECAY);
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
  const size_t need = scratch_bytes(p, dlog_decay != nullptr);
  const RowTensor none = floats(nullptr, 0);
  const RowTensor in[9] = {rows(x, p, p->x), rows(gate, p, p->gate),
                           input_gate ? rows(input_gate, p, p->input_gate) : none, rows(dout, p, p->dout),
                           floats(log_decay, p->width), floats(lengths, p->batch), floats(state_in, state),
                           floats(marks, marks_of(p) * state), floats(dstate_out, state)};
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
  if (dlog_decay) {
    a.partial = at;
    at += partial_rows(p) * p->width;
  }
  a.state_in = state_in;
  a.vec = std::min(alignment_of(in, 4), alignment_of(res, 3));
  a.marks = const_cast<float*>(marks);
  if (!marks && a.n_marks > 0) {
    a.marks = at;
    st = launch_gated_fwd(a, p->dtype, p->kind, s);  // the states alone
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
  if (st == MHLA_OK) st = launch_gated_bwd(a, p->dtype, p->kind, s);
  if (st == MHLA_OK && dlog_decay) {
    const int e = launch_pdl(gated_reduce_kernel, dim3((unsigned)((p->width + 31) / 32)), dim3(1024), 0, s,
                             (const float*)a.partial, (int)partial_rows(p), p->width, dlog_decay);
    if (e != cudaSuccess) st = record_cuda_error((cudaError_t)e);
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
  a.vec = std::min(alignment_of(in, 3), alignment_of(res, 1));
  return launch_gated_step(a, p->dtype, p->kind, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
