// C entries of linear attention with a decay for each head (declared in
// include/mhla.h): checks, the segment plan and the passes of decay.h.
#include <algorithm>
#include <cmath>

#include "decay.h"
#include "ops.h"

namespace mhla {
namespace {

bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

mhla_status check_params(const mhla_decay_params* p) {
  if (!p || p->batch < 0 || p->heads < 0 || p->tokens < 0) return MHLA_ERR_INVALID_ARG;
  if (!dim_ok(p->key_dim) || !dim_ok(p->value_dim) || !ops_dtype_ok(p->dtype)) return MHLA_ERR_INVALID_ARG;
  if (p->variant < MHLA_DECAY_AUTO || p->variant > MHLA_DECAY_TENSOR || !std::isfinite(p->scale))
    return MHLA_ERR_INVALID_ARG;
  if (p->variant == MHLA_DECAY_TENSOR && p->dtype != MHLA_DTYPE_BF16) return MHLA_ERR_UNSUPPORTED;
  if ((int64_t)p->batch * p->heads > (1 << 24) || p->tokens > (1 << 30)) return MHLA_ERR_UNSUPPORTED;
  return MHLA_OK;
}

bool on_tensor_cores(const mhla_decay_params* p) {
  return p->dtype == MHLA_DTYPE_BF16 && p->variant != MHLA_DECAY_SIMT;
}

// The tcgen05 kernels take rows of 64 and 128 entries and slices of 64 columns
// (and 16-byte alignment, and at least one chunk of 128 tokens).  They are
// ahead of the mma.sync kernel there: 64 heads of 64 entries, 128 tokens 10.8
// against 12.8 us, 2k tokens 39 against 56, 32k tokens 287 against 414; of 128
// entries, 128 tokens 12.8 against 14.8, 60 heads of 2k tokens 54 against 111,
// 64 of 32k 621 against 1690 (graph launches, cold L2).
bool big_tiles(int dx, int dz) { return dx >= 64 && dz % 64 == 0; }

// Segments of a pass, and with them the slices of z.  CTAs (units x slices x
// segments) run in waves of those that are resident at once.  In each wave a
// segment costs its tokens and about a hundred more for its start, and all
// segments but the last cost half of that in the launch that forms their states
// (0.9 for 128-entry rows, with two CTAs an SM; two such launches serve the
// three gradients).  The launches themselves cost about 6 us = 250 tokens.  The
// cheapest count wins; segments are of at least 128 tokens (64 on the CUDA
// cores) and at most 64.  (32k tokens x 64 heads of 64: 19 segments 287 us, 9 to
// 16 306 to 336, 4 371; of 128: 14 617, 4 695, 1 713; backward on 3 x 200 tokens
// x 5 heads of 64: 1 14, 2 24; CUDA cores, 777 tokens x 15 heads of 64: 13
// segments 37 us, 7 48; 400 tokens x 8 heads: 29 with 64-token segments, 44; rows
// of 128, where one CTA fits an SM: 60 heads of 2k tokens 581 us in one segment,
// 714 in five, as for two CTAs.)
//
// The tcgen05 kernel for 128-entry rows also has a choice of slice: 64 columns
// take 0.8 of the time of 128, and where that fills the SMs with one segment,
// no states are needed (60 heads of 2k tokens: 54 us, 128 columns in one
// segment 66, in two 70; 64 heads of 4k: 99, 119 and 123).
//
// `passes` run side by side (the gradients) and share the SMs: 2 x 8k tokens x
// 16 heads of 64, 3 segments 111 us, 8 as for one pass 113; 4 x 2k tokens, one
// segment 55, 4 as for one pass 72.  On the CUDA cores: 2 x 500 tokens x 4 heads
// of 128, counted as two CTAs an SM 100 us, as one 148; 2 x 2k x 16 heads of 64 / 32,
// as three 178, as two 264.
constexpr int kSegMost = 64, kSegStart = 100, kSegLaunches = 250;
constexpr double kNarrow = 0.8, kStates = 0.5, kStatesWide = 0.9;

struct Plan {
  int nseg, seg_len;
  int slice;  // columns of z that a CTA takes
};

Plan plan_segments(const mhla_decay_params* p, int dx, int dz, int passes) {
  const bool tc = on_tensor_cores(p) && big_tiles(dx, dz), mma = on_tensor_cores(p) && !tc;
  const bool wide = tc && dx == 128;
  const int widest = std::min(dz, wide ? 128 : mma && dx == 128 ? 32 : 64);
  const int narrowest = wide ? 64 : widest;
  // CTAs of an SM.  Three passes on the CUDA cores never run all at once (the
  // states come first), and counting more of them than fit is ahead.
  const int resident = wide          ? 1
                       : tc          ? 2
                       : mma         ? 3
                       : passes == 1 ? decay_simt_resident(dx, widest)
                                     : (dx * widest <= 2048 ? 3 : 2);
  const int64_t slots = resident * kOpsSms, state_slots = (wide ? 2 : resident) * kOpsSms;
  const int quantum = on_tensor_cores(p) ? 128 : 64;  // a chunk, or the larger of two kernels' chunks
  const int tokens = std::max(1, (p->tokens + quantum - 1) / quantum) * quantum;
  Plan best = {};
  double least = 0.;
  for (int slice = widest; slice >= narrowest; slice /= 2) {
    const int64_t ctas = (int64_t)p->batch * p->heads * (dz / slice) * passes;
    for (int n = 1; n <= kSegMost; ++n) {
      const int len = (tokens / quantum + n - 1) / n * quantum;
      if (n > 1 && (p->tokens + len - 1) / len != n) continue;
      const double weight = wide && slice == 64 ? kNarrow : 1.;
      const double pass = weight * (double)((ctas * n + slots - 1) / slots) * (len + kSegStart);
      const int64_t parts = ctas / passes * std::min(passes, 2) * (n - 1);
      double states = (wide ? kStatesWide : kStates) * weight *
                      (double)((parts + state_slots - 1) / state_slots) * (len + kSegStart);
      if (n > 1) states += kSegLaunches;
      if (best.nseg == 0 || pass + states < least) {
        least = pass + states;
        best = {n, len, slice};
      }
    }
  }
  return best;
}

size_t pass_workspace(const mhla_decay_params* p, int dx, int dz, int passes) {
  const Plan plan = plan_segments(p, dx, dz, passes);
  const size_t bytes = plan.nseg > 1 ? sizeof(float) * (size_t)p->batch * p->heads * plan.nseg * dx * dz : 0;
  return (bytes + 255) / 256 * 256;
}

RowTensor tensor(const mhla_decay_params* p, const void* ptr, const mhla_strides& s, int dim) {
  return row_tensor(ptr, p->batch, p->heads, p->tokens, s, dim, ops_elem(p->dtype));
}

RowTensor state_tensor(const mhla_decay_params* p, const float* ptr) {
  return flat_tensor(ptr, ptr ? (int64_t)p->batch * p->heads * p->key_dim * p->value_dim : 0, 4);
}

bool state_ok(const RowTensor& t) { return row_tensor_ok(t, false) && (uintptr_t)t.ptr % 16 == 0; }

DecayPass pass_of(const mhla_decay_params* p, int dx, int dz, int passes, unsigned int* err) {
  DecayPass a = {};
  a.B = p->batch;
  a.H = p->heads;
  a.N = p->tokens;
  a.DX = dx;
  a.DZ = dz;
  const Plan plan = plan_segments(p, dx, dz, passes);
  a.nseg = plan.nseg;
  a.seg_len = plan.seg_len;
  a.slice = plan.slice;
  a.launches = 3;
  a.err = err;
  return a;
}

void set_rows(DecayPass& a, const RowTensor& x, const mhla_strides& sx, const RowTensor& y, const mhla_strides& sy,
              const RowTensor& z, const mhla_strides& sz, const RowTensor& o, const mhla_strides& so) {
  a.x = x.ptr;
  a.y = y.ptr;
  a.z = z.ptr;
  a.o = const_cast<void*>(o.ptr);
  a.sx = sx;
  a.sy = sy;
  a.sz = sz;
  a.so = so;
  a.vec = row_alignment(x, 16) == 16 && row_alignment(y, 16) == 16 && row_alignment(z, 16) == 16 &&
          row_alignment(o, 16) == 16;
}

mhla_status copy_state(const mhla_decay_params* p, const float* from, float* to, cudaStream_t s) {
  if (!to || to == from) return MHLA_OK;
  const size_t n = sizeof(float) * (size_t)p->batch * p->heads * p->key_dim * p->value_dim;
  const cudaError_t e =
      from ? cudaMemcpyAsync(to, from, n, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(to, 0, n, s);
  return e == cudaSuccess ? MHLA_OK : record_cuda_error(e);
}

cudaError_t launch_pass(const DecayPass& a, const mhla_decay_params* p, cudaStream_t s) {
  if (!on_tensor_cores(p)) return launch_decay_simt(a, p->dtype, s);
  if (big_tiles(a.DX, a.DZ) && a.vec && a.N >= 128) {
    // not supported: strides that a tensor map cannot hold, such as a broadcast axis
    const cudaError_t e = launch_decay_tc(a, s);
    if (e != cudaErrorNotSupported) return e;
  }
  return launch_decay_mma(a, s);
}

// Two side streams of one caller's stream, in the calling thread and on the
// current device.  The passes of the three gradients run side by side on them:
// alone, each of them leaves SMs idle at its start and end and wherever its
// segments do not fill a wave (2 x 8k tokens x 16 heads of 64: 134 us one after
// another, 111 side by side; 4 x 2k tokens: 91 and 55; 3 x 777 tokens x 5 heads,
// float32: 93 and 66; 16 tokens of one head: 27 and 14).  A capture of the
// caller's stream takes the side streams along, as branches of its graph.  Side
// streams that several callers' streams shared would order those streams' work
// behind one another; a thread keeps pairs for its first kPairs streams, and on
// further ones the passes run one after another.
constexpr int kGradients = 3;
constexpr int kPairs = 16;

class Branches {
 public:
  ~Branches() {
    for (int i = 0; i < 2; ++i) {
      if (stream_[i]) cudaStreamDestroy(stream_[i]);
      if (done_[i]) cudaEventDestroy(done_[i]);
    }
    if (ready_) cudaEventDestroy(ready_);
  }
  bool serves(int device, cudaStream_t s) const { return made_ && device_ == device && caller_ == s; }
  // Whether the side streams can follow s: they exist and are in no capture
  // but that of s.
  bool open(int device, cudaStream_t s) {
    if (!made_) made_ = make(s) ? 1 : -1;
    device_ = device;
    caller_ = s;
    used_ = 0;
    unsigned long long id[3] = {};
    bool same = made_ == 1 && capture(s, &id[2]);
    for (int i = 0; i < 2; ++i) same = same && capture(stream_[i], &id[i]) && id[i] == (id[i] ? id[2] : 0);
    if (!same) cudaGetLastError();
    return same;
  }
  // Side stream i, behind what s holds now; s itself if that fails.
  cudaStream_t fork(int i, cudaStream_t s) {
    if (cudaEventRecord(ready_, s) != cudaSuccess || cudaStreamWaitEvent(stream_[i], ready_, 0) != cudaSuccess) {
      cudaGetLastError();
      return s;
    }
    used_ |= 1 << i;
    return stream_[i];
  }
  // s waits for the side streams.
  cudaError_t join(cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 2; ++i) {
      if (!(used_ >> i & 1)) continue;
      cudaError_t j = cudaEventRecord(done_[i], stream_[i]);
      if (j == cudaSuccess) j = cudaStreamWaitEvent(s, done_[i], 0);
      if (e == cudaSuccess) e = j;
    }
    return e;
  }

 private:
  static bool capture(cudaStream_t s, unsigned long long* id) {  // its id, 0 outside one
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    if (cudaStreamGetCaptureInfo(s, &status, id) != cudaSuccess || status == cudaStreamCaptureStatusInvalidated)
      return false;
    if (status == cudaStreamCaptureStatusNone) *id = 0;
    return true;
  }
  bool make(cudaStream_t s) {
    // nothing here is part of a capture that may be under way
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    const bool relaxed = cudaThreadExchangeStreamCaptureMode(&mode) == cudaSuccess;
    int priority = 0;
    if (cudaStreamGetPriority(s, &priority) != cudaSuccess) priority = 0;
    bool ok = cudaEventCreateWithFlags(&ready_, cudaEventDisableTiming) == cudaSuccess;
    for (int i = 0; i < 2; ++i)
      ok = ok && cudaStreamCreateWithPriority(&stream_[i], cudaStreamNonBlocking, priority) == cudaSuccess &&
           cudaEventCreateWithFlags(&done_[i], cudaEventDisableTiming) == cudaSuccess;
    if (relaxed) cudaThreadExchangeStreamCaptureMode(&mode);
    return ok;
  }
  int made_ = 0, used_ = 0, device_ = 0;
  cudaStream_t caller_ = nullptr;
  cudaStream_t stream_[2] = {};
  cudaEvent_t ready_ = nullptr, done_[2] = {};
};

// The side streams of s, ready to follow it, or null.
Branches* branches(cudaStream_t s) {
  thread_local Branches pairs[kPairs];
  thread_local int used = 0;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return nullptr;
  int i = 0;
  while (i < used && !pairs[i].serves(device, s)) ++i;
  if (i == kPairs) return nullptr;
  if (i == used) ++used;
  return pairs[i].open(device, s) ? &pairs[i] : nullptr;
}

// Whether `out` shares memory with none of `in`.
bool apart_from_all(const RowTensor& out, const RowTensor* in, int n) {
  for (int i = 0; i < n; ++i)
    if (!row_tensors_apart(out, in[i])) return false;
  return true;
}

}  // namespace
}  // namespace mhla

extern "C" {

mhla_status mhla_decay_workspace_bytes(const mhla_decay_params* p, size_t* bytes) {
  using namespace mhla;
  if (!bytes) return MHLA_ERR_INVALID_ARG;
  const mhla_status st = check_params(p);
  if (st != MHLA_OK) return st;
  *bytes = pass_workspace(p, p->key_dim, p->value_dim, 1);
  return MHLA_OK;
}

mhla_status mhla_decay_forward(const void* q, const void* k, const void* v, const float* log_decay,
                               const int32_t* lengths, const float* state_in, const mhla_decay_params* p, void* out,
                               float* state_out, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace mhla;
  mhla_status st = check_params(p);
  if (st != MHLA_OK) return st;
  if ((int64_t)p->batch * p->heads == 0) return MHLA_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RowTensor in[6] = {tensor(p, q, p->q, p->key_dim),         tensor(p, k, p->k, p->key_dim),
                           tensor(p, v, p->v, p->value_dim),       flat_tensor(log_decay, p->heads, 4),
                           flat_tensor(lengths, lengths ? p->batch : 0, 4), state_tensor(p, state_in)};
  const RowTensor to = tensor(p, out, p->out, p->value_dim), ts = state_tensor(p, state_out);
  for (const RowTensor& t : in)
    if (!row_tensor_ok(t, false)) return MHLA_ERR_INVALID_ARG;
  if (!row_tensor_ok(to, true) || !state_ok(in[5]) || !state_ok(ts)) return MHLA_ERR_INVALID_ARG;
  if (!apart_from_all(to, in, 6) || !row_tensors_apart(to, ts) || !apart_from_all(ts, in, 5))
    return MHLA_ERR_INVALID_ARG;
  if (state_out != state_in && !row_tensors_apart(ts, in[5])) return MHLA_ERR_INVALID_ARG;
  if (p->tokens == 0) return copy_state(p, state_in, state_out, s);
  const size_t need = pass_workspace(p, p->key_dim, p->value_dim, 1);
  const RowTensor tw = flat_tensor(workspace, workspace ? (int64_t)need : 0, 1);
  if (!apart_from_all(tw, in, 6) || !row_tensors_apart(tw, to) || !row_tensors_apart(tw, ts))
    return MHLA_ERR_INVALID_ARG;
  Scratch scratch;
  if ((st = scratch.take(workspace, workspace_bytes, need, s)) != MHLA_OK) return st;
  unsigned int* err = nullptr;
  if ((st = ops_error_ptr(&err)) != MHLA_OK) return scratch.give_back(st);
  DecayPass a = pass_of(p, p->key_dim, p->value_dim, 1, err);
  set_rows(a, in[0], p->q, in[1], p->k, in[2], p->v, to, p->out);
  a.g = log_decay;
  a.lengths = lengths;
  a.s_in = state_in;
  a.s_out = state_out;
  a.s_ldx = p->value_dim;
  a.s_ldz = 1;
  a.seg = reinterpret_cast<float*>(scratch.ptr());
  a.e = 1;
  a.score = a.read = p->scale;
  a.update = 1.f;
  const cudaError_t e = launch_pass(a, p, s);
  return scratch.give_back(e == cudaSuccess ? MHLA_OK : record_cuda_error(e));
}

mhla_status mhla_decay_backward_workspace_bytes(const mhla_decay_params* p, size_t* bytes) {
  using namespace mhla;
  if (!bytes) return MHLA_ERR_INVALID_ARG;
  const mhla_status st = check_params(p);
  if (st != MHLA_OK) return st;
  *bytes = pass_workspace(p, p->value_dim, p->key_dim, kGradients) +
           pass_workspace(p, p->key_dim, p->value_dim, kGradients);
  return MHLA_OK;
}

mhla_status mhla_decay_backward(const void* q, const void* k, const void* v, const float* log_decay,
                                const int32_t* lengths, const float* state_in, const void* dout,
                                const float* dstate_out, const mhla_decay_params* p, void* dq, void* dk, void* dv,
                                float* dstate_in, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace mhla;
  mhla_status st = check_params(p);
  if (st != MHLA_OK) return st;
  if ((int64_t)p->batch * p->heads == 0) return MHLA_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RowTensor in[8] = {tensor(p, q, p->q, p->key_dim),     tensor(p, k, p->k, p->key_dim),
                           tensor(p, v, p->v, p->value_dim),   tensor(p, dout, p->dout, p->value_dim),
                           flat_tensor(log_decay, p->heads, 4), flat_tensor(lengths, lengths ? p->batch : 0, 4),
                           state_tensor(p, state_in),          state_tensor(p, dstate_out)};
  const RowTensor out[3] = {tensor(p, dq, p->dq, p->key_dim), tensor(p, dk, p->dk, p->key_dim),
                            tensor(p, dv, p->dv, p->value_dim)};
  const RowTensor ts = state_tensor(p, dstate_in);
  for (const RowTensor& t : in)
    if (!row_tensor_ok(t, false)) return MHLA_ERR_INVALID_ARG;
  if (!state_ok(in[6]) || !state_ok(in[7]) || !state_ok(ts)) return MHLA_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    if (!row_tensor_ok(out[i], true)) return MHLA_ERR_INVALID_ARG;
    if (!apart_from_all(out[i], in, 8) || !row_tensors_apart(out[i], ts)) return MHLA_ERR_INVALID_ARG;
    if (!apart_from_all(out[i], out, i)) return MHLA_ERR_INVALID_ARG;
  }
  if (!apart_from_all(ts, in, 7)) return MHLA_ERR_INVALID_ARG;
  if (dstate_in != dstate_out && !row_tensors_apart(ts, in[7])) return MHLA_ERR_INVALID_ARG;
  if (p->tokens == 0) return copy_state(p, dstate_out, dstate_in, s);
  size_t need = 0;
  if ((st = mhla_decay_backward_workspace_bytes(p, &need)) != MHLA_OK) return st;
  const RowTensor tw = flat_tensor(workspace, workspace ? (int64_t)need : 0, 1);
  if (!apart_from_all(tw, in, 8) || !apart_from_all(tw, out, 3) || !row_tensors_apart(tw, ts))
    return MHLA_ERR_INVALID_ARG;
  Scratch scratch;
  if ((st = scratch.take(workspace, workspace_bytes, need, s)) != MHLA_OK) return st;
  float* seg = reinterpret_cast<float*>(scratch.ptr());
  const int dkey = p->key_dim, dval = p->value_dim;

  unsigned int* err = nullptr;
  if ((st = ops_error_ptr(&err)) != MHLA_OK) return scratch.give_back(st);
  DecayPass a = pass_of(p, dval, dkey, kGradients, err);  // dq
  set_rows(a, in[3], p->dout, in[2], p->v, in[1], p->k, out[0], p->dq);
  a.g = log_decay;
  a.lengths = lengths;
  a.s_in = state_in;
  a.s_ldx = 1;
  a.s_ldz = dval;
  a.seg = seg;
  a.e = 1;
  a.score = a.read = p->scale;
  a.update = 1.f;

  // dk and dv carry the same states, transposed: the segments' own are formed
  // once, in dv's orientation.
  DecayPass c = pass_of(p, dkey, dval, kGradients, err);  // dv, and the gradient of the first state
  set_rows(c, in[1], p->k, in[0], p->q, in[3], p->dout, out[2], p->dv);
  c.g = log_decay;
  c.lengths = lengths;
  c.s_in = dstate_out;
  c.s_out = dstate_in;
  c.s_ldx = dval;
  c.s_ldz = 1;
  c.seg = seg + pass_workspace(p, dval, dkey, kGradients) / sizeof(float);
  c.reverse = 1;
  c.e = 0;
  c.score = p->scale;
  c.read = 1.f;
  c.update = p->scale;
  DecayPass b = c;  // dk
  b.DX = dval;
  b.DZ = dkey;
  set_rows(b, in[2], p->v, in[3], p->dout, in[0], p->q, out[1], p->dk);
  b.s_out = nullptr;
  b.s_ldx = 1;
  b.s_ldz = dval;
  b.launches = 2;
  c.launches = 1;
  Branches* side = branches(s);
  const cudaStream_t sa = side ? side->fork(0, s) : s;
  cudaError_t e = launch_pass(a, p, sa);
  if (e == cudaSuccess) e = launch_pass(c, p, s);
  // with one segment dk reads dstate_out while dv's pass writes dstate_in
  const cudaStream_t sb = side && (c.nseg > 1 || !dstate_in || dstate_in != dstate_out) ? side->fork(1, s) : s;
  if (e == cudaSuccess) e = launch_pass(b, p, sb);
  c.launches = 2;
  if (e == cudaSuccess) e = launch_pass(c, p, s);
  if (side) {
    const cudaError_t j = side->join(s);
    if (e == cudaSuccess) e = j;
  }
  return scratch.give_back(e == cudaSuccess ? MHLA_OK : record_cuda_error(e));
}

mhla_status mhla_decay_step(const void* q, const void* k, const void* v, const float* log_decay,
                            const float* state_in, const mhla_decay_params* p, void* out, float* state_out,
                            void* stream) {
  using namespace mhla;
  mhla_status st = check_params(p);
  if (st != MHLA_OK) return st;
  if (p->tokens != 1) return MHLA_ERR_INVALID_ARG;
  if ((int64_t)p->batch * p->heads == 0) return MHLA_OK;
  const RowTensor in[5] = {tensor(p, q, p->q, p->key_dim), tensor(p, k, p->k, p->key_dim),
                           tensor(p, v, p->v, p->value_dim), flat_tensor(log_decay, p->heads, 4),
                           state_tensor(p, state_in)};
  const RowTensor to = tensor(p, out, p->out, p->value_dim), ts = state_tensor(p, state_out);
  for (const RowTensor& t : in)
    if (!row_tensor_ok(t, false)) return MHLA_ERR_INVALID_ARG;
  if (!row_tensor_ok(to, true) || !state_ok(in[4]) || !state_ok(ts)) return MHLA_ERR_INVALID_ARG;
  if (!apart_from_all(to, in, 5) || !row_tensors_apart(to, ts) || !apart_from_all(ts, in, 4))
    return MHLA_ERR_INVALID_ARG;
  if (state_out != state_in && !row_tensors_apart(ts, in[4])) return MHLA_ERR_INVALID_ARG;
  DecayPass a = pass_of(p, p->key_dim, p->value_dim, 1, nullptr);
  set_rows(a, in[0], p->q, in[1], p->k, in[2], p->v, to, p->out);
  a.g = log_decay;
  a.s_in = state_in;
  a.s_out = state_out;
  a.read = p->scale;
  const cudaError_t e = launch_decay_step(a, p->dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MHLA_OK : record_cuda_error(e);
}

}  // extern "C"
