// Linear attention with a decay for each head on the fifth-generation tensor
// cores (bf16 rows of 64 entries, 16-byte aligned; see decay.h for the pass).
//
// Why beside the mma.sync kernel: there every product takes issue slots from
// the decay, split and state arithmetic around it (measured: 8 products and 32
// independent multiply-adds take 45 ns, 33 ns and 17 ns alone), which bounds it
// at about twice the time its memory traffic needs.  Here one thread issues
// the products, operands stay in shared and tensor memory, and two CTAs share
// an SM, each a plain sequence of steps that the other one's steps fill.
//
// A CTA of eight working warps and one that issues takes (unit, segment, 64
// columns of z) in 128-token chunks; row t of a chunk is lane t of tensor
// memory and belongs to two threads (a half of the columns each):
//   D = X Y^T and O = X S                               -> barrier A
//   w Y in bf16 parts: the high one over Y, the next beside it
//   O *= lambda^(t + e), P = D decayed and masked, as bf16 in tensor memory
//   O += P Z and U = Z^T [parts of w Y]                 -> barrier B
//   S = lambda^n S + sum of U's parts; O to memory
// U has 64 rows; its operand Z repeats (leading offset 0), so that lanes 64 to
// 127 hold the same rows again and all eight warps share the state update.
// Roundings: as in the mma.sync kernel.
//
// Columns of tensor memory (256 of 512 a CTA): D 0-127, overlaid by U once P
// is formed; P 128-191; O 192-255.  The first launch (OUT = false) forms the
// states alone: U 0-127.
#include <type_traits>

#include "decay.h"
#include "decay_tile.cuh"
#include "ops.h"
#include "tc_common.cuh"
#include "tc_host.h"

namespace mhla {
namespace {

using namespace tc;

constexpr int C = 128;       // tokens of a chunk
constexpr int D = 64;        // entries of a row, columns of a slice
constexpr int kWork = 256;   // working threads
constexpr int kThreads = kWork + 32;
constexpr uint32_t kTile = C * D * 2;
constexpr uint32_t kColP = 128, kColO = 192;

// Shared memory, from a 1024-byte boundary: y, y, z, z, mid, then x and s (OUT)
// or lo, then the rest.
template <bool OUT>
struct Layout {
  static constexpr uint32_t y = 0, z = 2 * kTile, mid = 4 * kTile;
  static constexpr uint32_t x = 5 * kTile;   // OUT; its last use in a chunk over, the third part of w Y
  static constexpr uint32_t lo = 5 * kTile;
  static constexpr uint32_t s = 6 * kTile;   // OUT
  static constexpr uint32_t tail = OUT ? 6 * kTile + kTile / 2 : 6 * kTile;
  static constexpr uint32_t bytes = tail + 1024;
};
struct alignas(16) Tail {
  float tab[64];     // lambda^d of the diagonal block at 31 + d, 0 for d < 0
  float cw[32];      // lambda^(32 - j)
  float p32[4];      // lambda^(32 m)
  uint64_t bar[2];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Tail) <= 1024, "");

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

template <bool OUT>
__global__ void __launch_bounds__(kThreads, 2) decay_tc_kernel(const DecayPass p) {
  using L = Layout<OUT>;
  using T = __nv_bfloat16;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* mem = raw + (base - smem_u32(raw));
  Tail& tail = *reinterpret_cast<Tail*>(mem + L::tail);
  constexpr uint32_t kCols = OUT ? 256 : 128;

  const int unit = blockIdx.x, seg = blockIdx.y, z0 = blockIdx.z * D;
  const int b = unit / p.H, h = unit % p.H;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int q = warp & 3, half = (warp >> 2) & 1;  // lanes 32 q .. of tensor memory, half of the columns
  const float g = p.g[h];
  const int length = decay_length(p, b);
  const int begin = seg * p.seg_len;
  const int end = min(begin + p.seg_len, p.N);
  const int valid = max(0, min(end, length) - begin);
  const bool last = seg == (length > 0 ? (length - 1) / p.seg_len : 0);
  const bool exact = p.s_out && (!OUT || last);  // three parts where a final state comes of it
  const int t0 = valid > 0 ? decay_token(p, begin, length) : 0;
  const int64_t sign = p.reverse ? -1 : 1;
  T* o = static_cast<T*>(p.o) + b * p.so.batch + h * p.so.head + z0;
  const int64_t one = (int64_t)D * p.DZ, state = unit * one;
  float* segs = p.seg + (p.nseg > 1 ? (int64_t)unit * p.nseg * one : 0);

  const uint32_t bar_a = smem_u32(&tail.bar[0]), bar_b = smem_u32(&tail.bar[1]);
  if (tid == 0) {
    mbar_init(bar_a, 1);
    mbar_init(bar_b, 1);
    tail.abort = 0;
    fence_barrier_init();
  }
  if (warp == kWork / 32) {
    tmem_alloc(smem_u32(&tail.tmem), kCols);
    tmem_relinquish();
  }

  // the ninth warp loads the chunks and issues the products
  RowLoader<D, C, C, 32> lx, ly, lz;
  if (warp == kWork / 32) {
    if (OUT)
      lx.init(static_cast<const T*>(p.x) + b * p.sx.batch + h * p.sx.head + t0 * p.sx.token, sign * p.sx.token, 0, lane);
    ly.init(static_cast<const T*>(p.y) + b * p.sy.batch + h * p.sy.head + t0 * p.sy.token, sign * p.sy.token, 0, lane);
    lz.init(static_cast<const T*>(p.z) + b * p.sz.batch + h * p.sz.head + t0 * p.sz.token + z0, sign * p.sz.token, 0, lane);
    if (valid > 0) {
      ly.load(reinterpret_cast<T*>(mem + L::y), min(C, valid), true);
      if (OUT) lx.load(reinterpret_cast<T*>(mem + L::x), min(C, valid), true);
      lz.load(reinterpret_cast<T*>(mem + L::z), min(C, valid), true);
    }
  }
  if (tid < 64) {
    const float2 w = decay_power(g, max(tid - 31, 0));
    tail.tab[tid] = tid >= 31 ? (w.x + w.y) * p.score : 0.f;
  } else if (tid < 96) {
    const float2 w = decay_power(g, 32 - lane);
    tail.cw[lane] = w.x + w.y;
  } else if (tid < 100) {
    const float2 w = decay_power(g, 32 * (tid - 96));
    tail.p32[tid - 96] = w.x + w.y;
  }
  if (!OUT) decay_dependents();
  if (OUT && p.nseg > 1) decay_wait();

  // This thread's part of the state: column dz of z, entries dx0 .. dx0 + 15.
  const int dz = 32 * (q & 1) + lane, dx0 = 16 * ((q >> 1) * 2 + half);
  float s[16];
  const float* before = !OUT ? nullptr : p.nseg > 1 ? segs + seg * one : p.s_in ? p.s_in + state : nullptr;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    s[i] = before && tid < kWork ? before[(int64_t)(dx0 + i) * p.s_ldx + (int64_t)(z0 + dz) * p.s_ldz] : 0.f;
  auto publish = [&]() {  // S as the second operand of X S: row dz, its entries along the row
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = pack2(s[2 * i], s[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint4*>(mem + L::s + tile_off<D>(dz, dx0 / 8 + i)) =
          make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  };
  if (OUT && tid < kWork) publish();

  // weights of this thread's rows: row t of the outputs, row j of w Y
  const int row = 32 * q + lane;
  const float2 w_read = decay_power(g, row + p.e);
  const float read = (w_read.x + w_read.y) * p.read;
  const uint64_t read2 = pair(read, read);
  const float2 w_lane = decay_power(g, lane);
  const float lane_score = (w_lane.x + w_lane.y) * p.score;
  const int j_row = tid & (C - 1);
  const float2 w_full = decay_power(g, C - j_row - p.e);
  const float2 carry = decay_power(g, C);

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tail.tmem, tmq = tm + ((uint32_t)(32 * q) << 16);
  if (OUT && tid < kWork) {  // blocks of P above the diagonal stay zero
    uint32_t zero[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) zero[i] = 0u;
    tmem_st32(tmq + kColP + 32 * half, zero);
    tmem_wait_st();
  }

  volatile int* abort_flag = &tail.abort;
  bool ok = true;
  if (warp == kWork / 32) {
    // ------------------------------------------------ issues the products
    constexpr uint32_t id_d = idesc_bf16_f32(128, 128, false, false), id_o = idesc_bf16_f32(128, 64, false, false);
    constexpr uint32_t id_p = idesc_bf16_f32(128, 64, false, true);
    constexpr uint32_t id_u = idesc_bf16_f32(128, 128, true, true), id_l = idesc_bf16_f32(128, 64, true, true);
    for (int c0 = 0; c0 < valid; c0 += C) {
      const uint32_t st = (uint32_t)(c0 / C) & 1u;
      const uint32_t ya = base + L::y + st * kTile, za = base + L::z + st * kTile;
      const bool more = c0 + C < valid;
      const int n_next = min(C, valid - c0 - C);
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async();
      if (__syncthreads_or(!ok)) break;
      if (OUT && lane == 0) {
        tc_fence_after();
        const uint64_t xd = sdesc_sw128(base + L::x, 0u, 1024u), yd = sdesc_sw128(ya, 0u, 1024u);
        const uint64_t sd = sdesc_sw128(base + L::s, 0u, 1024u);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_bf16(tm, xd + 2 * k, yd + 2 * k, id_d, k > 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_bf16(tm + kColO, xd + 2 * k, sd + 2 * k, id_o, k > 0);
        umma_commit(bar_a);
      }
      __syncwarp();
      if (more) {
        ly.load(reinterpret_cast<T*>(mem + L::y + (st ^ 1u) * kTile), n_next, true);
        lz.load(reinterpret_cast<T*>(mem + L::z + (st ^ 1u) * kTile), n_next, true);
        if (OUT && !exact) {
          ok = mbar_wait(bar_a, st, p.err, 0xd03, abort_flag);
          lx.load(reinterpret_cast<T*>(mem + L::x), n_next, true);
        }
      }
      if (__syncthreads_or(!ok)) break;
      if (lane == 0) {
        tc_fence_after();
        const uint64_t zd = sdesc_sw128(za, 0u, 1024u);
        if (OUT) {
#pragma unroll
          for (int k = 0; k < 8; ++k) umma_tmem_a(tm + kColO, tm + kColP + 8u * k, zd + 128 * k, id_p, 1u);
        }
        const uint64_t wd = sdesc_sw128(ya, base + L::mid - ya, 1024u);
#pragma unroll
        for (int k = 0; k < 8; ++k) umma_bf16(tm, zd + 128 * k, wd + 128 * k, id_u, k > 0);
        if (exact) {  // the third part adds to the second
          const uint64_t ld = sdesc_sw128(base + L::lo, 0u, 1024u);
#pragma unroll
          for (int k = 0; k < 8; ++k) umma_bf16(tm + 64u, zd + 128 * k, ld + 128 * k, id_l, 1u);
        }
        umma_commit(bar_b);
      }
      __syncwarp();
      if (OUT && more && exact) {  // x has held the third part of w Y
        ok = mbar_wait(bar_b, st, p.err, 0xd04, abort_flag);
        lx.load(reinterpret_cast<T*>(mem + L::x), n_next, true);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    for (int c0 = 0; c0 < valid; c0 += C) {
      const int n = min(C, valid - c0);
      const uint32_t st = (uint32_t)(c0 / C) & 1u;
      uint8_t* yt = mem + L::y + st * kTile;
      fence_proxy_async();
      if (__syncthreads_or(!ok)) break;  // the chunk and the state's copy are there
      // half a row of w Y; a tile's pieces are read and written by one thread
      float wj = (w_full.x + w_full.y) * p.update;
      if (n < C) {
        const float2 w = decay_power(g, max(n - j_row - p.e, 0));
        wj = (w.x + w.y) * p.update;
      }
      const uint64_t wj2 = pair(wj, wj);
      const int piece0 = 4 * (tid >> 7);
      // pieces i of the row as PARTS parts; the first part takes the row's place
      auto split = [&](auto parts, auto&& first) {
        constexpr int kParts = decltype(parts)::value;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t off = tile_off<D>(j_row, piece0 + i);
          const uint4 v = *reinterpret_cast<const uint4*>(yt + off);
          uint32_t a[kParts], c[kParts], d[kParts], e[kParts];
          scale_split2<kParts>(v.x, wj2, a);
          scale_split2<kParts>(v.y, wj2, c);
          scale_split2<kParts>(v.z, wj2, d);
          scale_split2<kParts>(v.w, wj2, e);
          first(i, off, make_uint4(a[0], c[0], d[0], e[0]));
          *reinterpret_cast<uint4*>(mem + L::mid + off) = make_uint4(a[1], c[1], d[1], e[1]);
          if constexpr (kParts == 3)
            *reinterpret_cast<uint4*>(mem + L::lo + off) = make_uint4(a[2], c[2], d[2], e[2]);
        }
      };
      using Two = std::integral_constant<int, 2>;
      using Three = std::integral_constant<int, 3>;
      auto in_place = [&](int, uint32_t off, uint4 v) { *reinterpret_cast<uint4*>(yt + off) = v; };
      if (OUT && !exact) {  // while the first products still read the rows
        uint4 hi[4];
        split(Two(), [&](int i, uint32_t, uint4 v) { hi[i] = v; });
        ok = mbar_wait(bar_a, st, p.err, 0xd01, abort_flag);
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(yt + tile_off<D>(j_row, piece0 + i)) = hi[i];
      } else {
        if (OUT) {
          ok = mbar_wait(bar_a, st, p.err, 0xd01, abort_flag);
          tc_fence_after();
        }
        if (exact)
          split(Three(), in_place);
        else
          split(Two(), in_place);
      }
      if (OUT) {
        float v[32];
        tmem_ld32(tmq + kColO + 32 * half, v);
        tmem_wait_ld();
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 f = unpair(mul2(pair(v[2 * i], v[2 * i + 1]), read2));
          r[2 * i] = __float_as_uint(f.x), r[2 * i + 1] = __float_as_uint(f.y);
        }
        tmem_st32(tmq + kColO + 32 * half, r);
        // P in blocks of 32 columns up to the diagonal, shared out over the
        // two warps of a row
        const int blocks = q + 1, middle = (blocks + 1) / 2;
        for (int k = half ? middle : 0; k < (half ? blocks : middle); ++k) {
          tmem_ld32(tmq + 32 * k, v);
          tmem_wait_ld();
          uint32_t pk[16];
          if (k == q) {
            // masked entries are dropped by selection: their scores may be infinite
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = lane >= i ? v[i] * tail.tab[31 + lane - i] : 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = pack2(v[2 * i], v[2 * i + 1]);
          } else {
            const float f = lane_score * tail.p32[q - k - 1];
            const uint64_t f2 = pair(f, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 c = reinterpret_cast<const float4*>(tail.cw)[i];
              pk[2 * i] = pack2(mul2(mul2(pair(v[4 * i], v[4 * i + 1]), f2), pair(c.x, c.y)));
              pk[2 * i + 1] = pack2(mul2(mul2(pair(v[4 * i + 2], v[4 * i + 3]), f2), pair(c.z, c.w)));
            }
          }
          tmem_st16(tmq + kColP + 16 * k, pk);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      fence_proxy_async();
      if (__syncthreads_or(!ok)) break;  // P, O and the parts of w Y are there
      ok = mbar_wait(bar_b, st, p.err, 0xd02, abort_flag);
      tc_fence_after();
      const float2 w = n == C ? carry : decay_power(g, n);
      float u0[16], u1[16];
      tmem_ld16(tmq + dx0, u0);
      tmem_ld16(tmq + 64 + dx0, u1);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t old = pair(s[2 * i], s[2 * i + 1]);
        const uint64_t u = add2(pair(u0[2 * i], u0[2 * i + 1]), pair(u1[2 * i], u1[2 * i + 1]));
        const float2 f = unpair(fma2(old, pair(w.x, w.x), fma2(old, pair(w.y, w.y), u)));
        s[2 * i] = f.x, s[2 * i + 1] = f.y;
      }
      if (OUT) {
        publish();
        float v[32];
        tmem_ld32(tmq + kColO + 32 * half, v);
        tmem_wait_ld();
        // rows to memory through the warp's own part of a tile, so that eight
        // rows' 64-byte halves leave together
        uint8_t* stage = mem + L::mid;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(stage + tile_off<D>(row, 4 * half + i)) =
              make_uint4(pack2(v[8 * i], v[8 * i + 1]), pack2(v[8 * i + 2], v[8 * i + 3]),
                         pack2(v[8 * i + 4], v[8 * i + 5]), pack2(v[8 * i + 6], v[8 * i + 7]));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 32 * q + 8 * i + lane / 4, piece = 4 * half + lane % 4;
          const uint4 t = *reinterpret_cast<const uint4*>(stage + tile_off<D>(r, piece));
          if (r < n)
            __stcs(reinterpret_cast<uint4*>(o + decay_token(p, begin + c0 + r, length) * p.so.token + piece * 8), t);
        }
      }
      tc_fence_before();
    }
  }

  __syncthreads();
  if (warp == kWork / 32) {
    tmem_dealloc(tm, kCols);
    return;
  }
  if (OUT) {
    for (int i = tid; i < (end - begin - valid) * D; i += kWork)
      o[(int64_t)(begin + valid + i / D) * p.so.token + i % D] = __float2bfloat16_rn(0.f);
    if (!last || !p.s_out) return;
  } else if (valid == 0) {
    return;
  }
  float* to = OUT ? p.s_out + state : segs + (seg + 1) * one;
#pragma unroll
  for (int i = 0; i < 16; ++i) to[(int64_t)(dx0 + i) * p.s_ldx + (int64_t)(z0 + dz) * p.s_ldz] = s[i];
}

template <bool OUT>
cudaError_t prepare() {
  return cudaFuncSetAttribute(decay_tc_kernel<OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)(Layout<OUT>::bytes + 1024));
}

}  // namespace

cudaError_t launch_decay_tc(const DecayPass& p, cudaStream_t s) {
  const unsigned units = (unsigned)(p.B * p.H), slices = (unsigned)(p.DZ / D);
  cudaError_t e;
  if (p.nseg > 1 && (p.launches & 1)) {
    if ((e = prepare<false>()) != cudaSuccess) return e;
    decay_tc_kernel<false><<<dim3(units, (unsigned)(p.nseg - 1), slices), kThreads, Layout<false>::bytes + 1024, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_decay_scan(p, s)) != cudaSuccess) return e;
  }
  if (!(p.launches & 2)) return cudaSuccess;
  if ((e = prepare<true>()) != cudaSuccess) return e;
  const dim3 grid(units, (unsigned)p.nseg, slices);
  constexpr size_t smem = Layout<true>::bytes + 1024;
  if (p.nseg > 1) return (cudaError_t)launch_pdl(decay_tc_kernel<true>, grid, dim3(kThreads), smem, s, p);
  decay_tc_kernel<true><<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace mhla
