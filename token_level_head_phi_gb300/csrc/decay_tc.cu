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
// A CTA of eight working warps and one that loads (TMA) and issues takes (unit,
// segment, 64 columns of z) in 128-token chunks; row t of a chunk is lane t of tensor
// memory and belongs to two threads (a half of the columns each):
//   D = X Y^T and O = X S                               -> barrier A
//   w Y in bf16 parts: the high one over Y, the next beside it
//   O *= lambda^(t + e), P = D decayed and masked, as bf16 in tensor memory
//   U = Z^T [parts of w Y]                              -> barrier U
//   O += P Z                                            -> barrier B
//   S = lambda^n S + sum of U's parts, then O to memory
// U has 64 rows; its operand Z repeats (leading offset 0), so that lanes 64 to
// 127 hold the same rows again and all eight warps share the state update.
// Roundings: as in the mma.sync kernel.
//
// A pass from the last token to the first (REV) takes its chunks from the end
// and keeps the tokens of a chunk in their order in memory: row r is place 127
// - r of the pass, and the triangle of P is mirrored.  The first tokens' chunk
// then starts before the sequence, where loads give zeros.
//
// Columns of tensor memory (256 of 512 a CTA): D 0-127, overlaid by U once P
// is formed; P 128-191; O 192-255.
//
// The first launch forms the segments' states alone.  A chunk there is a chain
// of waits (load, split, products, update) that other CTAs' chains fill: where
// there are CTAs enough for four on every SM, a kernel of its own takes
// 64-token chunks with four working warps (32k tokens x 64 heads: 287 against
// 300 us in all); with fewer, this one (OUT = false, U in columns 0-127) is
// ahead (8k tokens x 64 heads: 105 against 113 us; backward on 8k x 32 heads:
// 109 against 122 us).  For rows of 128 entries the 64-token kernel forms the
// states and decay_tc_wide.cu has the pass.
//
// Measured, 16k tokens x 64 heads alone: states 55 us, pass 96 us = 5.3 TB/s.
// Bound by the chains of a chunk, with shared memory (loads, parts, operands of
// the products, outputs) busy for two thirds of the time.
#include <type_traits>

#include "decay_tc.cuh"
#include "decay_tile.cuh"
#include "ops.h"

namespace mhla {
namespace {

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
  float cw[32];      // lambda^(32 - j), reversed for REV
  float p32[4];      // lambda^(32 m)
  uint64_t bar[4], full[2], full_x;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Tail) <= 1024, "");

template <bool OUT, bool REV>
__global__ void __launch_bounds__(kThreads, 2) decay_tc_kernel(const __grid_constant__ TcArgs a) {
  const DecayPass& p = a.p;
  using L = Layout<OUT>;
  using T = __nv_bfloat16;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* mem = raw + (base - smem_u32(raw));
  Tail& tail = *reinterpret_cast<Tail*>(mem + L::tail);
  constexpr uint32_t kCols = OUT ? 256 : 128;

  const int unit = blockIdx.x, seg = blockIdx.y, z0 = blockIdx.z * D;
  const int b = unit / p.H, h = unit % p.H;
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid / 32, 0), lane = tid % 32;
  const int q = warp & 3, half = (warp >> 2) & 1;  // lanes 32 q .. of tensor memory, half of the columns
  const float g = p.g[h];
  const int length = decay_length(p, b);
  const int begin = seg * p.seg_len;
  const int end = min(begin + p.seg_len, p.N);
  const int valid = max(0, min(end, length) - begin);
  const bool last = seg == (length > 0 ? (length - 1) / p.seg_len : 0);
  const bool exact = p.s_out && (!OUT || last);  // three parts where a final state comes of it
  auto first_token = [&](int c0) { return REV ? length - begin - c0 - C : begin + c0; };  // of row 0
  T* o = static_cast<T*>(p.o) + b * p.so.batch + h * p.so.head + z0;
  const int64_t one = (int64_t)D * p.DZ, state = unit * one;
  float* segs = p.seg + (p.nseg > 1 ? (int64_t)unit * p.nseg * one : 0);

  const uint32_t bar_a = smem_u32(&tail.bar[0]), bar_b = smem_u32(&tail.bar[1]), bar_u = smem_u32(&tail.bar[2]);
  const uint32_t bar_r = smem_u32(&tail.bar[3]);  // the outputs before have been read out of shared memory (8 warps)
  const uint32_t full[2] = {smem_u32(&tail.full[0]), smem_u32(&tail.full[1])}, full_x = smem_u32(&tail.full_x);
  // the ninth warp's first lane loads the chunks and issues the products
  const bool issuer = warp == kWork / 32 && elect_one();
  int loaded = 0, loaded_x = 0, seen = 0, seen_x = 0;  // chunks asked for, and waited for
  auto fetch = [&](int c0) {
    const uint32_t st = (uint32_t)(c0 / C) & 1u;
    mbar_arrive_expect_tx(full[st], 2 * kTile);
    load_rows(base + L::y + st * kTile, a.y, full[st], 0, first_token(c0), h, b);
    load_rows(base + L::z + st * kTile, a.z, full[st], z0, first_token(c0), h, b);
    ++loaded;
  };
  auto fetch_x = [&](int c0) {
    mbar_arrive_expect_tx(full_x, kTile);
    load_rows(base + L::x, a.x, full_x, 0, first_token(c0), h, b);
    ++loaded_x;
  };
  if (issuer) {
    mbar_init(bar_a, 1);
    mbar_init(bar_b, 1);
    mbar_init(bar_u, 1);
    mbar_init(bar_r, kWork / 32);
    mbar_init(full[0], 1);
    mbar_init(full[1], 1);
    mbar_init(full_x, 1);
    tail.abort = 0;
    fence_barrier_init();
    if (valid > 0) {
      fetch(0);
      if (OUT) fetch_x(0);
    }
  }
  if (warp == kWork / 32) {
    __syncwarp();
    tmem_alloc(smem_u32(&tail.tmem), kCols);
    tmem_relinquish();
  }
  if (tid < 64) {
    const float2 w = decay_power(g, max(tid - 31, 0));
    tail.tab[tid] = tid >= 31 ? (w.x + w.y) * p.score : 0.f;
  } else if (tid < 96) {
    const float2 w = decay_power(g, 32 - lane);
    tail.cw[REV ? 31 - lane : lane] = w.x + w.y;
  } else if (tid < 100) {
    const float2 w = decay_power(g, 32 * (tid - 96));
    tail.p32[tid - 96] = w.x + w.y;
  }
  if (!OUT) decay_dependents();
  if (OUT && p.nseg > 1) decay_wait();

  // This thread's part of the state: column dz of z, entries dx0 .. dx0 + 15.
  const int dz = 32 * (q & 1) + lane, dx0 = 16 * ((q >> 1) * 2 + half);
  const int64_t at = (int64_t)dx0 * p.s_ldx + (int64_t)(z0 + dz) * p.s_ldz;
  float s[16] = {};
  const float* before = !OUT ? nullptr : p.nseg > 1 ? segs + seg * one : p.s_in ? p.s_in + state : nullptr;
  if (before && tid < kWork) read_state(s, before + at, p.s_ldx);
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

  // weights of this thread's rows, by their places in the pass: row t of the
  // outputs, row j of w Y
  const int row = 32 * q + lane, place = REV ? C - 1 - row : row;
  const int qp = REV ? 3 - q : q, lp = REV ? 31 - lane : lane;  // its block and its place in the block
  const float2 w_read = decay_power(g, place + p.e);
  const float read = (w_read.x + w_read.y) * p.read;
  const uint64_t read2 = pair(read, read);
  const float2 w_lane = decay_power(g, lp);
  const float lane_score = (w_lane.x + w_lane.y) * p.score;
  const int j_row = tid & (C - 1), j_place = REV ? C - 1 - j_row : j_row;
  const float2 w_full = decay_power(g, C - j_place - p.e);
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
  // a chunk with rows past a sequence's length: they hold whatever the padding holds
  auto dirty = [&](int c0) { return !REV && valid - c0 < C && begin + valid < p.N; };
  bool ok = true;
  if (warp == kWork / 32) {
    // ------------------------------------------------ issues the products
    constexpr uint32_t id_d = idesc_bf16_f32(128, 128, false, false), id_o = idesc_bf16_f32(128, 64, false, false);
    constexpr uint32_t id_p = idesc_bf16_f32(128, 64, false, true);
    constexpr uint32_t id_u = idesc_bf16_f32(128, 128, true, true), id_l = idesc_bf16_f32(128, 64, true, true);
    const bool leader = elect_one();
    for (int c0 = 0; c0 < valid; c0 += C) {
      const uint32_t st = (uint32_t)(c0 / C) & 1u;
      const uint32_t ya = base + L::y + st * kTile, za = base + L::z + st * kTile;
      const bool more = c0 + C < valid;
      if (leader) {
        ok = mbar_wait(full[st], (uint32_t)(c0 / C >> 1) & 1u, p.err, 0xd06, abort_flag);
        if (OUT) ok = mbar_wait(full_x, st, p.err, 0xd07, abort_flag) && ok;
        if (ok) ++seen, seen_x += OUT;
      }
      if (__syncthreads_or(!ok)) break;
      if (dirty(c0)) __syncthreads();
      if (OUT && leader) {
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
      if (more && leader) {
        // the outputs of the chunk before leave through its y
        if (OUT) ok = mbar_wait(bar_r, st, p.err, 0xd0b, abort_flag);
        fetch(c0 + C);
        if (OUT && !exact) {
          ok = mbar_wait(bar_a, st, p.err, 0xd03, abort_flag) && ok;
          fetch_x(c0 + C);
        }
      }
      __syncwarp();
      if (__syncthreads_or(!ok)) break;
      if (leader) {
        tc_fence_after();
        const uint64_t zd = sdesc_sw128(za, 0u, 1024u);
        const uint64_t wd = sdesc_sw128(ya, base + L::mid - ya, 1024u);
#pragma unroll
        for (int k = 0; k < 8; ++k) umma_bf16(tm, zd + 128 * k, wd + 128 * k, id_u, k > 0);
        if (exact) {  // the third part adds to the second
          const uint64_t ld = sdesc_sw128(base + L::lo, 0u, 1024u);
#pragma unroll
          for (int k = 0; k < 8; ++k) umma_bf16(tm + 64u, zd + 128 * k, ld + 128 * k, id_l, 1u);
        }
        umma_commit(bar_u);
        if (OUT) {
#pragma unroll
          for (int k = 0; k < 8; ++k) umma_tmem_a(tm + kColO, tm + kColP + 8u * k, zd + 128 * k, id_p, 1u);
          umma_commit(bar_b);
        }
      }
      __syncwarp();
      if (OUT && more && exact && leader) {  // x has held the third part of w Y
        ok = mbar_wait(bar_u, st, p.err, 0xd04, abort_flag);
        fetch_x(c0 + C);
      }
      __syncwarp();
    }
    if (leader) {  // after an early end: no copy may land once the CTA is gone
      for (; seen < loaded; ++seen) mbar_wait(full[seen & 1], (uint32_t)(seen >> 1) & 1u, p.err, 0xd08);
      for (; seen_x < loaded_x; ++seen_x) mbar_wait(full_x, (uint32_t)seen_x & 1u, p.err, 0xd09);
    }
    __syncwarp();
  } else {
    for (int c0 = 0; c0 < valid; c0 += C) {
      const int n = min(C, valid - c0);
      const uint32_t st = (uint32_t)(c0 / C) & 1u;
      uint8_t* yt = mem + L::y + st * kTile;
      fence_proxy_async();
      if (__syncthreads_or(!ok)) break;  // the chunk and the state's copy are there
      if (dirty(c0)) {
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        for (int i = n * 8 + tid; i < C * 8; i += kWork) {
          *reinterpret_cast<uint4*>(yt + 16 * i) = zero;
          *reinterpret_cast<uint4*>(mem + L::z + st * kTile + 16 * i) = zero;
          if (OUT) *reinterpret_cast<uint4*>(mem + L::x + 16 * i) = zero;
        }
        fence_proxy_async();
        __syncthreads();
      }
      // half a row of w Y; a tile's pieces are read and written by one thread
      float wj = (w_full.x + w_full.y) * p.update;
      if (n < C) {
        const float2 w = decay_power(g, max(n - j_place - p.e, 0));
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
      auto outputs_read = [&]() {
        if (lane == 0) {
          bulk_wait_read<0>();
          mbar_arrive(bar_r);
        }
        __syncwarp();
      };
      if (OUT && !exact) {  // while the first products still read the rows
        uint4 hi[4];
        split(Two(), [&](int i, uint32_t, uint4 v) { hi[i] = v; });
        outputs_read();
        ok = mbar_wait(bar_a, st, p.err, 0xd01, abort_flag);
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(yt + tile_off<D>(j_row, piece0 + i)) = hi[i];
      } else {
        if (OUT) {
          outputs_read();
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
        const int blocks = qp + 1, middle = (blocks + 1) / 2;
        for (int k = half ? middle : 0; k < (half ? blocks : middle); ++k) {
          const int kc = REV ? 3 - k : k;  // its place among the columns
          tmem_ld32(tmq + 32 * kc, v);
          tmem_wait_ld();
          uint32_t pk[16];
          if (k == qp) {
            // masked entries are dropped by selection: their scores may be infinite
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int d = REV ? i - lane : lane - i;
              v[i] = d >= 0 ? v[i] * tail.tab[31 + d] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = pack2(v[2 * i], v[2 * i + 1]);
          } else {
            const float f = lane_score * tail.p32[qp - k - 1];
            const uint64_t f2 = pair(f, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 c = reinterpret_cast<const float4*>(tail.cw)[i];
              pk[2 * i] = pack2(mul2(mul2(pair(v[4 * i], v[4 * i + 1]), f2), pair(c.x, c.y)));
              pk[2 * i + 1] = pack2(mul2(mul2(pair(v[4 * i + 2], v[4 * i + 3]), f2), pair(c.z, c.w)));
            }
          }
          tmem_st16(tmq + kColP + 16 * kc, pk);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      fence_proxy_async();
      if (__syncthreads_or(!ok)) break;  // P, O and the parts of w Y are there
      ok = mbar_wait(bar_u, st, p.err, 0xd02, abort_flag);
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
        ok = mbar_wait(bar_b, st, p.err, 0xd0a, abort_flag) && ok;
        tc_fence_after();
        float v[32];
        tmem_ld32(tmq + kColO + 32 * half, v);
        tmem_wait_ld();
        // A warp's 32 rows x 64 bytes leave as one TMA store (64-byte swizzle);
        // a part of a chunk row by row, since a store may not start before the
        // sequence or run past its length.
        uint8_t* stage = yt + 2048 * warp;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(stage + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)) =
              make_uint4(pack2(v[8 * i], v[8 * i + 1]), pack2(v[8 * i + 2], v[8 * i + 3]),
                         pack2(v[8 * i + 4], v[8 * i + 5]), pack2(v[8 * i + 6], v[8 * i + 7]));
        const int token = first_token(c0) + 32 * q;
        if (n == C) {
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            tma_store_4d(&a.o.map, smem_u32(stage), z0 + 32 * half, coordinate(a.o, 1, token, h, b),
                         coordinate(a.o, 2, token, h, b), coordinate(a.o, 3, token, h, b));
            bulk_commit();
          }
        } else {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + lane / 4, piece = lane % 4;
            const uint4 t = *reinterpret_cast<const uint4*>(stage + r * 64 + ((piece ^ (r >> 1 & 3)) << 4));
            const int at = 32 * q + r;
            if ((REV ? C - 1 - at : at) < n)
              *reinterpret_cast<uint4*>(o + (int64_t)(token + r) * p.so.token + 32 * half + piece * 8) = t;
          }
        }
        __syncwarp();
      }
      tc_fence_before();
    }
    if (OUT && lane == 0) bulk_wait<0>();
    __syncwarp();
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
  write_state(s, (OUT ? p.s_out + state : segs + (seg + 1) * one) + at, p.s_ldx);
}

// ------------------- the segments' own states, many at once: 64-token chunks

constexpr int kStateChunk = 64;
template <int XB>
constexpr int kStateThreads = 128 * XB;
constexpr uint32_t kStateBlock = kStateChunk * D * 2;
template <int XB, int ZB>  // blocks of 64 entries of a row and of 64 columns of z
struct StateLayout {
  static constexpr uint32_t kY = XB * kStateBlock, kZ = ZB * kStateBlock;
  static constexpr uint32_t y = 0, z = 2 * kY, mid = z + 2 * kZ, lo = mid + kY;
  static constexpr uint32_t tail = lo + kY;
  static constexpr uint32_t bytes = tail + 64;
};
struct StateTail {
  uint64_t bar, full[2];
  uint32_t tmem;
  int abort;
};

// One block of z repeats, so that all 128 lanes of U hold rows.  With 64-entry
// rows U's first part is in columns 0-63 and the others in 64-127, two of them
// in one product; with 128 all parts add to one sum, the small ones first.
template <bool REV, int XB, int ZB>
__global__ void __launch_bounds__(kStateThreads<XB> + 32, XB == 1 ? 4 : 2)
    decay_tc_state_kernel(const __grid_constant__ TcArgs a) {
  static_assert(ZB <= XB, "");
  const DecayPass& p = a.p;
  using L = StateLayout<XB, ZB>;
  constexpr int kStateWork = kStateThreads<XB>;
  constexpr int N = kStateChunk;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* mem = raw + (base - smem_u32(raw));
  StateTail& tail = *reinterpret_cast<StateTail*>(mem + L::tail);

  const int unit = blockIdx.x, seg = blockIdx.y, z0 = blockIdx.z * (ZB * D);
  const int b = unit / p.H, h = unit % p.H;
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid / 32, 0), lane = tid % 32;
  const float g = p.g[h];
  const int length = decay_length(p, b);
  const int begin = seg * p.seg_len;
  const int valid = max(0, min(min(begin + p.seg_len, p.N), length) - begin);
  const bool exact = p.s_out != nullptr;  // three parts where a final state comes of it
  const uint32_t bar = smem_u32(&tail.bar), full[2] = {smem_u32(&tail.full[0]), smem_u32(&tail.full[1])};
  int loaded = 0, seen = 0;
  auto fetch = [&](int c0) {
    const uint32_t st = (uint32_t)(c0 / N) & 1u;
    const int token = REV ? length - begin - c0 - N : begin + c0;
    mbar_arrive_expect_tx(full[st], L::kY + L::kZ);
#pragma unroll
    for (int k = 0; k < XB; ++k) load_rows(base + L::y + st * L::kY + k * kStateBlock, a.y64, full[st], k * D, token, h, b);
#pragma unroll
    for (int k = 0; k < ZB; ++k)
      load_rows(base + L::z + st * L::kZ + k * kStateBlock, a.z64, full[st], z0 + k * D, token, h, b);
    ++loaded;
  };
  if (warp == kStateWork / 32 && elect_one()) {
    mbar_init(bar, 1);
    mbar_init(full[0], 1);
    mbar_init(full[1], 1);
    tail.abort = 0;
    fence_barrier_init();
    if (valid > 0) fetch(0);
  }
  if (warp == kStateWork / 32) {
    __syncwarp();
    tmem_alloc(smem_u32(&tail.tmem), 128);
    tmem_relinquish();
  }
  decay_dependents();
  const int row = tid & (N - 1), place = REV ? N - 1 - row : row;
  const float2 w_full = decay_power(g, N - place - p.e);
  const float2 carry = decay_power(g, N);
  // This thread's part of the state: column dz of z, entries dx0 .. dx0 + E - 1.
  constexpr int E = 32 * ZB;
  const int dz = 32 * (warp & (2 * ZB - 1)) + lane, dx0 = E * (ZB == 1 ? warp >> 1 : warp >> 2);
  float s[E];
#pragma unroll
  for (int i = 0; i < E; ++i) s[i] = 0.f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tail.tmem, tmq = tm + ((uint32_t)(32 * (warp & 3)) << 16);
  volatile int* abort_flag = &tail.abort;
  bool ok = true;
  auto dirty = [&](int c0) { return !REV && valid - c0 < N && begin + valid < p.N; };

  if (warp == kStateWork / 32) {
    constexpr uint32_t id_u = idesc_bf16_f32(128, 128, true, true), id_l = idesc_bf16_f32(128, XB * D, true, true);
    constexpr uint32_t kZStep = ZB == 1 ? 0u : kStateBlock;
    const bool leader = elect_one();
    for (int c0 = 0; c0 < valid; c0 += N) {
      const uint32_t st = (uint32_t)(c0 / N) & 1u;
      const uint32_t ya = base + L::y + st * L::kY, za = base + L::z + st * L::kZ;
      if (leader) {
        ok = mbar_wait(full[st], (uint32_t)(c0 / N >> 1) & 1u, p.err, 0xd0c, abort_flag);
        if (ok) ++seen;
      }
      if (__syncthreads_or(!ok)) break;
      if (dirty(c0)) __syncthreads();
      if (leader && c0 + N < valid) fetch(c0 + N);
      __syncwarp();
      if (__syncthreads_or(0)) break;
      if (leader) {
        tc_fence_after();
        const uint64_t zd = sdesc_sw128(za, kZStep, 1024u), ld = sdesc_sw128(base + L::lo, kStateBlock, 1024u);
        if constexpr (XB == 1) {
          const uint64_t wd = sdesc_sw128(ya, base + L::mid - ya, 1024u);
#pragma unroll
          for (int k = 0; k < N / 16; ++k) umma_bf16(tm, zd + 128 * k, wd + 128 * k, id_u, k > 0);
          if (exact) {  // the third part adds to the second
#pragma unroll
            for (int k = 0; k < N / 16; ++k) umma_bf16(tm + 64u, zd + 128 * k, ld + 128 * k, id_l, 1u);
          }
        } else {
          if (exact) {
#pragma unroll
            for (int k = 0; k < N / 16; ++k) umma_bf16(tm, zd + 128 * k, ld + 128 * k, id_l, k > 0);
          }
          const uint64_t md = sdesc_sw128(base + L::mid, kStateBlock, 1024u), hd = sdesc_sw128(ya, kStateBlock, 1024u);
#pragma unroll
          for (int k = 0; k < N / 16; ++k) umma_bf16(tm, zd + 128 * k, md + 128 * k, id_l, k > 0 || exact);
#pragma unroll
          for (int k = 0; k < N / 16; ++k) umma_bf16(tm, zd + 128 * k, hd + 128 * k, id_l, 1u);
        }
        umma_commit(bar);
      }
      __syncwarp();
    }
    if (leader)
      for (; seen < loaded; ++seen) mbar_wait(full[seen & 1], (uint32_t)(seen >> 1) & 1u, p.err, 0xd0d);
    __syncwarp();
  } else {
    for (int c0 = 0; c0 < valid; c0 += N) {
      const int n = min(N, valid - c0);
      const uint32_t st = (uint32_t)(c0 / N) & 1u;
      uint8_t* yt = mem + L::y + st * L::kY;
      if (__syncthreads_or(!ok)) break;  // the chunk is there
      if (dirty(c0)) {
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        for (int i = n * 8 + tid; i < N * 8; i += kStateWork) {
#pragma unroll
          for (int k = 0; k < XB; ++k) *reinterpret_cast<uint4*>(yt + k * kStateBlock + 16 * i) = zero;
#pragma unroll
          for (int k = 0; k < ZB; ++k)
            *reinterpret_cast<uint4*>(mem + L::z + st * L::kZ + k * kStateBlock + 16 * i) = zero;
        }
        fence_proxy_async();
        __syncthreads();
      }
      float wj = (w_full.x + w_full.y) * p.update;
      if (n < N) {
        const float2 w = decay_power(g, max(n - place - p.e, 0));
        wj = (w.x + w.y) * p.update;
      }
      const uint64_t wj2 = pair(wj, wj);
      auto split = [&](auto parts) {  // 32 entries of a row; the first part takes the row's place
        constexpr int kParts = decltype(parts)::value;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t off = tid / (2 * N) * kStateBlock + tile_off<D>(row, 4 * (tid / N & 1) + i);
          const uint4 v = *reinterpret_cast<const uint4*>(yt + off);
          uint32_t a[kParts], c[kParts], d[kParts], e[kParts];
          scale_split2<kParts>(v.x, wj2, a);
          scale_split2<kParts>(v.y, wj2, c);
          scale_split2<kParts>(v.z, wj2, d);
          scale_split2<kParts>(v.w, wj2, e);
          *reinterpret_cast<uint4*>(yt + off) = make_uint4(a[0], c[0], d[0], e[0]);
          *reinterpret_cast<uint4*>(mem + L::mid + off) = make_uint4(a[1], c[1], d[1], e[1]);
          if constexpr (kParts == 3)
            *reinterpret_cast<uint4*>(mem + L::lo + off) = make_uint4(a[2], c[2], d[2], e[2]);
        }
      };
      if (exact)
        split(std::integral_constant<int, 3>());
      else
        split(std::integral_constant<int, 2>());
      fence_proxy_async();
      if (__syncthreads_or(0)) break;  // the parts of w Y are there
      const float2 w = n == N ? carry : decay_power(g, n);
      ok = mbar_wait(bar, st, p.err, 0xd05, abort_flag);
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < E / 16; ++k) {
        float u0[16], u1[16];
        tmem_ld16(tmq + dx0 + 16 * k, u0);
        if (XB == 1) tmem_ld16(tmq + 64 + dx0 + 16 * k, u1);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float& s0 = s[16 * k + 2 * i];
          float& s1 = s[16 * k + 2 * i + 1];
          uint64_t u = pair(u0[2 * i], u0[2 * i + 1]);
          if (XB == 1) u = add2(u, pair(u1[2 * i], u1[2 * i + 1]));
          const float2 f = unpair(fma2(pair(s0, s1), pair(w.x, w.x), fma2(pair(s0, s1), pair(w.y, w.y), u)));
          s0 = f.x, s1 = f.y;
        }
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == kStateWork / 32) {
    tmem_dealloc(tm, 128);
    return;
  }
  if (valid == 0) return;
  float* to = p.seg + ((int64_t)unit * p.nseg + seg + 1) * (XB * D) * p.DZ;
  write_state(s, to + (int64_t)dx0 * p.s_ldx + (int64_t)(z0 + dz) * p.s_ldz, p.s_ldx);
}

template <bool REV, int XB, int ZB>
cudaError_t states(const TcArgs& a, cudaStream_t s) {
  const DecayPass& p = a.p;
  const unsigned units = (unsigned)(p.B * p.H), slices = (unsigned)(p.DZ / (ZB * D));
  const dim3 grid(units, (unsigned)(p.nseg - 1), slices);
  cudaError_t e;
  auto small_chunks = [&]() {
    constexpr size_t smem = StateLayout<XB, ZB>::bytes + 1024;
    auto* k = decay_tc_state_kernel<REV, XB, ZB>;
    if ((e = room(k, smem)) == cudaSuccess) k<<<grid, kStateThreads<XB> + 32, smem, s>>>(a);
  };
  if constexpr (XB == 1) {
    if ((int64_t)units * (p.nseg - 1) * slices >= 4 * kOpsSms) {
      small_chunks();
    } else {
      constexpr size_t smem = Layout<false>::bytes + 1024;
      auto* k = decay_tc_kernel<false, REV>;
      if ((e = room(k, smem)) == cudaSuccess) k<<<grid, kThreads, smem, s>>>(a);
    }
  } else {
    small_chunks();
  }
  if (e != cudaSuccess || (e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_decay_scan(p, s);
}

template <bool REV>
cudaError_t pass(const TcArgs& a, cudaStream_t s) {
  const DecayPass& p = a.p;
  constexpr size_t smem = Layout<true>::bytes + 1024;
  auto* k = decay_tc_kernel<true, REV>;
  const cudaError_t e = room(k, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(p.B * p.H), (unsigned)p.nseg, (unsigned)(p.DZ / D));
  if (p.nseg > 1) return (cudaError_t)launch_pdl(k, grid, dim3(kThreads), smem, s, a);
  k<<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_tc(const DecayPass& p, cudaStream_t s) {
  TcArgs a;
  a.p = p;
  if (!make_map(&a.x, p.x, p.sx, p.DX, p, D, C, 128) || !make_map(&a.y, p.y, p.sy, p.DX, p, D, C, 128) ||
      !make_map(&a.z, p.z, p.sz, p.DZ, p, D, C, 128) || !make_map(&a.o, p.o, p.so, p.DZ, p, 32, 32, 64) ||
      !make_map(&a.y64, p.y, p.sy, p.DX, p, D, kStateChunk, 128) ||
      !make_map(&a.z64, p.z, p.sz, p.DZ, p, D, kStateChunk, 128))
    return cudaErrorNotSupported;
  const bool wide = p.DX == 2 * D;
  if (p.nseg > 1 && (p.launches & 1)) {
    const cudaError_t e = !wide            ? (p.reverse ? states<true, 1, 1>(a, s) : states<false, 1, 1>(a, s))
                          : p.DZ == 2 * D ? (p.reverse ? states<true, 2, 2>(a, s) : states<false, 2, 2>(a, s))
                                          : (p.reverse ? states<true, 2, 1>(a, s) : states<false, 2, 1>(a, s));
    if (e != cudaSuccess) return e;
  }
  if (!(p.launches & 2)) return cudaSuccess;
  if (wide) return launch_decay_tc_wide(a, s);
  return p.reverse ? pass<true>(a, s) : pass<false>(a, s);
}

}  // namespace mhla
