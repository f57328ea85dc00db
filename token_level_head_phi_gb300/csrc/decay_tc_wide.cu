// Linear attention with a decay for each head on the fifth-generation tensor
// cores, rows of 128 entries (bf16, 16-byte aligned; see decay.h for the pass
// and decay_tc.cu for the steps of a 128-token chunk and their roundings).
//
// Operands of that size leave room for one CTA an SM, so that nothing fills
// the waits of a chain of steps.  Two groups of eight warps take turns with the
// tensor cores instead:
//   outputs: D = X Y^T is there -> P decayed and masked, in the place of D
//            O = X S and P Z are there -> lambda^(t + e) O + P Z to memory
//   states:  Y is there and D has been formed -> parts of w Y, over Y and beside it
//            U = Z^T [w Y] is there -> S = lambda^n S + U, published as bf16
// and one thread loads (TMA) and issues X S, P Z, U and the next chunk's D as
// their operands come.  Every hand-over is an mbarrier.
//
// Columns of tensor memory: D and P 0-127, U 128-255, O of X S from 256, O of
// P Z behind it.  U adds the parts of w Y to one sum, the small ones first.
//
// Measured: 32k tokens x 64 heads of 128 621 us (pass, states and scan; the
// chain of one group of warps 764, products issued by `lane == 0` 678), 60
// heads of 2k tokens 54 us in slices of 64 columns.  A 128-token chunk of 128
// columns takes 6000 cycles, its transfers through shared memory about 4600:
// that bounds it, then the hand-overs between the groups.
#include <type_traits>

#include "decay_tc.cuh"
#include "decay_tile.cuh"
#include "ops.h"

namespace mhla {
namespace {

constexpr int C = 128;   // tokens of a chunk
constexpr int D = 64;    // entries of a block of 128-byte rows
constexpr int DX = 128;  // entries of a row of x and y
constexpr int kGroup = 256, kWork = 2 * kGroup, kThreads = kWork + 32;
constexpr uint32_t kBlock = C * D * 2;
constexpr uint32_t kColU = 128, kColO = 256;

// ZB blocks of 64 columns of z.  The third part of w Y and the outputs on their
// way to memory have places of their own with one block; with two, the third
// part takes the place of s once X S is formed, and the outputs that of y.
template <int ZB>
struct Layout {
  static constexpr bool own = ZB == 1;
  static constexpr uint32_t kY = 2 * kBlock, kZ = ZB * kBlock, kS = ZB * D * DX * 2;
  static constexpr uint32_t y = 0, z = 2 * kY, mid = z + 2 * kZ, x = mid + kY, s = x + kY;
  static constexpr uint32_t lo = own ? s + kS : s, stage = lo + kY;
  static constexpr uint32_t tail = own ? stage + kZ : s + kS;
  static constexpr uint32_t bytes = tail + 1024;
};
enum Bar { kD, kA, kU, kB, kP, kO, kW, kS, kR, kX, kFull, kBars = kFull + 2 };
struct alignas(16) Tail {
  float tab[64];  // lambda^d of the diagonal block at 31 + d, 0 for d < 0
  float cw[32];   // lambda^(32 - j), reversed for REV
  float p32[4];   // lambda^(32 m)
  uint64_t bar[kBars];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Tail) <= 1024, "");

template <bool REV, int ZB>
__global__ void __launch_bounds__(kThreads, 1) decay_tc_wide_kernel(const __grid_constant__ TcArgs a) {
  const DecayPass& p = a.p;
  using L = Layout<ZB>;
  constexpr int DZ = ZB * D;
  constexpr uint32_t kColZ = kColO + DZ;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* mem = raw + (base - smem_u32(raw));
  Tail& tail = *reinterpret_cast<Tail*>(mem + L::tail);

  const int unit = blockIdx.x, seg = blockIdx.y, z0 = blockIdx.z * DZ;
  const int b = unit / p.H, h = unit % p.H;
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid / 32, 0), lane = tid % 32;
  const int q = warp & 3, half = (warp >> 2) & 1;  // lanes 32 q .. of tensor memory, half of the columns
  const bool outputs = warp < kGroup / 32, issues = warp == kWork / 32;
  const float g = p.g[h];
  const int length = decay_length(p, b);
  const int begin = seg * p.seg_len;
  const int end = min(begin + p.seg_len, p.N);
  const int valid = max(0, min(end, length) - begin);
  const bool last = seg == (length > 0 ? (length - 1) / p.seg_len : 0);
  const bool exact = p.s_out && last;  // three parts where a final state comes of it
  auto first_token = [&](int c0) { return REV ? length - begin - c0 - C : begin + c0; };  // of row 0
  // a chunk with rows past a sequence's length: they hold whatever the padding holds
  auto dirty = [&](int c0) { return !REV && valid - c0 < C && begin + valid < p.N; };
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + b * p.so.batch + h * p.so.head + z0;
  const int64_t one = (int64_t)DX * p.DZ;
  const float* segs = p.seg + (p.nseg > 1 ? ((int64_t)unit * p.nseg + seg) * one : 0);

  volatile int* abort_flag = &tail.abort;
  auto bar = [&](int i) { return smem_u32(&tail.bar[i]); };
  // waits for the i-th completion of a barrier
  auto wait = [&](int which, int i) {
    return mbar_wait(bar(which), (uint32_t)i & 1u, p.err, 0xd20u + (uint32_t)which, abort_flag);
  };
  auto wait_rows = [&](int i) {
    return mbar_wait(bar(kFull + (i & 1)), (uint32_t)i >> 1 & 1u, p.err, 0xd30u, abort_flag);
  };
  auto arrive = [&](int which) {  // once a warp, after all its lanes
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(which));
  };
  int loaded = 0, loaded_x = 0, seen = 0, seen_x = 0;  // chunks asked for, and waited for
  auto fetch = [&](int c0) {
    const uint32_t st = (uint32_t)(c0 / C) & 1u, full = bar(kFull + (int)st);
    mbar_arrive_expect_tx(full, L::kY + L::kZ);
    for (int k = 0; k < 2; ++k) load_rows(base + L::y + st * L::kY + k * kBlock, a.y, full, k * D, first_token(c0), h, b);
    for (int k = 0; k < ZB; ++k)
      load_rows(base + L::z + st * L::kZ + k * kBlock, a.z, full, z0 + k * D, first_token(c0), h, b);
    ++loaded;
  };
  auto fetch_x = [&](int c0) {
    mbar_arrive_expect_tx(bar(kX), L::kY);
    for (int k = 0; k < 2; ++k) load_rows(base + L::x + k * kBlock, a.x, bar(kX), k * D, first_token(c0), h, b);
    ++loaded_x;
  };
  if (issues && elect_one()) {
    for (int i = 0; i < kBars; ++i)
      mbar_init(bar(i), i == kP || i == kO || i == kW || i == kS || i == kR ? kGroup / 32 : 1);
    tail.abort = 0;
    fence_barrier_init();
    if (valid > 0) {
      fetch(0);
      fetch_x(0);
    }
  }
  if (issues) {
    __syncwarp();
    tmem_alloc(smem_u32(&tail.tmem), 512);
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
  if (p.nseg > 1) decay_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tail.tmem, tmq = tm + ((uint32_t)(32 * q) << 16);

  bool ok = true;
  if (issues) {
    // ------------------------------------------------ loads and issues
    constexpr uint32_t id_d = idesc_bf16_f32(128, 128, false, false), id_o = idesc_bf16_f32(128, DZ, false, false);
    constexpr uint32_t id_p = idesc_bf16_f32(128, DZ, false, true), id_u = idesc_bf16_f32(128, 128, true, true);
    // from one block of 64 columns of z to the next; a single one repeats, so
    // that all lanes of U hold rows
    constexpr uint32_t kZStep = ZB == 1 ? 0u : kBlock;
    if (elect_one()) {
      const uint64_t xd = sdesc_sw128(base + L::x, 0u, 1024u), sd = sdesc_sw128(base + L::s, 0u, 1024u);
      auto scores = [&](int c0) {
        const int i = c0 / C;
        ok = wait_rows(i) && ok;
        seen += ok;
        ok = ok && wait(kX, i);
        seen_x += ok;
        if (i > 0) ok = ok && wait(kB, i - 1);  // P before has been read
        if (!ok) return;
        tc_fence_after();
        const uint64_t yd = sdesc_sw128(base + L::y + (uint32_t)(i & 1) * L::kY, 0u, 1024u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t at = (k / 4) * (kBlock / 16) + 2 * (k % 4);
          umma_bf16(tm, xd + at, yd + at, id_d, k > 0);
        }
        umma_commit(bar(kD));
      };
      if (valid > 0) scores(0);
      for (int c0 = 0; ok && c0 < valid; c0 += C) {
        const int i = c0 / C, st = i & 1;
        const uint32_t ya = base + L::y + (uint32_t)st * L::kY;
        const bool more = c0 + C < valid;
        if (i > 0) ok = wait(kO, i - 1);
        if (!(ok = ok && wait(kS, i))) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_bf16(tm + kColO, xd + (k / 4) * (kBlock / 16) + 2 * (k % 4), sd + (k / 4) * (L::kS / 32) + 2 * (k % 4),
                    id_o, k > 0);
        umma_commit(bar(kA));
        if (more) {
          // y of the chunk before has been read, the outputs in its place included
          if (i > 0) ok = L::own ? wait(kU, i - 1) : wait(kR, i - 1);
          if (!ok) break;
          fetch(c0 + C);
          if (!(ok = wait(kA, i))) break;
          fetch_x(c0 + C);
        }
        ok = wait(kP, i);
        if (dirty(c0)) ok = ok && wait(kW, i);  // rows of z are cleared
        if (!ok) break;
        tc_fence_after();
        const uint64_t zd = sdesc_sw128(base + L::z + (uint32_t)st * L::kZ, kBlock, 1024u);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_tmem_a(tm + kColZ, tm + 32u * (k / 2) + 8u * (k % 2), zd + 128 * k, id_p, k > 0);
        umma_commit(bar(kB));
        if (!(ok = wait(kW, i))) break;
        tc_fence_after();
        const uint64_t td = sdesc_sw128(base + L::z + (uint32_t)st * L::kZ, kZStep, 1024u);
        if (exact) {
          const uint64_t ld = sdesc_sw128(base + L::lo, kBlock, 1024u);
#pragma unroll
          for (int k = 0; k < 8; ++k) umma_bf16(tm + kColU, td + 128 * k, ld + 128 * k, id_u, k > 0);
        }
        const uint64_t md = sdesc_sw128(base + L::mid, kBlock, 1024u), hd = sdesc_sw128(ya, kBlock, 1024u);
#pragma unroll
        for (int k = 0; k < 8; ++k) umma_bf16(tm + kColU, td + 128 * k, md + 128 * k, id_u, k > 0 || exact);
#pragma unroll
        for (int k = 0; k < 8; ++k) umma_bf16(tm + kColU, td + 128 * k, hd + 128 * k, id_u, 1u);
        umma_commit(bar(kU));
        if (more) scores(c0 + C);  // runs under this chunk's last steps
      }
      // after an early end: no copy may land once the CTA is gone
      for (; seen < loaded; ++seen) mbar_wait(bar(kFull + (seen & 1)), (uint32_t)seen >> 1 & 1u, p.err, 0xd31);
      for (; seen_x < loaded_x; ++seen_x) mbar_wait(bar(kX), (uint32_t)seen_x & 1u, p.err, 0xd32);
    }
    __syncwarp();
  } else if (outputs) {
    // ------------------------------------------------ scores and outputs
    // weights of this thread's row t, by its place in the pass
    const int place = REV ? C - 1 - 32 * q - lane : 32 * q + lane;
    const int qp = REV ? 3 - q : q, lp = REV ? 31 - lane : lane;  // its block and its place in the block
    const float2 w_read = decay_power(g, place + p.e);
    const float read = (w_read.x + w_read.y) * p.read;
    const uint64_t read2 = pair(read, read);
    const float2 w_lane = decay_power(g, lp);
    const float lane_score = (w_lane.x + w_lane.y) * p.score;
    for (int c0 = 0; c0 < valid; c0 += C) {
      const int i = c0 / C, n = min(C, valid - c0);
      if (!(ok = wait(kD, i))) break;
      tc_fence_after();
      if (!L::own && i > 0) {
        if (lane == 0) bulk_wait_read<0>();
        arrive(kR);
      }
      // P in blocks of 32 columns, each in the place of its scores
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int k = 2 * m + half;      // place among the columns
        const int kp = REV ? 3 - k : k;  // and in the pass
        uint32_t pk[16];
        if (kp > qp) {
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = 0u;
        } else {
          float v[32];
          tmem_ld32(tmq + 32 * k, v);
          tmem_wait_ld();
          if (kp == qp) {
            // masked entries are dropped by selection: their scores may be infinite
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int d = REV ? j - lane : lane - j;
              v[j] = d >= 0 ? v[j] * tail.tab[31 + d] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) pk[j] = pack2(v[2 * j], v[2 * j + 1]);
          } else {
            const float f = lane_score * tail.p32[qp - kp - 1];
            const uint64_t f2 = pair(f, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 c = reinterpret_cast<const float4*>(tail.cw)[j];
              pk[2 * j] = pack2(mul2(mul2(pair(v[4 * j], v[4 * j + 1]), f2), pair(c.x, c.y)));
              pk[2 * j + 1] = pack2(mul2(mul2(pair(v[4 * j + 2], v[4 * j + 3]), f2), pair(c.z, c.w)));
            }
          }
        }
        tmem_st16(tmq + 32 * k, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      arrive(kP);

      if (!(ok = wait(kB, i))) break;  // X S is older
      tc_fence_after();
      uint32_t out[16 * ZB];
#pragma unroll
      for (int m = 0; m < ZB; ++m) {
        const int col = 32 * (2 * m + half);
        float v[32];
        tmem_ld32(tmq + kColZ + col, v);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float t[16];
          tmem_ld16(tmq + kColO + col + 16 * k, t);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; j += 2)
            out[16 * m + 8 * k + j / 2] = pack2(fma2(pair(t[j], t[j + 1]), read2, pair(v[16 * k + j], v[16 * k + j + 1])));
        }
      }
      tc_fence_before();
      arrive(kO);
      uint8_t* stage = mem + (L::own ? L::stage : L::y + (uint32_t)(i & 1) * L::kY) + 2048 * ZB * warp;
      if (L::own) {
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
      } else if (!(ok = wait(kU, i))) {
        break;
      }
      // A warp's 32 rows x 64 bytes leave as one TMA store (64-byte swizzle);
      // a part of a chunk row by row, since a store may not start before the
      // sequence or run past its length.
      const int token = first_token(c0) + 32 * q;
#pragma unroll
      for (int m = 0; m < ZB; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(stage + 2048 * m + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)) =
              make_uint4(out[16 * m + 4 * j], out[16 * m + 4 * j + 1], out[16 * m + 4 * j + 2], out[16 * m + 4 * j + 3]);
      if (n == C) {
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int m = 0; m < ZB; ++m)
            tma_store_4d(&a.o.map, smem_u32(stage + 2048 * m), z0 + 32 * (2 * m + half),
                         coordinate(a.o, 1, token, h, b), coordinate(a.o, 2, token, h, b),
                         coordinate(a.o, 3, token, h, b));
          bulk_commit();
        }
      } else {
        __syncwarp();
#pragma unroll
        for (int m = 0; m < ZB; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 8 * j + lane / 4, piece = lane % 4;
            const uint4 t = *reinterpret_cast<const uint4*>(stage + 2048 * m + r * 64 + ((piece ^ (r >> 1 & 3)) << 4));
            const int at = 32 * q + r;
            if ((REV ? C - 1 - at : at) < n)
              *reinterpret_cast<uint4*>(o + (int64_t)(token + r) * p.so.token + 32 * (2 * m + half) + piece * 8) = t;
          }
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
  } else {
    // ------------------------------------------------ parts of w Y and states
    // This thread's part of the state: column dz of z, entries dx0 .. dx0 + E - 1.
    constexpr int E = 32 * ZB;
    const int dz = ZB == 1 ? 32 * (q & 1) + lane : 32 * q + lane;
    const int dx0 = ZB == 1 ? E * ((q >> 1) * 2 + half) : E * half;
    const int64_t at = (int64_t)dx0 * p.s_ldx + (int64_t)(z0 + dz) * p.s_ldz;
    float s[E] = {};
    const float* before = p.nseg > 1 ? segs : p.s_in ? p.s_in + unit * one : nullptr;
    if (before) read_state(s, before + at, p.s_ldx);
    auto publish = [&]() {  // S as the second operand of X S: row dz, its entries along the row
      uint8_t* to = mem + L::s + (dx0 / D) * (L::kS / 2);
#pragma unroll
      for (int i = 0; i < E / 8; ++i)
        *reinterpret_cast<uint4*>(to + tile_off<D>(dz, dx0 % D / 8 + i)) =
            make_uint4(pack2(s[8 * i], s[8 * i + 1]), pack2(s[8 * i + 2], s[8 * i + 3]),
                       pack2(s[8 * i + 4], s[8 * i + 5]), pack2(s[8 * i + 6], s[8 * i + 7]));
      fence_proxy_async();
      arrive(kS);
    };
    publish();
    // row j of w Y, its weight by its place in the pass
    const int j_row = tid & (C - 1), j_place = REV ? C - 1 - j_row : j_row;
    const uint32_t block0 = (uint32_t)half * kBlock;
    const float2 w_full = decay_power(g, C - j_place - p.e);
    const float2 carry = decay_power(g, C);
    for (int c0 = 0; c0 < valid; c0 += C) {
      const int i = c0 / C, n = min(C, valid - c0), st = i & 1;
      uint8_t* yt = mem + L::y + (uint32_t)st * L::kY + block0;
      const bool clear = dirty(c0);
      float wj = (w_full.x + w_full.y) * p.update;
      float2 w = carry;
      if (n < C) {
        const float2 wp = decay_power(g, max(n - j_place - p.e, 0));
        wj = (wp.x + wp.y) * p.update;
        w = decay_power(g, n);
      }
      const uint64_t wj2 = pair(wj, wj);
      ok = wait_rows(i) && wait(kD, i);             // y is read and free
      if (exact && !L::own) ok = ok && wait(kA, i);  // and s
      if (!ok) break;
      if (clear) {
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        for (int m = n * 8 + tid - kGroup; m < C * 8; m += kGroup)
#pragma unroll
          for (int k = 0; k < ZB; ++k)
            *reinterpret_cast<uint4*>(mem + L::z + (uint32_t)st * L::kZ + k * kBlock + 16 * m) = zero;
      }
      auto split = [&](auto parts) {  // the first part takes the row's place
        constexpr int kParts = decltype(parts)::value;
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const uint32_t off = tile_off<D>(j_row, m);
          uint4 v = *reinterpret_cast<const uint4*>(yt + off);
          if (clear && j_row >= n) v = make_uint4(0u, 0u, 0u, 0u);
          uint32_t a[kParts], c[kParts], d[kParts], e[kParts];
          scale_split2<kParts>(v.x, wj2, a);
          scale_split2<kParts>(v.y, wj2, c);
          scale_split2<kParts>(v.z, wj2, d);
          scale_split2<kParts>(v.w, wj2, e);
          *reinterpret_cast<uint4*>(yt + off) = make_uint4(a[0], c[0], d[0], e[0]);
          *reinterpret_cast<uint4*>(mem + L::mid + block0 + off) = make_uint4(a[1], c[1], d[1], e[1]);
          if constexpr (kParts == 3)
            *reinterpret_cast<uint4*>(mem + L::lo + block0 + off) = make_uint4(a[2], c[2], d[2], e[2]);
        }
      };
      if (exact)
        split(std::integral_constant<int, 3>());
      else
        split(std::integral_constant<int, 2>());
      fence_proxy_async();
      tc_fence_before();
      arrive(kW);
      if (!(ok = wait(kU, i))) break;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < E / 16; ++k) {
        float u[16];
        tmem_ld16(tmq + kColU + dx0 + 16 * k, u);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          float& s0 = s[16 * k + j];
          float& s1 = s[16 * k + j + 1];
          const float2 f =
              unpair(fma2(pair(s0, s1), pair(w.x, w.x), fma2(pair(s0, s1), pair(w.y, w.y), pair(u[j], u[j + 1]))));
          s0 = f.x, s1 = f.y;
        }
      }
      if (c0 + C < valid) publish();
    }
    if (last && p.s_out) write_state(s, p.s_out + unit * one + at, p.s_ldx);
    tc_fence_before();
  }

  __syncthreads();
  if (issues) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
    return;
  }
  for (int i = tid; i < (end - begin - valid) * DZ; i += kWork)
    o[(int64_t)(begin + valid + i / DZ) * p.so.token + i % DZ] = __float2bfloat16_rn(0.f);
}

template <bool REV, int ZB>
cudaError_t run(const TcArgs& a, cudaStream_t s) {
  const DecayPass& p = a.p;
  constexpr size_t smem = Layout<ZB>::bytes + 1024;
  static_assert(smem <= 232448, "");
  auto* k = decay_tc_wide_kernel<REV, ZB>;
  const cudaError_t e = room(k, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(p.B * p.H), (unsigned)p.nseg, (unsigned)(p.DZ / (ZB * D)));
  if (p.nseg > 1) return (cudaError_t)launch_pdl(k, grid, dim3(kThreads), smem, s, a);
  k<<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_tc_wide(const TcArgs& a, cudaStream_t s) {
  if (a.p.slice == 2 * D) return a.p.reverse ? run<true, 2>(a, s) : run<false, 2>(a, s);
  return a.p.reverse ? run<true, 1>(a, s) : run<false, 1>(a, s);
}

}  // namespace mhla
