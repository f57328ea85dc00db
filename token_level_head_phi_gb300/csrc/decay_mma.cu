// Linear attention with a decay for each head on the tensor cores (bf16; see
// decay.h for the pass).
//
// One CTA of four warps per (unit, segment, slice of at most 64 columns of z;
// 32 with 128-entry rows) walks its segment in 64-token chunks; the next
// chunk's rows arrive by asynchronous copies while the current one is worked
// on.  Per chunk, with float32 accumulators throughout:
//   o    = X S                  S in shared memory as bf16, rows scaled by lambda^(i + e)
//   P    = X Y^T                16 x 16 tiles up to the diagonal, decayed and masked in registers
//   o   += P Z                  P goes from accumulator to operand registers
//   U    = (w Y)^T Z            w_j = lambda^(n - j - e), w Y split into two bf16 parts
//   S    = lambda^n S + U       float32 in registers, lambda^n as high + low parts
// Roundings to bf16: P and the operand copy of S once each (relative error at
// most 2^-8 a term, as large as the rounding of the output itself; 2^-16 for
// prompts shorter than 128 tokens).  w Y is
// held as three bf16 parts (24 bits) where a final state comes of it, so that
// the state is as exact as float32 sums are, and as two (16 bits) where it
// feeds rounded outputs only; U starts from zero in every chunk, so the tensor
// cores' truncating additions never run over the long sum.
// Bound by issue slots: products and the arithmetic around them share them.
// Measured: 32k tokens x 64 heads of 32 / 64 entries 283 us, of 64 414 us, of
// 128 1690 us (the last two run here where rows are not 16-byte aligned).
#include <type_traits>

#include "common.cuh"
#include "decay.h"
#include "decay_tile.cuh"
#include "ops.h"
#include "tc_host.h"

namespace mhla {
namespace {

constexpr int C = 64;  // tokens of a chunk
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The first product of a sum: nothing to add to.
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void stsm4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// Transposes the 4 x 4 words that four neighbouring lanes hold: lane c's word
// i becomes lane i's word c.
__device__ __forceinline__ void quad_transpose(uint32_t (&v)[4], int lane) {
  const bool odd = lane & 1, high = lane & 2;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t t = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], 1);
    if (odd) v[i] = t;
    else v[i + 1] = t;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t t = __shfl_xor_sync(0xffffffffu, high ? v[i] : v[i + 2], 2);
    if (high) v[i] = t;
    else v[i + 2] = t;
  }
}

template <int DX, int DZS, bool OUT, bool FINE>
struct alignas(16) MmaSmem {
  __nv_bfloat16 x[OUT ? C * DX : 8];
  __nv_bfloat16 y[2][C * DX];
  __nv_bfloat16 z[2][C * DZS];
  __nv_bfloat16 s[2][OUT ? DX * DZS : 8];
  __nv_bfloat16 s_lo[2][OUT && FINE ? DX * DZS : 8];
  float4 wt[OUT ? 4 : 1][OUT ? 32 : 1];  // a lane's weights of a 16 x 16 score tile: off (2), on (2) the diagonal
  float uw[2][C];   // weights of the chunk's tokens in the state: full chunks, the last one
  float pw[C + 1];  // lambda^n
};

// OUT: the pass itself; otherwise only the segment's own final state.  FINE:
// P and the operand copy of S keep 16 bits too, as high + low parts.
template <int DX, int DZS, bool OUT, bool FINE>
__global__ void __launch_bounds__(kThreads, 3) decay_mma_kernel(const DecayPass p) {
  extern __shared__ char raw[];
  using Smem = MmaSmem<DX, DZS, OUT, FINE>;
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  // the state's 16-row tiles over the warps; with fewer tiles than warps the
  // columns are shared out too
  constexpr int kTiles = DX / 16;
  constexpr int kOwn = kTiles > kWarps ? kTiles / kWarps : 1;      // row tiles of a warp
  constexpr int kSplit = kTiles < kWarps ? kWarps / kTiles : 1;    // warps that share a row tile
  constexpr int kZ16 = DZS / 16;
  constexpr int kCols = kZ16 >= kSplit ? kZ16 / kSplit : 1;        // 16-column groups of a warp
  using T = __nv_bfloat16;
  const int unit = blockIdx.x, seg = blockIdx.y, z0 = blockIdx.z * DZS;
  const int b = unit / p.H, h = unit % p.H;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int gr = lane / 4, gc = 2 * (lane % 4);  // row and first column of a fragment entry
  const float g = p.g[h];
  const int length = decay_length(p, b);
  const int begin = seg * p.seg_len;
  const int end = min(begin + p.seg_len, p.N);
  const int valid = max(0, min(end, length) - begin);
  const bool last = seg == (length > 0 ? (length - 1) / p.seg_len : 0);
  // the first token's rows and the step to the next token's
  const int t0 = valid > 0 ? decay_token(p, begin, length) : 0;
  const int64_t sign = p.reverse ? -1 : 1;
  const T* x = static_cast<const T*>(p.x) + b * p.sx.batch + h * p.sx.head + t0 * p.sx.token;
  const T* y = static_cast<const T*>(p.y) + b * p.sy.batch + h * p.sy.head + t0 * p.sy.token;
  const T* z = static_cast<const T*>(p.z) + b * p.sz.batch + h * p.sz.head + t0 * p.sz.token + z0;
  T* o = static_cast<T*>(p.o) + b * p.so.batch + h * p.so.head + z0;
  const int64_t one = (int64_t)DX * p.DZ, state = unit * one;
  float* segs = p.seg + (p.nseg > 1 ? (int64_t)unit * p.nseg * one : 0);
  const bool vec = p.vec != 0;

  RowLoader<DX, C, C, kThreads> ly;
  RowLoader<DZS, C, C, kThreads> lz;
  ly.init(y, sign * p.sy.token, 0, tid);
  lz.init(z, sign * p.sz.token, 0, tid);
  auto fetch = [&](int c0) {
    const int st = (c0 / C) & 1, n = min(C, valid - c0);
    ly.load(sm.y[st], n, vec);
    lz.load(sm.z[st], n, vec);
  };
  // x has one buffer: the warp that has read a row tile refills it
  auto fetch_x = [&](int c0, int tile) {
    RowLoader<DX, C, 16, 32> lx;
    lx.init(x + sign * c0 * p.sx.token, sign * p.sx.token, tile * 16, lane);
    lx.load(sm.x, min(C, valid - c0), vec);
  };
  if (valid > 0) {
    fetch(0);
    if (OUT) fetch_x(0, warp);
  }

  if (tid <= C) {
    const float2 w = decay_power(g, tid);
    sm.pw[tid] = w.x + w.y;
  }
  if (tid < C) {
    const int ends[2] = {C, valid % C};  // tokens of a full chunk and of a part of one
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 w = decay_power(g, max(0, ends[i] - tid - p.e));
      sm.uw[i][tid] = (w.x + w.y) * p.update;
    }
  }

  const int own_tile = warp % (kTiles < kWarps ? kTiles : kWarps);
  const int own_col = kSplit > 1 ? (warp / kTiles) * kCols : 0;
  const bool owner = own_col < kZ16;
  float s[kOwn][2 * kCols][4];
  auto entry = [&](int i, int n8, int r) {  // row and column of accumulator entry r
    return make_int2((own_tile + i * kWarps) * 16 + gr + (r >> 1) * 8, own_col * 16 + n8 * 8 + gc + (r & 1));
  };
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
#pragma unroll
    for (int n8 = 0; n8 < 2 * kCols; ++n8)
#pragma unroll
      for (int r = 0; r < 4; ++r) s[i][n8][r] = 0.f;
  if (!OUT) decay_dependents();
  // the state before the segment: the first launch starts every one from zero
  if (OUT && p.nseg > 1) decay_wait();
  const float* before = !OUT ? nullptr : p.nseg > 1 ? segs + seg * one : p.s_in ? p.s_in + state : nullptr;
  if (owner && before) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
#pragma unroll
      for (int n8 = 0; n8 < 2 * kCols; ++n8)
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          const int2 at = entry(i, n8, r);
          const float* f = before + (int64_t)at.x * p.s_ldx + (int64_t)(z0 + at.y) * p.s_ldz;
          const float2 v = p.s_ldz == 1 ? *reinterpret_cast<const float2*>(f) : make_float2(f[0], f[p.s_ldz]);
          s[i][n8][r] = v.x;
          s[i][n8][r + 1] = v.y;
        }
  }
  // addresses inside a 16 x 16 block for ldmatrix / stmatrix: rows are the
  // first 8 / last 8 in lanes 0-7, 16-23 / 8-15, 24-31 for A (and for
  // transposed B and accumulators), columns the other way round for B
  const int ra = (lane & 7) + ((lane >> 3) & 1) * 8, ca = lane >> 4;
  const int rb = (lane & 7) + (lane >> 4) * 8, cb = (lane >> 3) & 1;
  auto publish = [&](int at) {  // an operand copy of the state
    if (!OUT || !owner) return;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
#pragma unroll
      for (int m = 0; m < kCols; ++m) {
        const float(&a)[4] = s[i][2 * m];
        const float(&c)[4] = s[i][2 * m + 1];
        const uint32_t off = tile_off<DZS>((own_tile + i * kWarps) * 16 + ra, 2 * (own_col + m) + ca);
        const uint32_t h[4] = {pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(c[0], c[1]), pack2(c[2], c[3])};
        stsm4(smem_addr(sm.s[at]) + off, h[0], h[1], h[2], h[3]);
        if constexpr (FINE)
          stsm4(smem_addr(sm.s_lo[at]) + off, pack2(a[0] - lo_f(h[0]), a[1] - hi_f(h[0])),
                pack2(a[2] - lo_f(h[1]), a[3] - hi_f(h[1])), pack2(c[0] - lo_f(h[2]), c[1] - hi_f(h[2])),
                pack2(c[2] - lo_f(h[3]), c[3] - hi_f(h[3])));
      }
  };
  publish(0);
  const float2 carry = decay_power(g, C);
  // Where no final state comes of it, a state feeds outputs rounded to bf16
  // only: two parts (16 bits) are plenty.  A final state takes three.
  const bool exact = p.s_out && (!OUT || last);
  __syncthreads();

  // Weights of a score tile's entries, the same for every warp: on the diagonal
  // (0 above it), and lambda^(16 + t - j) for the others, to be multiplied by
  // lambda^(16 (tiles in between)).
  if (OUT) {
    float w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // warp: off, off, on, on; n8 tile warp & 1, row half k / 2, column k & 1
      const int d = gr + (k >> 1) * 8 - ((warp & 1) * 8 + gc + (k & 1));
      w[k] = warp < 2 ? sm.pw[16 + d] * p.score : d >= 0 ? sm.pw[d] * p.score : 0.f;
    }
    sm.wt[OUT ? warp : 0][OUT ? lane : 0] = make_float4(w[0], w[1], w[2], w[3]);
    static_assert(kWarps == 4, "");
  }

  for (int c0 = 0; c0 < valid; c0 += C) {
    const int n = min(C, valid - c0), st = (c0 / C) & 1;
    // The one barrier of a chunk: its rows and the state's copy are there, and
    // the buffers of the chunk before are free.
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // Row tile t has t + 1 score tiles; each warp takes another one in every
    // chunk, so that the four schedulers of an SM get the same work.
    const int rt = (warp + (c0 / C)) % kWarps;
    if (c0 + C < valid) fetch(c0 + C);
    const uint32_t ya = smem_addr(sm.y[st]), za = smem_addr(sm.z[st]);
    if (OUT) {
      const uint32_t xa = smem_addr(sm.x), sa = smem_addr(sm.s[st]);
      uint32_t xf[kTiles][4];
#pragma unroll
      for (int k = 0; k < kTiles; ++k) ldsm4(xf[k], xa + tile_off<DX>(rt * 16 + ra, 2 * k + ca));
      __syncwarp();
      if (c0 + C < valid) fetch_x(c0 + C, rt);
      const float read0 = sm.pw[rt * 16 + gr + p.e] * p.read, read1 = sm.pw[rt * 16 + gr + 8 + p.e] * p.read;
      float acc[2 * kZ16][4];
#pragma unroll
      for (int k = 0; k < kTiles; ++k)
#pragma unroll
        for (int m = 0; m < kZ16; ++m) {
          uint32_t f[4];
          ldsm4t(f, sa + tile_off<DZS>(k * 16 + ra, 2 * m + ca));
          if (k == 0) {
            mma0(acc[2 * m], xf[k], f[0], f[1]);
            mma0(acc[2 * m + 1], xf[k], f[2], f[3]);
          } else {
            mma(acc[2 * m], xf[k], f[0], f[1]);
            mma(acc[2 * m + 1], xf[k], f[2], f[3]);
          }
          if constexpr (FINE) {
            ldsm4t(f, smem_addr(sm.s_lo[st]) + tile_off<DZS>(k * 16 + ra, 2 * m + ca));
            mma(acc[2 * m], xf[k], f[0], f[1]);
            mma(acc[2 * m + 1], xf[k], f[2], f[3]);
          }
        }
#pragma unroll
      for (int i = 0; i < 2 * kZ16; ++i) {
        acc[i][0] *= read0;
        acc[i][1] *= read0;
        acc[i][2] *= read1;
        acc[i][3] *= read1;
      }
      #pragma unroll 2
      for (int jt = 0; jt <= rt; ++jt) {
        float d[2][4];
#pragma unroll
        for (int k = 0; k < kTiles; ++k) {
          uint32_t f[4];
          ldsm4(f, ya + tile_off<DX>(jt * 16 + rb, 2 * k + cb));
          if (k == 0) {
            mma0(d[0], xf[k], f[0], f[1]);
            mma0(d[1], xf[k], f[2], f[3]);
          } else {
            mma(d[0], xf[k], f[0], f[1]);
            mma(d[1], xf[k], f[2], f[3]);
          }
        }
        uint32_t pf[4];
        const int table = jt == rt ? 2 : 0;
        const float4 wa = sm.wt[OUT ? table : 0][OUT ? lane : 0], wb = sm.wt[OUT ? table + 1 : 0][OUT ? lane : 0];
        const float wk[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
        if (jt == rt) {
          // masked entries are dropped by selection: their scores may be infinite
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int dist = gr + ((k >> 1) & 1) * 8 - ((k >> 2) * 8 + gc + (k & 1));
            d[k >> 2][k & 3] = dist >= 0 ? d[k >> 2][k & 3] * wk[k] : 0.f;
          }
        } else {
          const float f = sm.pw[16 * (rt - jt - 1)];
#pragma unroll
          for (int k = 0; k < 8; ++k) d[k >> 2][k & 3] *= wk[k] * f;
        }
        pf[0] = pack2(d[0][0], d[0][1]);
        pf[1] = pack2(d[0][2], d[0][3]);
        pf[2] = pack2(d[1][0], d[1][1]);
        pf[3] = pack2(d[1][2], d[1][3]);
        uint32_t pl[4];
        if constexpr (FINE) {
          pl[0] = pack2(d[0][0] - lo_f(pf[0]), d[0][1] - hi_f(pf[0]));
          pl[1] = pack2(d[0][2] - lo_f(pf[1]), d[0][3] - hi_f(pf[1]));
          pl[2] = pack2(d[1][0] - lo_f(pf[2]), d[1][1] - hi_f(pf[2]));
          pl[3] = pack2(d[1][2] - lo_f(pf[3]), d[1][3] - hi_f(pf[3]));
        }
#pragma unroll
        for (int m = 0; m < kZ16; ++m) {
          uint32_t f[4];
          ldsm4t(f, za + tile_off<DZS>(jt * 16 + ra, 2 * m + ca));
          mma(acc[2 * m], pf, f[0], f[1]);
          mma(acc[2 * m + 1], pf, f[2], f[3]);
          if constexpr (FINE) {
            mma(acc[2 * m], pl, f[0], f[1]);
            mma(acc[2 * m + 1], pl, f[2], f[3]);
          }
        }
      }
      // Rows to memory: four lanes hold two columns each of every 8-column
      // piece of a row; a 4 x 4 exchange gives each lane a whole piece.
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = rt * 16 + gr + half * 8;
        T* row = o + decay_token(p, begin + c0 + r, length) * p.so.token;
#pragma unroll
        for (int q = 0; q < (2 * kZ16 + 3) / 4; ++q) {
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = 4 * q + i < 2 * kZ16 ? pack2(acc[(4 * q + i) % (2 * kZ16)][2 * half], acc[(4 * q + i) % (2 * kZ16)][2 * half + 1]) : 0;
          quad_transpose(v, lane);
          const int piece = 4 * q + (lane & 3);
          if (r >= n || piece >= 2 * kZ16) continue;
          if (vec) {
            __stcs(reinterpret_cast<uint4*>(row + piece * 8), make_uint4(v[0], v[1], v[2], v[3]));
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              row[piece * 8 + 2 * j] = __float2bfloat16_rn(lo_f(v[j]));
              row[piece * 8 + 2 * j + 1] = __float2bfloat16_rn(hi_f(v[j]));
            }
          }
        }
      }
    }
    // U of each row tile, then the state
    const float2 w = n == C ? carry : decay_power(g, n);
    auto update = [&](auto parts) {
      constexpr int kParts = decltype(parts)::value;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        float u[2 * kCols][4];
#pragma unroll
        for (int k = 0; k < C / 16; ++k) {
          uint32_t f[4], wy[4][kParts];
          // (w Y)^T: the transposed load gives rows of x against tokens
          ldsm4t(f, ya + tile_off<DX>(k * 16 + rb, 2 * (own_tile + i * kWarps) + cb));
          const float2 w0 = *reinterpret_cast<const float2*>(&sm.uw[n < C][k * 16 + gc]);
          const float2 w1 = *reinterpret_cast<const float2*>(&sm.uw[n < C][k * 16 + 8 + gc]);
          scale_split<kParts>(f[0], w0.x, w0.y, wy[0]);
          scale_split<kParts>(f[1], w0.x, w0.y, wy[1]);
          scale_split<kParts>(f[2], w1.x, w1.y, wy[2]);
          scale_split<kParts>(f[3], w1.x, w1.y, wy[3]);
          // 32 columns at a time, the parts in turn over all of them, so that
          // consecutive MMAs do not share an accumulator
          constexpr int kHalf = kCols > 2 ? 2 : kCols;
#pragma unroll
          for (int m0 = 0; m0 < kCols; m0 += kHalf) {
            uint32_t zf[kHalf][4];
#pragma unroll
            for (int m = 0; m < kHalf; ++m)
              ldsm4t(zf[m], za + tile_off<DZS>(k * 16 + ra, 2 * (own_col + m0 + m) + ca));
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
              const uint32_t part[4] = {wy[0][q], wy[1][q], wy[2][q], wy[3][q]};
#pragma unroll
              for (int m = 0; m < kHalf; ++m) {
                if (k == 0 && q == 0) {
                  mma0(u[2 * (m0 + m)], part, zf[m][0], zf[m][1]);
                  mma0(u[2 * (m0 + m) + 1], part, zf[m][2], zf[m][3]);
                } else {
                  mma(u[2 * (m0 + m)], part, zf[m][0], zf[m][1]);
                  mma(u[2 * (m0 + m) + 1], part, zf[m][2], zf[m][3]);
                }
              }
            }
          }
        }
#pragma unroll
        for (int m = 0; m < 2 * kCols; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) s[i][m][r] = fmaf(s[i][m][r], w.x, fmaf(s[i][m][r], w.y, u[m][r]));
      }
    };
    if (owner) {
      if (exact)
        update(std::integral_constant<int, 3>());
      else
        update(std::integral_constant<int, 2>());
    }
    publish(st ^ 1);
  }

  if (OUT) {
    for (int i = tid; i < (end - begin - valid) * DZS; i += kThreads)
      o[(int64_t)(begin + valid + i / DZS) * p.so.token + i % DZS] = __float2bfloat16_rn(0.f);
    if (!last || !p.s_out) return;
  } else if (valid == 0) {
    return;
  }
  if (!owner) return;
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
#pragma unroll
    for (int n8 = 0; n8 < 2 * kCols; ++n8)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int2 at = entry(i, n8, r);
        const int64_t in = (int64_t)at.x * p.s_ldx + (int64_t)(z0 + at.y) * p.s_ldz;
        if (OUT)
          p.s_out[state + in] = s[i][n8][r];
        else
          segs[(seg + 1) * one + in] = s[i][n8][r];
      }
}

template <int DX, int DZS, bool OUT, bool FINE>
cudaError_t launch(const DecayPass& p, int segments, bool dependent, cudaStream_t s) {
  constexpr int smem = (int)sizeof(MmaSmem<DX, DZS, OUT, FINE>);
  auto* k = decay_mma_kernel<DX, DZS, OUT, FINE>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((unsigned)(p.B * p.H), (unsigned)segments, (unsigned)(p.DZ / DZS));
  if (dependent) return (cudaError_t)launch_pdl(k, grid, dim3(kThreads), smem, s, p);
  k<<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int DX, int DZS>
cudaError_t run(const DecayPass& p, cudaStream_t s) {
  cudaError_t e;
  if (p.nseg > 1 && (p.launches & 1)) {
    if ((e = launch<DX, DZS, false, false>(p, p.nseg - 1, false, s)) != cudaSuccess) return e;
    if ((e = launch_decay_scan(p, s)) != cudaSuccess) return e;
  }
  if (!(p.launches & 2)) return cudaSuccess;
  // Two roundings as large as the output's own make its error 1.4 times one
  // rounding, on average; over the few outputs of a short prompt the average
  // says little, and the 16-bit operands cost nothing that shows there.  The
  // tokens of the call decide, padding included: a sequence's own length is on
  // the device, and the tcgen05 kernels, as laid out, have no place for the low
  // parts (tensor memory is full; the 128-entry rows fill shared memory too).
  if (p.N < 128) return launch<DX, DZS, true, true>(p, p.nseg, p.nseg > 1, s);
  return launch<DX, DZS, true, false>(p, p.nseg, p.nseg > 1, s);
}

template <int DX>
cudaError_t run_z(const DecayPass& p, cudaStream_t s) {
  if (p.DZ == 16) return run<DX, 16>(p, s);
  if (p.DZ == 32) return run<DX, 32>(p, s);
  // rows of 128: with 64 columns a warp holds 128 registers of state, two CTAs
  // fit an SM, and 2k tokens x 60 ragged heads take 105 us; with 32 columns the
  // scores are formed twice as often, three CTAs fit, and it is 88 us
  if constexpr (DX == 128) return run<DX, 32>(p, s);
  else return run<DX, 64>(p, s);
}

}  // namespace

cudaError_t launch_decay_mma(const DecayPass& p, cudaStream_t s) {
  if (p.DX == 16) return run_z<16>(p, s);
  if (p.DX == 32) return run_z<32>(p, s);
  if (p.DX == 64) return run_z<64>(p, s);
  return run_z<128>(p, s);
}

}  // namespace mhla
