// Linear attention with a decay for each head on the tensor cores (bf16; see
// decay.h for the pass).
//
// One CTA of four warps per (unit, segment, slice of at most 64 columns of z)
// walks its segment in 64-token chunks; the next chunk's rows arrive by
// asynchronous copies while the current one is worked on.  Per chunk, with
// float32 accumulators throughout:
//   o    = X S                  S in shared memory as bf16, rows scaled by lambda^(i + e)
//   P    = X Y^T                16 x 16 tiles up to the diagonal, decayed and masked in registers
//   o   += P Z                  P goes from accumulator to operand registers
//   U    = (w Y)^T Z            w_j = lambda^(n - j - e), w Y split into two bf16 parts
//   S    = lambda^n S + U       float32 in registers, lambda^n as high + low parts
// Roundings to bf16: P and the operand copy of S once each (relative error at
// most 2^-9 a term, as large as the rounding of the output itself); the state
// sees none: w Y keeps 16 bits as a high + low pair (rms 5e-7 of a term) and U
// starts from zero in every chunk, so the tensor cores' truncating additions
// never run over the long sum.
#include "common.cuh"
#include "decay.h"
#include "ops.h"

namespace mhla {
namespace {

constexpr int C = 64;  // tokens of a chunk
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

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
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two bf16 values times their weights, as sums of three bf16 parts (24 bits).
__device__ __forceinline__ void scale_split(uint32_t v, float w0, float w1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  float a = lo_f(v) * w0, b = hi_f(v) * w1;
  hi = pack2(a, b);
  a -= lo_f(hi), b -= hi_f(hi);
  mid = pack2(a, b);
  lo = pack2(a - lo_f(mid), b - hi_f(mid));
}

template <int DX, int DZS, bool OUT>
struct alignas(16) MmaSmem {
  __nv_bfloat16 x[OUT ? 2 : 1][OUT ? C * DX : 8];
  __nv_bfloat16 y[2][C * DX];
  __nv_bfloat16 z[2][C * DZS];
  __nv_bfloat16 s[OUT ? DX * DZS : 8];
  __nv_bfloat16 o[OUT && DX < DZS ? C * DZS : 8];
  float uw[C];      // weights of the chunk's tokens in the state
  float pw[C + 1];  // lambda^n
};

// A chunk's rows of one tensor into a tile; rows from n on are zeros.
template <int D>
__device__ __forceinline__ void load_tile(__nv_bfloat16* tile, const __nv_bfloat16* first, int64_t step, int n,
                                          bool vec) {
  constexpr int kPieces = D / 8;
  const uint32_t base = smem_addr(tile);
#pragma unroll
  for (int i = threadIdx.x; i < C * kPieces; i += kThreads) {
    const int r = i / kPieces, piece = i % kPieces;
    const __nv_bfloat16* src = first + (r < n ? r * step : 0) + piece * 8;
    const uint32_t dst = base + tile_off<D>(r, piece);
    if (vec) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(r < n ? 16 : 0) : "memory");
    } else {
      alignas(16) __nv_bfloat16 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = r < n ? src[j] : __float2bfloat16_rn(0.f);
      *reinterpret_cast<uint4*>(reinterpret_cast<char*>(tile) + tile_off<D>(r, piece)) = *reinterpret_cast<uint4*>(v);
    }
  }
}

// OUT: the pass itself; otherwise only the segment's own final state.
template <int DX, int DZS, bool OUT>
__global__ void __launch_bounds__(kThreads, DX == 128 ? 2 : 3) decay_mma_kernel(const DecayPass p) {
  extern __shared__ char raw[];
  MmaSmem<DX, DZS, OUT>& sm = *reinterpret_cast<MmaSmem<DX, DZS, OUT>*>(raw);
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

  auto fetch = [&](int c0) {
    const int st = (c0 / C) & 1, n = min(C, valid - c0);
    if (OUT) load_tile<DX>(sm.x[OUT ? st : 0], x + sign * c0 * p.sx.token, sign * p.sx.token, n, vec);
    load_tile<DX>(sm.y[st], y + sign * c0 * p.sy.token, sign * p.sy.token, n, vec);
    load_tile<DZS>(sm.z[st], z + sign * c0 * p.sz.token, sign * p.sz.token, n, vec);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (valid > 0) fetch(0);

  if (tid <= C) {
    const float2 w = decay_power(g, tid);
    sm.pw[tid] = w.x + w.y;
  }
  auto token_weights = [&](int n) {  // of a chunk of n tokens
    if (tid < C) {
      const float2 w = decay_power(g, max(0, n - tid - p.e));
      sm.uw[tid] = (w.x + w.y) * p.update;
    }
  };
  token_weights(min(C, valid));

  // the state before the segment.  s_in may be overwritten by the last
  // segment's CTA, so with several segments the second launch reads the copy
  // that the first one left in the last slot
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
  if (owner && seg == 0 && p.s_in) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
#pragma unroll
      for (int n8 = 0; n8 < 2 * kCols; ++n8)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int2 at = entry(i, n8, r);
          const int64_t slot = (p.nseg - 1) * one + (int64_t)at.x * p.DZ + z0 + at.y;
          if (OUT && p.nseg > 1) {
            s[i][n8][r] = segs[slot];
          } else {
            s[i][n8][r] = p.s_in[state + (int64_t)at.x * p.s_ldx + (int64_t)(z0 + at.y) * p.s_ldz];
            if (!OUT) segs[slot] = s[i][n8][r];
          }
        }
  }
  if (OUT && owner && valid > 0) {
    for (int q = 0; q < seg; ++q) {
      const float2 w = decay_power(g, (seg - 1 - q) * p.seg_len);
      const float* u = segs + q * one + z0;
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
#pragma unroll
        for (int n8 = 0; n8 < 2 * kCols; ++n8)
#pragma unroll
          for (int r = 0; r < 4; r += 2) {
            const int2 at = entry(i, n8, r);
            const float2 v = *reinterpret_cast<const float2*>(u + (int64_t)at.x * p.DZ + at.y);
            s[i][n8][r] = fmaf(v.x, w.x, fmaf(v.x, w.y, s[i][n8][r]));
            s[i][n8][r + 1] = fmaf(v.y, w.x, fmaf(v.y, w.y, s[i][n8][r + 1]));
          }
    }
  }
  auto publish = [&]() {  // the operand copy of the state
    if (!OUT || !owner) return;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
#pragma unroll
      for (int n8 = 0; n8 < 2 * kCols; ++n8)
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          const int2 at = entry(i, n8, r);
          const uint32_t off = tile_off<DZS>(at.x, at.y / 8) + (at.y % 8) * 2;
          *reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(sm.s) + off) = pack2(s[i][n8][r], s[i][n8][r + 1]);
        }
  };
  publish();
  const float2 carry = decay_power(g, C);
  // a state that ends inside this CTA only feeds outputs rounded to bf16
  const bool exact = !OUT || (last && p.s_out);
  __syncthreads();

  // Weights of a warp's 16 output rows: of the state (two rows a thread), of a
  // tile on the diagonal (0 above it) and, for the others, lambda^(16 + t - j)
  // to be multiplied by lambda^(16 (tiles in between)).
  float read0 = 0.f, read1 = 0.f, on[8], off[8];
  if (OUT) {
    read0 = sm.pw[warp * 16 + gr + p.e] * p.read;
    read1 = sm.pw[warp * 16 + gr + 8 + p.e] * p.read;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // entry k: n8 tile k / 4, row half (k / 2) % 2, column k % 2
      const int d = gr + ((k >> 1) & 1) * 8 - ((k >> 2) * 8 + gc + (k & 1));
      on[k] = d >= 0 ? sm.pw[d] * p.score : 0.f;
      off[k] = sm.pw[16 + d] * p.score;
    }
  }
  // addresses inside a 16 x 16 block for ldmatrix: rows are the first 8 / last
  // 8 in lanes 0-7, 16-23 / 8-15, 24-31 for A (and for transposed B), columns
  // the other way round for B
  const int ra = (lane & 7) + ((lane >> 3) & 1) * 8, ca = lane >> 4;
  const int rb = (lane & 7) + (lane >> 4) * 8, cb = (lane >> 3) & 1;

  for (int c0 = 0; c0 < valid; c0 += C) {
    const int n = min(C, valid - c0), st = (c0 / C) & 1;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the chunk's rows and the state's copy are there
    if (c0 + C < valid) fetch(c0 + C);
    const uint32_t ya = smem_addr(sm.y[st]), za = smem_addr(sm.z[st]);
    if (OUT) {
      const uint32_t xa = smem_addr(sm.x[OUT ? st : 0]), sa = smem_addr(sm.s);
      uint32_t xf[kTiles][4];
#pragma unroll
      for (int k = 0; k < kTiles; ++k) ldsm4(xf[k], xa + tile_off<DX>(warp * 16 + ra, 2 * k + ca));
      float acc[2 * kZ16][4];
#pragma unroll
      for (int i = 0; i < 2 * kZ16; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][r] = 0.f;
#pragma unroll
      for (int k = 0; k < kTiles; ++k)
#pragma unroll
        for (int m = 0; m < kZ16; ++m) {
          uint32_t f[4];
          ldsm4t(f, sa + tile_off<DZS>(k * 16 + ra, 2 * m + ca));
          mma(acc[2 * m], xf[k], f[0], f[1]);
          mma(acc[2 * m + 1], xf[k], f[2], f[3]);
        }
#pragma unroll
      for (int i = 0; i < 2 * kZ16; ++i) {
        acc[i][0] *= read0;
        acc[i][1] *= read0;
        acc[i][2] *= read1;
        acc[i][3] *= read1;
      }
      for (int jt = 0; jt <= warp; ++jt) {
        float d[2][4] = {};
#pragma unroll
        for (int k = 0; k < kTiles; ++k) {
          uint32_t f[4];
          ldsm4(f, ya + tile_off<DX>(jt * 16 + rb, 2 * k + cb));
          mma(d[0], xf[k], f[0], f[1]);
          mma(d[1], xf[k], f[2], f[3]);
        }
        uint32_t pf[4];
        if (jt == warp) {
          // masked entries are dropped by selection: their scores may be infinite
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int dist = gr + ((k >> 1) & 1) * 8 - ((k >> 2) * 8 + gc + (k & 1));
            d[k >> 2][k & 3] = dist >= 0 ? d[k >> 2][k & 3] * on[k] : 0.f;
          }
        } else {
          const float f = sm.pw[16 * (warp - jt - 1)];
#pragma unroll
          for (int k = 0; k < 8; ++k) d[k >> 2][k & 3] *= off[k] * f;
        }
        pf[0] = pack2(d[0][0], d[0][1]);
        pf[1] = pack2(d[0][2], d[0][3]);
        pf[2] = pack2(d[1][0], d[1][1]);
        pf[3] = pack2(d[1][2], d[1][3]);
#pragma unroll
        for (int m = 0; m < kZ16; ++m) {
          uint32_t f[4];
          ldsm4t(f, za + tile_off<DZS>(jt * 16 + ra, 2 * m + ca));
          mma(acc[2 * m], pf, f[0], f[1]);
          mma(acc[2 * m + 1], pf, f[2], f[3]);
        }
      }
      // rows to memory through this warp's own rows of a shared tile
      __syncwarp();
      constexpr bool kOwnTile = DX < DZS;
      char* os = reinterpret_cast<char*>(kOwnTile ? sm.o : sm.x[OUT ? st : 0]) + (kOwnTile ? 0 : warp * 16 * (DX - DZS) * 2);
#pragma unroll
      for (int i = 0; i < 2 * kZ16; ++i) {
        *reinterpret_cast<uint32_t*>(os + tile_off<DZS>(warp * 16 + gr, i) + gc * 2) = pack2(acc[i][0], acc[i][1]);
        *reinterpret_cast<uint32_t*>(os + tile_off<DZS>(warp * 16 + gr + 8, i) + gc * 2) = pack2(acc[i][2], acc[i][3]);
      }
      __syncwarp();
      constexpr int kPieces = DZS / 8;
#pragma unroll
      for (int i = lane; i < 16 * kPieces; i += 32) {
        const int r = warp * 16 + i / kPieces, piece = i % kPieces;
        if (r >= n) continue;
        const uint4 v = *reinterpret_cast<const uint4*>(os + tile_off<DZS>(r, piece));
        T* dst = o + decay_token(p, begin + c0 + r, length) * p.so.token + piece * 8;
        if (vec) {
          __stcs(reinterpret_cast<uint4*>(dst), v);
        } else {
          const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
          for (int j = 0; j < 8; ++j) dst[j] = e[j];
        }
      }
    }
    // U of each row tile, then the state
    const float2 w = n == C ? carry : decay_power(g, n);
    if (owner) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        float u[2 * kCols][4];
#pragma unroll
        for (int m = 0; m < 2 * kCols; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) u[m][r] = 0.f;
#pragma unroll
        for (int k = 0; k < C / 16; ++k) {
          uint32_t f[4], hi[4], mid[4], lo[4];
          // (w Y)^T: the transposed load gives rows of x against tokens
          ldsm4t(f, ya + tile_off<DX>(k * 16 + rb, 2 * (own_tile + i * kWarps) + cb));
          const float2 w0 = *reinterpret_cast<const float2*>(&sm.uw[k * 16 + gc]);
          const float2 w1 = *reinterpret_cast<const float2*>(&sm.uw[k * 16 + 8 + gc]);
          scale_split(f[0], w0.x, w0.y, hi[0], mid[0], lo[0]);
          scale_split(f[1], w0.x, w0.y, hi[1], mid[1], lo[1]);
          scale_split(f[2], w1.x, w1.y, hi[2], mid[2], lo[2]);
          scale_split(f[3], w1.x, w1.y, hi[3], mid[3], lo[3]);
          // the parts in turn over all columns: consecutive MMAs never share an
          // accumulator
          uint32_t zf[kCols][4];
#pragma unroll
          for (int m = 0; m < kCols; ++m) ldsm4t(zf[m], za + tile_off<DZS>(k * 16 + ra, 2 * (own_col + m) + ca));
#pragma unroll
          for (int m = 0; m < kCols; ++m) {
            mma(u[2 * m], hi, zf[m][0], zf[m][1]);
            mma(u[2 * m + 1], hi, zf[m][2], zf[m][3]);
          }
#pragma unroll
          for (int m = 0; m < kCols; ++m) {
            mma(u[2 * m], mid, zf[m][0], zf[m][1]);
            mma(u[2 * m + 1], mid, zf[m][2], zf[m][3]);
          }
          if (exact) {
#pragma unroll
            for (int m = 0; m < kCols; ++m) {
              mma(u[2 * m], lo, zf[m][0], zf[m][1]);
              mma(u[2 * m + 1], lo, zf[m][2], zf[m][3]);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < 2 * kCols; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) s[i][m][r] = fmaf(s[i][m][r], w.x, fmaf(s[i][m][r], w.y, u[m][r]));
      }
    }
    __syncthreads();  // every warp has read the chunk and the state's copy
    publish();
    const int rest = valid - c0 - C;
    if (rest > 0 && rest < C) token_weights(rest);
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
        if (OUT)
          p.s_out[state + (int64_t)at.x * p.s_ldx + (int64_t)(z0 + at.y) * p.s_ldz] = s[i][n8][r];
        else
          segs[seg * one + (int64_t)at.x * p.DZ + z0 + at.y] = s[i][n8][r];
      }
}

template <int DX, int DZS>
cudaError_t run(const DecayPass& p, cudaStream_t s) {
  const unsigned units = (unsigned)(p.B * p.H), slices = (unsigned)(p.DZ / DZS);
  cudaError_t e;
  if (p.nseg > 1) {
    constexpr int smem = (int)sizeof(MmaSmem<DX, DZS, false>);
    auto* k = decay_mma_kernel<DX, DZS, false>;
    if (smem > 48 * 1024 &&
        (e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
      return e;
    k<<<dim3(units, (unsigned)(p.nseg - 1), slices), kThreads, smem, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  constexpr int smem = (int)sizeof(MmaSmem<DX, DZS, true>);
  auto* k = decay_mma_kernel<DX, DZS, true>;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
    return e;
  k<<<dim3(units, (unsigned)p.nseg, slices), kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int DX>
cudaError_t run_z(const DecayPass& p, cudaStream_t s) {
  if (p.DZ == 16) return run<DX, 16>(p, s);
  if (p.DZ == 32) return run<DX, 32>(p, s);
  return run<DX, 64>(p, s);
}

}  // namespace

cudaError_t launch_decay_mma(const DecayPass& p, cudaStream_t s) {
  if (p.DX == 16) return run_z<16>(p, s);
  if (p.DX == 32) return run_z<32>(p, s);
  if (p.DX == 64) return run_z<64>(p, s);
  return run_z<128>(p, s);
}

}  // namespace mhla
