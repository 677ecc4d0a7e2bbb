// sekv_states_logprobs, sekv_states_surprisal and sekv_states_logprobs_backward: log-probabilities
// of tokens from a model's last states h_r and its vocabulary matrix w_v, and their gradient,
// without the logits.
//
// With x_rv = scale h_r . w_v:
//   lse_r = ln sum_v e^(x_rv),  logprob_r = x_r,tok - lse_r
//   gradient of sum_r g_r logprob_r + e_r lse_r:
//     G_rv = scale ((e_r - g_r) e^(x_rv - lse_r) + g_r [v = tok_r]),  dh = G W,  dw = G^T H
// All three products run on the fifth generation's tensor cores, 16-bit operands, fp32 sums.  A
// tile of logits lives in tensor memory only: the loss keeps a maximum and a sum of each row and
// half tile, the gradient a tile of G as 16-bit numbers, for one piece of the vocabulary at a time,
// which the other two products read.  G is written once and read twice, across K in the second product
// (dW), so that no transposed copy is made.  Its rounding to 16 bits adds to that of the results
// (a mean over 96 to 1024 rows: errors 1.02 to 1.04 times those of rounding the results alone in bf16, 1.06 to 1.09 in
// f16); two numbers for G would remove that and double both products.
//
// One kernel does all: a pair of CTAs takes 256 x 256 tiles (each brings half of both operands, so that an
// operand byte is read from L2 for 256 products, not 128), one CTA 128 x 256 where there are up to 128 rows.
// What bounds it: with many rows the tensor cores, or the power that they draw (4096 x 128000 x 4096: loss 2.1 ms,
// 2.0 PFLOP/s, beside 2.05 ms of a library product of the same sizes that only makes the logits;
// gradient 7.3 ms, 1.77 PFLOP/s; 1024 x 32000 x 4096, each product 146 to 166 us, tensor pipe 69 to 83% busy); with few
// the weight's bytes (128 x 128000 x 4096: 170 us, 6.2 TB/s; 1 x 32000 x 4096: 48 us, 5.5 TB/s, 9 us above the
// bytes' time).  Rows whose length is no multiple of 128 bytes may cost as much again (1003 x 50021 x 1000 in f16: 97 us,
// with rows 1024 elements apart 69), or nothing (1021 x 50021 x 2000: 131 and 136 us).
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include <algorithm>

#include "decode_host.h"
#include "host_common.h"
#include "tc.cuh"

using namespace sekv;

namespace {

constexpr int kRowsOfCta = 128;  // lanes of tensor memory
constexpr int kBlockK = 64;      // 128 bytes of an operand's row
constexpr int kColumns = 256;    // of an accumulator; two of them fill tensor memory
constexpr int kBytesA = kRowsOfCta * kBlockK * 2;
constexpr int kEpilogueWarps = 8;  // two for each 32 lanes, half of the columns each
constexpr int kHalf = kColumns / 2;
// Blocks of K that one accumulator sums, of the logits and of the products with G.  The tensor cores cut their sums off
// towards zero, and what is added outside is rounded properly: in 256 additions (K 4096) 1.8e-6 of lse, after each 1024 of
// K 4e-7.  The products' results are rounded to 16 bits; terms of one sign were off by 3.9e-4 with K 60000 (f16 rounds
// by 2.0e-4 in the mean square), after each 4096 of K by 2.4e-5.
constexpr int kSegmentLogits = 16, kSegmentProduct = 64;
constexpr int kTileThreads = (kEpilogueWarps + 2) * 32;
constexpr uint64_t kStatesWaitNs = 2000000000ull;
constexpr int64_t kRowsAtOnce = 8192;  // rows whose tiles' sums are kept at a time
constexpr int kShareCtas = 320;        // tiles of 128 rows, times the shares that their sums over K are cut into, at most
constexpr int kSplitBlocks = 8;        // of 64 in a share of k, at least
constexpr int64_t kPiece = 8192;       // tokens of the vocabulary in a piece, at least

template <int CG>
struct Ring {
  static constexpr int kStages = CG == 2 ? 6 : 4;
  static constexpr int kBytesB = kColumns / CG * kBlockK * 2;
  static constexpr int kBytes = kBytesA + kBytesB;
};

template <int CG>
struct __align__(1024) TileShared {
  uint8_t ring[Ring<CG>::kStages][Ring<CG>::kBytes];
  uint64_t full[Ring<CG>::kStages], empty[Ring<CG>::kStages], acc_full[2], acc_empty[2], drained;
  uint32_t tmem;
  // of a pair, for its end: blocks that each CTA's copies were issued for, and whether a warp of the
  // pair gave up (the copies' of either CTA, the products'); of a place's last block, the bytes of this
  // CTA's copies and of the other's
  uint32_t issued[2], gave_up[3], own[Ring<CG>::kStages], others[Ring<CG>::kStages];
};

enum Mode { kSums, kGradient, kProduct };

struct TileParams {
  CUtensorMap a, b;
  CUtensorMap a_edge, b_edge;  // boxes of what is left at the ends (map_operand)
  int m, n, k;              // of the product
  int m_tiles, n_tiles, width;  // width: columns of a tile
  int n_first;              // neighbouring tiles share rows of A (1) or of B (0)
  uint32_t shape;
  int32_t* status;
  uint64_t wait_ns;
  // kSums, kGradient: rows are tokens, columns the vocabulary
  const void* tokens;
  int tokens_64;
  int64_t token_skip;       // row r's token is r + token_skip
  int64_t token_period;     // sequences' lengths where the last row of each has no token; 0: all do
  int64_t row0;             // of the call
  float factor;             // on products, logits to the base 2
  float2* sums;             // [n_tiles][ld][2]: reference (log2), sum of a tile's halves
  float* at_token;          // [rows]: the token's logit, base 2
  int64_t ld;
  // kGradient
  const float *lse, *grad, *grad_lse;
  const float* unit;        // of G: what brings its rows' factors there, and what takes the sums back
  int col0, vocab;          // this piece's first token
  void* g;                  // [m][ld]
  // kProduct
  float* acc;               // [m][n] sums of earlier pieces
  void* out;                // [m][n], or null: sums stay in acc
  int first;                // nothing in acc yet
  int whole;                // tiles that are summed in one go; the sums of the others are cut into
  int shares;               // shares of K, which meet in
  float* parts;             // [tile][share][rows of a tile][kColumns]
  int wide_out;             // rows of out are 32-byte aligned
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) { return pack_bf16(a, b); }
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 32 bytes, a sector, in one store
__device__ __forceinline__ void store32(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Token of row r of the call: -1 for none
__device__ __forceinline__ int64_t token_of(const void* tokens, int wide, int64_t skip, int64_t period, int64_t r) {
  if (period > 0 && r % period == period - 1) return -1;
  return wide ? static_cast<const int64_t*>(tokens)[r + skip] : static_cast<const int32_t*>(tokens)[r + skip];
}

// One tile of kSums: this thread's row and half of the columns, `x` their products.
__device__ __forceinline__ void tile_sums(const TileParams& P, float (&x)[kHalf], int row, int tile, int half, int n0, int held) {
  int64_t tok = -1;
  if (row < P.m) tok = token_of(P.tokens, P.tokens_64, P.token_skip, P.token_period, P.row0 + row) - n0;
  const int hit = tok >= 0 && tok < held ? int(tok) : -1;
  if (__any_sync(~0u, hit >= 0)) {
    float at = 0.f;
#pragma unroll
    for (int i = 0; i < kHalf; ++i)
      if (hit == i) at = x[i];
    if (hit >= 0) P.at_token[row] = at * P.factor;
  }
  if (held < kHalf) {
#pragma unroll
    for (int i = 0; i < kHalf; ++i)
      if (i >= held) x[i] = -INFINITY;
  }
  float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int i = 4; i < kHalf; ++i) mx[i % 4] = fmaxf(mx[i % 4], x[i]);
  const float ref = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * P.factor;
  const float from = ref == -INFINITY ? 0.f : ref;
  Pair s0(0.f, 0.f), s1(0.f, 0.f);
  const Pair by(P.factor, P.factor), less(-from, -from);
#pragma unroll
  for (int i = 0; i < kHalf; i += 4) {
    float e[4];
    fma2(Pair(x[i], x[i + 1]), by, less).get(e[0], e[1]);
    fma2(Pair(x[i + 2], x[i + 3]), by, less).get(e[2], e[3]);
    s0 = add2(s0, Pair(ex2(e[0]), ex2(e[1])));
    s1 = add2(s1, Pair(ex2(e[2]), ex2(e[3])));
  }
  float a, b;
  add2(s0, s1).get(a, b);
  if (row < P.m) P.sums[(int64_t(tile) * P.ld + row) * 2 + half] = make_float2(ref, a + b);
}

template <typename T>
__device__ __forceinline__ void tile_gradient(const TileParams& P, uint32_t at, int row, int n0, int held) {
  float on_p = 0.f, on_tok = 0.f, lse = 0.f;
  bool none = true;  // nothing of the row counts, whatever it holds
  int64_t tok = -1;
  if (row < P.m) {
    tok = token_of(P.tokens, P.tokens_64, P.token_skip, P.token_period, P.row0 + row);
    const bool ok = tok >= 0 && tok < P.vocab;
    if (!ok && tok != -1) on_tok = NAN;
    if (ok && P.grad) on_tok = P.grad[row];
    on_p = (P.grad_lse ? P.grad_lse[row] : 0.f) - on_tok;
    none = on_p == 0.f && on_tok == 0.f;
    const float up = P.unit[0];
    on_p *= up;
    on_tok *= up;
    lse = P.lse[row] * kLog2e;
    tok -= P.col0 + n0;
  }
  const int hit = row < P.m && tok >= 0 && tok < held ? int(tok) : -1;
  T* g = static_cast<T*>(P.g) + int64_t(row) * P.ld + n0;
  // whole groups of 32, which a row of g has room for; beyond `held` it is not read
  for (int c = 0; c < held; c += 32) {
    uint32_t r[32];
    tmem_load32(r, at + c);
    tmem_wait(r);
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = none ? 0.f : on_p * ex2(fmaf(__uint_as_float(r[i]), P.factor, -lse));
    if (__any_sync(~0u, hit >= c && hit < c + 32)) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (hit == c + i) x[i] += on_tok;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = pack2(x[2 * i], x[2 * i + 1], T());
    if (row < P.m) {
      store32(g + c, r);
      store32(g + c + 16, r + 8);
    }
  }
}

// The same of products that are in registers: loops that leave the columns' numbers known
template <typename T>
__device__ __forceinline__ void tile_gradient(const TileParams& P, const float (&y)[kHalf], int row, int n0, int held) {
  float on_p = 0.f, on_tok = 0.f, lse = 0.f;
  bool none = true;
  int64_t tok = -1;
  if (row < P.m) {
    tok = token_of(P.tokens, P.tokens_64, P.token_skip, P.token_period, P.row0 + row);
    const bool ok = tok >= 0 && tok < P.vocab;
    if (!ok && tok != -1) on_tok = NAN;
    if (ok && P.grad) on_tok = P.grad[row];
    on_p = (P.grad_lse ? P.grad_lse[row] : 0.f) - on_tok;
    none = on_p == 0.f && on_tok == 0.f;
    const float up = P.unit[0];
    on_p *= up;
    on_tok *= up;
    lse = P.lse[row] * kLog2e;
    tok -= P.col0 + n0;
  }
  const int hit = row < P.m && tok >= 0 && tok < held ? int(tok) : -1;
  T* g = static_cast<T*>(P.g) + int64_t(row) * P.ld + n0;
#pragma unroll
  for (int c = 0; c < kHalf; c += 32) {
    if (c >= held) break;
    uint32_t r[16];
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = none ? 0.f : on_p * ex2(fmaf(y[c + i], P.factor, -lse));
    if (__any_sync(~0u, hit >= c && hit < c + 32)) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (hit == c + i) x[i] += on_tok;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = pack2(x[2 * i], x[2 * i + 1], T());
    if (row < P.m) {
      store32(g + c, r);
      store32(g + c + 16, r + 8);
    }
  }
}

// r (8 numbers), times `down`, as 16 bytes
template <typename T>
__device__ __forceinline__ uint4 rounded8(const uint32_t* r, float down) {
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(r[j]) * down;
  return make_uint4(pack2(x[0], x[1], T()), pack2(x[2], x[3], T()), pack2(x[4], x[5], T()), pack2(x[6], x[7], T()));
}

// part: where this thread's row of a share goes, or null
template <typename T>
__device__ __forceinline__ void tile_product(const TileParams& P, uint32_t at, int row, int n0, int held, float* part) {
  const float down = P.unit[1];
  float* acc = part ? part : P.acc + int64_t(row) * P.n + n0;
  const bool add = !part && !P.first;
  T* out = part ? nullptr : static_cast<T*>(P.out) + int64_t(row) * P.n + n0;
  for (int c = 0; c < held; c += 32) {  // held: a multiple of 8
    uint32_t r[32];
    tmem_load32(r, at + c);
    tmem_wait(r);
    if (row < P.m) {
      if (add) {
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          if (c + i < held) {
            const float4 u = *reinterpret_cast<const float4*>(acc + c + i);
            r[i] = __float_as_uint(__uint_as_float(r[i]) + u.x);
            r[i + 1] = __float_as_uint(__uint_as_float(r[i + 1]) + u.y);
            r[i + 2] = __float_as_uint(__uint_as_float(r[i + 2]) + u.z);
            r[i + 3] = __float_as_uint(__uint_as_float(r[i + 3]) + u.w);
          }
      }
      if (part || !P.out) {
#pragma unroll
        for (int i = 0; i < 32; i += 8)
          if (c + i < held) store32(acc + c + i, r + i);
      } else if (P.wide_out && c + 32 <= held) {  // whole sectors: G^T H of 1024 x 32000 x 4096 takes 151 us, with halves 179
#pragma unroll
        for (int i = 0; i < 32; i += 16) {
          const uint4 a = rounded8<T>(r + i, down), b = rounded8<T>(r + i + 8, down);
          const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          store32(out + c + i, w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; i += 8)
          if (c + i < held) *reinterpret_cast<uint4*>(out + c + i) = rounded8<T>(r + i, down);
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void tile_product(const TileParams& P, float (&x)[kHalf], int row, int n0, int held, float* part) {
  if (row >= P.m) return;
  const float down = P.unit[1];
  float* acc = part ? part : P.acc + int64_t(row) * P.n + n0;
  const bool add = !part && !P.first;
  T* out = part ? nullptr : static_cast<T*>(P.out) + int64_t(row) * P.n + n0;
#pragma unroll
  for (int c = 0; c < kHalf; c += 32) {
    if (c >= held) break;
    if (add) {
#pragma unroll
      for (int i = c; i < c + 32; i += 4)
        if (i < held) {
          const float4 u = *reinterpret_cast<const float4*>(acc + i);
          x[i] += u.x;
          x[i + 1] += u.y;
          x[i + 2] += u.z;
          x[i + 3] += u.w;
        }
    }
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(x[c + i]);
    if (part || !P.out) {
#pragma unroll
      for (int i = 0; i < 32; i += 8)
        if (c + i < held) store32(acc + c + i, r + i);
    } else if (P.wide_out && c + 32 <= held) {
#pragma unroll
      for (int i = 0; i < 32; i += 16) {
        const uint4 a = rounded8<T>(r + i, down), b = rounded8<T>(r + i + 8, down);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        store32(out + c + i, w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 8)
        if (c + i < held) *reinterpret_cast<uint4*>(out + c + i) = rounded8<T>(r + i, down);
    }
  }
}

// What one block of k of an operand's tile brings into shared memory: `there` rows (ACROSS: columns, 64
// to a box) by `k_held` of K.  The parts of a box that lie beyond a tensor's ends are slow to come
// (128 rows of which one exists: 0.9 us, all of them: 0.2), so the ends have boxes of their own.  What is
// left as it was in shared memory reaches rows and columns of the product that nothing reads; along
// K, products stop at the last 16 that hold something, and what is left of those is zero.
template <bool ACROSS>
__device__ __forceinline__ uint32_t operand_bytes(int there, int k_held) {
  return ACROSS ? uint32_t((there + 63) / 64 * ((k_held + 15) / 16)) * 2048u : uint32_t(there) * 128u;
}
template <bool ACROSS, bool PAIR, int MOST>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, int x0, int there, int k0, uint32_t bar) {
  if (ACROSS) {
#pragma unroll
    for (int i = 0; i < MOST; i += 64)
      if (i < there) tma_g2s_2d<PAIR>(dst + i * 128, map, x0 + i, k0, bar);
  } else if (there > 0) {
    tma_g2s_2d<PAIR>(dst, map, k0, x0, bar);
  }
}
// The tiles of a CTA (or pair) in turn: t, t + step, ..., without divisions on the way, which the
// ring would run empty for (together 5% at 4096 x 128000 x 4096).  `inner` tiles are neighbours.  From `whole` on
// items are shares of a tile's sum over K, a share of all those tiles after the other (CUT).
template <bool CUT>
struct Walk {
  int t, step, inner, outer, share;  // share: -1 of a whole tile
  int d_inner, d_outer, n_inner, whole, rest, blocks, each, more;
  bool n_first;
  __device__ __forceinline__ Walk(const TileParams& P, int first, int step_) : t(first), step(step_), n_first(P.n_first) {
    n_inner = n_first ? P.n_tiles : P.m_tiles;
    whole = P.whole;
    rest = P.m_tiles * P.n_tiles - whole;
    d_inner = step % n_inner;
    d_outer = step / n_inner;
    blocks = (P.k + kBlockK - 1) / kBlockK;
    each = CUT ? blocks / P.shares : blocks;
    more = CUT ? blocks - each * P.shares : 0;
    place();
  }
  __device__ __forceinline__ void place() {
    int tile = t;
    share = -1;
    if (CUT && t >= whole) {
      share = rest > 0 ? (t - whole) / rest : 0;
      tile = t - share * rest;
    }
    outer = tile / n_inner;
    inner = tile - outer * n_inner;
  }
  __device__ __forceinline__ void next() {
    t += step;
    if (CUT && t >= whole) {
      place();
      return;
    }
    inner += d_inner;
    outer += d_outer;
    if (inner >= n_inner) inner -= n_inner, ++outer;
  }
  __device__ __forceinline__ int mt() const { return n_first ? outer : inner; }
  __device__ __forceinline__ int nt() const { return n_first ? inner : outer; }
  __device__ __forceinline__ int cut() const { return outer * n_inner + inner - whole; }  // of the tiles that are cut
  // blocks of K
  __device__ __forceinline__ int from() const { return !CUT || share < 0 ? 0 : share * each + min(share, more); }
  __device__ __forceinline__ int to() const { return !CUT || share < 0 ? blocks : (share + 1) * each + min(share + 1, more); }
};
// A place in the ring and the parity of its barriers' phases
template <int STAGES>
struct Place {
  uint32_t s = 0, odd = 0;
  __device__ __forceinline__ void next() {
    if (++s == STAGES) {
      s = 0;
      odd ^= 1;
    }
  }
};

// A persistent kernel: one CTA an SM, or a pair of CTAs on two (CG 2), takes tiles of 128 CG rows and
// `width` columns in turn.  One warp copies operands, one issues the products, eight turn the finished
// accumulator into results while the next one fills.
// SEG: sums over K in segments of kSegmentLogits or kSegmentProduct blocks.
template <typename T, int CG, Mode MODE, bool SEG, bool AX, bool BX>
__global__ void __launch_bounds__(kTileThreads, 1) tile_kernel(const __grid_constant__ TileParams P) {
  extern __shared__ uint8_t smem_raw[];
  TileShared<CG>& sh = *reinterpret_cast<TileShared<CG>*>(smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023));
  constexpr int kStages = Ring<CG>::kStages, kSegment = MODE == kProduct ? kSegmentProduct : kSegmentLogits;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1);
      mbar_init(&sh.acc_empty[i], kEpilogueWarps * CG);
    }
    mbar_init(&sh.drained, 1);
    fence_mbar_init();
  }
  if (warp == kEpilogueWarps) tmem_alloc<CG>(&sh.tmem, 2 * kColumns);
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  follow_previous();

  const int items = MODE == kProduct ? P.whole + (P.m_tiles * P.n_tiles - P.whole) * P.shares : P.m_tiles * P.n_tiles;
  const int step = gridDim.x / CG;

  if (warp == kEpilogueWarps) {
    if (lane == 0) {
      const int width = P.width / CG;  // of B's columns that this CTA brings
      const int k_rest = P.k % kBlockK;
      const uint32_t whole_bytes = CG * (operand_bytes<AX>(kRowsOfCta, kBlockK) + operand_bytes<BX>(width, kBlockK));
      const uint32_t whole_end = CG * (operand_bytes<AX>(kRowsOfCta, k_rest) + operand_bytes<BX>(width, k_rest));
      const uint32_t full0 = CG == 2 ? peer_u32(&sh.full[0], 0) : smem_u32(&sh.full[0]), ring0 = smem_u32(sh.ring[0]);
      Place<kStages> at;
      uint32_t done = 0;
      bool lost = false;
      for (Walk<MODE == kProduct> w(P, blockIdx.x / CG, step); w.t < items && !lost; w.next()) {
        const int k_end = w.to();
        const int m0 = w.mt() * kRowsOfCta * CG, n0 = w.nt() * P.width;
        auto there = [](int x0, int extent, int limit) { return min(max(limit - x0, 0), extent); };
        const int a0 = m0 + int(rank) * kRowsOfCta, b0 = n0 + int(rank) * width;
        const int a_there = there(a0, kRowsOfCta, P.m), b_there = there(b0, width, P.n);
        uint32_t bytes = whole_bytes, bytes_end = whole_end;  // of both CTAs
        if (m0 + CG * kRowsOfCta > P.m || n0 + P.width > P.n) {
          bytes = bytes_end = 0;
#pragma unroll
          for (int r = 0; r < CG; ++r) {
            const int ta = there(m0 + r * kRowsOfCta, kRowsOfCta, P.m), tb = there(n0 + r * width, width, P.n);
            bytes += operand_bytes<AX>(ta, kBlockK) + operand_bytes<BX>(tb, kBlockK);
            bytes_end += operand_bytes<AX>(ta, k_rest) + operand_bytes<BX>(tb, k_rest);
          }
        }
        auto bring = [&](int kb, const CUtensorMap* ma, const CUtensorMap* mb, uint32_t n, int k_held) {
          if (!mbar_wait_parked(&sh.empty[at.s], at.odd ^ 1, P.wait_ns)) {
            set_device_error(P.status, DEV_WAIT_TIMEOUT, 4);
            return false;
          }
          if (rank == 0) mbar_arrive_expect_tx(&sh.full[at.s], n);
          if constexpr (CG == 2) {
            const uint32_t own = operand_bytes<AX>(a_there, k_held) + operand_bytes<BX>(b_there, k_held);
            sh.own[at.s] = own;
            sh.others[at.s] = n - own;
          }
          const uint32_t bar = full0 + at.s * 8, a = ring0 + at.s * Ring<CG>::kBytes;
          load_operand<AX, CG == 2, kRowsOfCta>(a, ma, a0, a_there, kb * kBlockK, bar);
          load_operand<BX, CG == 2, kColumns / CG>(a + kBytesA, mb, b0, b_there, kb * kBlockK, bar);
          at.next();
          ++done;
          return true;
        };
        // across, the end of K has boxes of its own; along K, the last rows
        const CUtensorMap *ma = AX || a_there == kRowsOfCta ? &P.a : &P.a_edge, *mb = BX || b_there == width ? &P.b : &P.b_edge;
        int kb = w.from();
        const int whole = min(k_end, P.k / kBlockK);
        for (; kb < whole && !lost; ++kb) lost = !bring(kb, ma, mb, bytes, kBlockK);
        if (kb < k_end && !lost) lost = !bring(kb, AX ? &P.a_edge : ma, BX ? &P.b_edge : mb, bytes_end, k_rest);
      }
      // no copy may be in flight when the CTA ends; a pair sees to that when both know of each other
      if constexpr (CG == 2) {
        store_both(&sh.issued[rank], done);
        store_both(&sh.gave_up[rank], lost);
      } else {
        for (uint32_t i = done < kStages ? 0 : done - kStages; i < done; ++i)
          if (!mbar_wait_parked(&sh.full[i % kStages], i / kStages & 1, kStatesWaitNs)) break;
      }
    }
  } else if (warp == kEpilogueWarps + 1) {
    if (rank == 0 && lane == 0) {
      Place<kStages> at;
      uint32_t i = 0;
      bool lost = false;
      const uint64_t desc_a = tc_operand(smem_u32(sh.ring[0]), AX, 64 * 128), desc_b = tc_operand(smem_u32(sh.ring[0]) + kBytesA, BX, 64 * 128);
      for (Walk<MODE == kProduct> w(P, blockIdx.x / CG, step); w.t < items && !lost; w.next(), ++i) {
        const int k_end = w.to();
        uint32_t buf = 0;
        bool add = false;
        auto open = [&]() {  // the next accumulator
          buf = i & 1;
          add = false;
          if (!mbar_wait_parked(&sh.acc_empty[buf], (i >> 1 & 1) ^ 1, P.wait_ns)) {
            set_device_error(P.status, DEV_WAIT_TIMEOUT, 5);
            return false;
          }
          tc_fence_after();
          return true;
        };
        auto multiply = [&](int steps) {
          if (!mbar_wait_parked(&sh.full[at.s], at.odd, P.wait_ns)) {
            set_device_error(P.status, DEV_WAIT_TIMEOUT, 4);
            return false;
          }
          tc_fence_after();
          const uint64_t a = desc_a + at.s * (Ring<CG>::kBytes / 16), b = desc_b + at.s * (Ring<CG>::kBytes / 16);
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k)
            if (k < steps) {
              tc_mma<CG>(tmem + buf * kColumns, a + k * (AX ? 128 : 2), b + k * (BX ? 128 : 2), P.shape, add);
              add = true;
            }
          tc_commit<CG>(&sh.empty[at.s]);
          at.next();
          return true;
        };
        int kb = w.from();
        const int whole = min(k_end, P.k / kBlockK);
        if (SEG) {
          // an accumulator for each kSegment blocks
          while (kb < k_end && !lost) {
            const int end = min(kb + kSegment, k_end), end_whole = min(end, whole);
            lost = !open();
            for (; kb < end_whole && !lost; ++kb) lost = !multiply(kBlockK / 16);
            for (; kb < end && !lost; ++kb) lost = !multiply((P.k % kBlockK + 15) / 16);
            if (!lost) tc_commit<CG>(&sh.acc_full[buf]);
            if (kb < k_end) ++i;
          }
        } else {
          lost = !open();
          for (; kb < whole && !lost; ++kb) lost = !multiply(kBlockK / 16);
          if (kb < k_end && !lost) lost = !multiply((P.k % kBlockK + 15) / 16);
          if (!lost) tc_commit<CG>(&sh.acc_full[buf]);
        }
      }
      // nor may a product
      tc_commit<CG>(&sh.drained);
      mbar_wait_parked(&sh.drained, 0, kStatesWaitNs);
      if constexpr (CG == 2) store_both(&sh.gave_up[2], lost);
    }
  } else {
    uint32_t i = 0;
    bool lost = false;
    const int half = warp / 4 * kHalf;
    const uint32_t lanes = uint32_t(warp % 4 * 32) << 16;
    auto take = [&]() {  // the next accumulator, when it is full
      if (!__all_sync(~0u, mbar_wait_parked(&sh.acc_full[i & 1], i >> 1 & 1, P.wait_ns))) {
        if (lane == 0) set_device_error(P.status, DEV_WAIT_TIMEOUT, 7);
        lost = true;
      }
      tc_fence_after();
      return tmem + (i & 1) * kColumns + lanes + half;
    };
    auto give = [&]() {  // it is free again
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2)
          mbar_arrive_cluster(peer_u32(&sh.acc_empty[i & 1], 0));
        else
          mbar_arrive(&sh.acc_empty[i & 1]);
      }
      ++i;
    };
    auto part_of = [&](const Walk<MODE == kProduct>& w, int row) {
      return w.share < 0 ? nullptr
                         : P.parts + ((int64_t(w.cut()) * P.shares + w.share) * CG * kRowsOfCta + row - w.mt() * CG * kRowsOfCta) * kColumns + half;
    };
    for (Walk<MODE == kProduct> w(P, blockIdx.x / CG, step); w.t < items && !lost; w.next()) {
      const int row = (w.mt() * CG + int(rank)) * kRowsOfCta + warp % 4 * 32 + lane, n0 = w.nt() * P.width + half;
      const int held = min(kHalf, min(P.width - half, P.n - n0));  // of this half; may be none
      if constexpr (SEG) {
        float x[kHalf];
        uint32_t at = take();
        if (lost) break;
#pragma unroll
        for (int c = 0; c < kHalf; c += 32) {
          uint32_t r[32];
          tmem_load32(r, at + c);
          tmem_wait(r);
#pragma unroll
          for (int j = 0; j < 32; ++j) x[c + j] = __uint_as_float(r[j]);
        }
        give();
        for (int kb = w.from() + kSegment; kb < w.to(); kb += kSegment) {
          at = take();
          if (lost) break;
#pragma unroll
          for (int c = 0; c < kHalf; c += 32) {
            uint32_t r[32];
            tmem_load32(r, at + c);
            tmem_wait(r);
#pragma unroll
            for (int j = 0; j < 32; j += 2)
              add2(Pair(x[c + j], x[c + j + 1]), Pair(__uint_as_float(r[j]), __uint_as_float(r[j + 1]))).get(x[c + j], x[c + j + 1]);
          }
          give();
        }
        if (lost) break;
        if constexpr (MODE == kSums)
          tile_sums(P, x, row, w.nt(), warp / 4, n0, held);
        else if constexpr (MODE == kGradient)
          tile_gradient<T>(P, x, row, n0, held);
        else
          tile_product<T>(P, x, row, n0, held, part_of(w, row));
      } else {
        const uint32_t at = take();
        if (lost) break;
        if constexpr (MODE == kGradient)
          tile_gradient<T>(P, at, row, n0, held);
        else
          tile_product<T>(P, at, row, n0, held, part_of(w, row));
        give();
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) {
    cluster_sync_all();
    // The products' commits arrive in both CTAs: this CTA's last arrival, before it may end
    if (rank != 0 && warp == kEpilogueWarps + 1) mbar_wait_parked(&sh.drained, 0, kStatesWaitNs);
    // Where nobody gave up, the products have waited for every copy.  Otherwise each CTA stopped copying on
    // its own, and copies of either signal the first one's barriers: a block that only one of them copied is
    // waited for without the other's bytes.  (One is ahead by kStages blocks at most: a place is free again only
    // when a product of both CTAs' copies has read it.)
    if (sh.gave_up[0] || sh.gave_up[1] || sh.gave_up[2]) {  // the same in both
      if (rank == 0 && threadIdx.x == kEpilogueWarps * 32) {
        const uint32_t here = sh.issued[0], there = sh.issued[1], most = max(here, there);
        for (uint32_t i = most < kStages ? 0 : most - kStages; i < most; ++i) {
          uint64_t* bar = &sh.full[i % kStages];
          if (i >= here)
            mbar_arrive_expect_tx(bar, load_peer(&sh.own[i % kStages], 1));
          else if (i >= there)
            mbar_complete_tx(bar, sh.others[i % kStages]);
          if (!mbar_wait_parked(bar, i / kStages & 1, kStatesWaitNs)) break;
        }
      }
      __syncwarp();
      cluster_sync_all();
    }
  }
  tc_fence_after();
  if (warp == kEpilogueWarps) tmem_free<CG>(tmem, 2 * kColumns);
}

// Joins the tiles' sums of each row: 16 rows a block, the tiles in 32 shares.
struct JoinParams {
  const float4* sums;
  const float* at_token;
  const void* tokens;
  float *logprob, *lse;
  int32_t* status;
  int64_t ld, token_skip, token_period, row0, vocab;
  int rows, n_tiles, tokens_64, negate;
};
constexpr int kJoinRows = 16, kJoinShares = 32;

__device__ __forceinline__ void join_sums(float2& a, float2 b) {
  const float m = fmaxf(a.x, b.x), from = m == -INFINITY ? 0.f : m;
  a.y = a.y * ex2(a.x - from) + b.y * ex2(b.x - from);
  a.x = m;
}

__global__ void __launch_bounds__(kJoinRows * kJoinShares) join_kernel(const JoinParams P) {
  __shared__ float2 part[kJoinShares][kJoinRows];
  follow_previous();
  const int share = threadIdx.x / kJoinRows, i = threadIdx.x % kJoinRows, row = blockIdx.x * kJoinRows + i;
  float2 s = make_float2(-INFINITY, 0.f);
  if (row < P.rows) {
#pragma unroll 4
    for (int t = share; t < P.n_tiles; t += kJoinShares) {
      const float4 v = P.sums[int64_t(t) * P.ld + row];
      join_sums(s, make_float2(v.x, v.y));
      join_sums(s, make_float2(v.z, v.w));
    }
  }
  part[share][i] = s;
  __syncthreads();
  if (share > 0 || row >= P.rows) return;
  for (int k = 1; k < kJoinShares; ++k) join_sums(s, part[k][i]);
  const bool bad = isnan(s.y) || s.x == INFINITY;
  const float ln_s = logf(s.y);
  const int64_t r = P.row0 + row;
  const int64_t tok = token_of(P.tokens, P.tokens_64, P.token_skip, P.token_period, r);
  float lp;
  if (tok == -1) {
    lp = bad ? NAN : 0.f;
  } else if (tok < 0 || tok >= P.vocab) {
    lp = NAN;
    set_device_error(P.status, DEV_BAD_LIST, int32_t(r));
  } else if (bad) {
    lp = NAN;
  } else {
    const float x = P.at_token[row];
    lp = x == -INFINITY ? -INFINITY : fmaf(x - s.x, kLn2, -ln_s);
  }
  if (P.negate) {
    // H[b][t + 1] from row t of sequence b; its last row has no token, and H[b][0] = 0
    const bool last = r % P.token_period == P.token_period - 1;
    if (last)
      P.logprob[r - (P.token_period - 1)] = 0.f;
    else
      P.logprob[r + 1] = isnan(lp) ? lp : 0.f - lp;
  } else {
    P.logprob[r] = lp;
    if (P.lse) P.lse[r] = bad ? NAN : s.y > 0.f ? fmaf(s.x, kLn2, ln_s) : -INFINITY;
  }
}

// G's unit: G is held as `up` times its rows' factors, with the largest of them at 2^13 (f16 has 2^-24 below 1), and
// the sums are multiplied by `down` = scale / up.  Where all rows have one factor, as those of a mean have, its
// rounding in a G is one and the same in all of them, and so an error of the gradient as a whole (of 1000 rows in f16 at
// a power of two: 2.1 times what rounding the results alone gives, by arithmetic in 64 bits); 2^13 is exact.
struct UnitParams {
  const float *grad, *grad_lse;
  const void* tokens;
  float* unit;
  float scale;
  int64_t rows, vocab;
  int tokens_64;
};
__global__ void __launch_bounds__(1024) unit_kernel(const UnitParams P) {
  __shared__ float part[32];
  follow_previous();
  float big = 0.f;
  for (int64_t r = threadIdx.x; r < P.rows; r += 1024) {
    const int64_t tok = token_of(P.tokens, P.tokens_64, 0, 0, r);
    // without a token grad counts for nothing, and may be anything
    const float g = P.grad && tok >= 0 && tok < P.vocab ? P.grad[r] : 0.f, e = P.grad_lse ? P.grad_lse[r] : 0.f;
    const float x = fmaxf(fabsf(g), fabsf(e - g));
    if (x < INFINITY) big = fmaxf(big, x);
  }
  for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, o));
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = big;
  __syncthreads();
  if (threadIdx.x < 32) {
    big = part[threadIdx.x];
    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, o));
    if (threadIdx.x == 0) {
      // 2^126: both stay normal numbers, for factors of any size
      const float up = big > 0.f ? fminf(8192.f / big, 0x1p126f) : 1.f;
      P.unit[0] = up;
      P.unit[1] = fminf(P.scale / up, FLT_MAX);
    }
  }
}

// Adds the shares of the tiles whose sums were cut, in order, eight numbers a thread.
struct AddParams {
  const float* parts;
  float* acc;
  const float* unit;
  void* out;  // or null: the sums stay in acc
  int m, n, m_tiles, n_tiles, n_first, whole, shares, rows, first;
};
constexpr int kAddThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kAddThreads) add_kernel(const AddParams P) {
  follow_previous();
  const int i = (blockIdx.x * kAddThreads + threadIdx.x) * 8, tile = P.whole + blockIdx.y;
  const int outer = tile / (P.n_first ? P.n_tiles : P.m_tiles), inner = tile - outer * (P.n_first ? P.n_tiles : P.m_tiles);
  const int row = (P.n_first ? outer : inner) * P.rows + i / kColumns, col = (P.n_first ? inner : outer) * kColumns + i % kColumns;
  if (row >= P.m || col >= P.n) return;
  const float* part = P.parts + int64_t(blockIdx.y) * P.shares * P.rows * kColumns + i;
  const int64_t at = int64_t(row) * P.n + col;
  float x[8] = {};
  auto add = [&](const float* p) {
    const float4 u = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + 4);
    x[0] += u.x; x[1] += u.y; x[2] += u.z; x[3] += u.w;
    x[4] += v.x; x[5] += v.y; x[6] += v.z; x[7] += v.w;
  };
  if (!P.first) add(P.acc + at);
#pragma unroll 4
  for (int s = 0; s < P.shares; ++s) add(part + int64_t(s) * P.rows * kColumns);
  uint32_t r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(x[j]);
  if (P.out)
    *reinterpret_cast<uint4*>(static_cast<T*>(P.out) + at) = rounded8<T>(r, P.unit[1]);
  else
    store32(P.acc + at, r);
}

// ---------------------------------------------------------------------- host
struct StatesWs {
  size_t unit, at_token, sums, parts, acc, g, total;
};
int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }
// Tokens of the vocabulary whose part of G is held at a time: at least kPiece, and 2^27 numbers
int64_t piece_of(int64_t rows, int64_t vocab) {
  const int64_t most = std::max(kPiece, (int64_t(1) << 27) / rows / kColumns * kColumns);
  return std::min(round_up(vocab, kColumns), most);
}
StatesWs states_ws(int64_t rows, int64_t vocab, int64_t dim, bool backward) {
  // every part grows with each of the sizes, so that smaller calls can use the workspace of larger ones
  const int64_t at_once = std::min(rows, kRowsAtOnce);
  StatesWs L{};
  L.unit = 256;
  L.at_token = 512;
  L.sums = L.at_token + align256(size_t(at_once) * 4);
  const size_t few = size_t((vocab + 223) / 224) * 2 * std::min<int64_t>(rows, kRowsOfCta) * 8;
  const size_t many = size_t((vocab + kColumns - 1) / kColumns) * 2 * at_once * 8;
  const size_t forward = L.sums + align256(std::max(few, many));
  L.total = forward;
  if (backward) {
    L.parts = 512;
    L.acc = L.parts + align256(size_t(kShareCtas) * kRowsOfCta * kColumns * 4);
    L.g = L.acc + align256(size_t(rows) * dim * 4);
    const int64_t all = rows * round_up(vocab, kColumns);
    L.total = std::max(forward, L.g + align256(size_t(std::min(all, std::max(rows * kPiece, int64_t(1) << 27))) * 2));
  }
  return L;
}

// An operand: rows of `inner` consecutive elements, `stride` elements apart.  Along K (inner is K, rows are
// the product's): boxes of `extent` rows, and of as many as are left at the end.  Across (rows are K): boxes
// of 64 by 64, and at the end of K of what is left, in sixteens.
bool map_operand(CUtensorMap* map, CUtensorMap* edge, int32_t dtype, bool across, const void* base, int64_t inner, int64_t rows,
                 int64_t stride, int extent) {
  const CUtensorMapDataType type = dtype == SEKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const uint64_t bytes = uint64_t(rows > 1 ? stride : round_up(inner, 8)) * 2;
  const int whole = across ? kBlockK : extent, left = int(rows % whole);
  const int rest = left == 0 ? whole : across ? int(round_up(left, 16)) : left;
  return encode_rows2d(map, type, base, uint64_t(inner), uint64_t(rows), bytes, kBlockK, uint32_t(whole)) &&
         encode_rows2d(edge, type, base, uint64_t(inner), uint64_t(rows), bytes, kBlockK, uint32_t(rest));
}

template <typename T, int CG, Mode MODE, bool SEG, bool AX, bool BX>
sekv_status launch_tiles(TileParams& P, int32_t dtype, int sms, cudaStream_t stream) {
  P.shape = tc_shape(kRowsOfCta * CG, P.width, dtype == SEKV_BF16, AX, BX);
  P.m_tiles = int((int64_t(P.m) + kRowsOfCta * CG - 1) / (kRowsOfCta * CG));
  P.n_tiles = (P.n + P.width - 1) / P.width;
  if (int64_t(P.m_tiles) * P.n_tiles > (1 << 30)) return SEKV_ERR_UNSUPPORTED;
  if (P.shares == 0) {  // all tiles whole
    P.whole = P.m_tiles * P.n_tiles;
    P.shares = 1;
  }
  auto fn = tile_kernel<T, CG, MODE, SEG, AX, BX>;
  const size_t shared = sizeof(TileShared<CG>) + 1024;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(shared)) != cudaSuccess) {
    cudaGetLastError();
    return SEKV_ERR_CUDA;
  }
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(unsigned(std::min(P.whole + (P.m_tiles * P.n_tiles - P.whole) * P.shares, sms / CG) * CG));
  lc.blockDim = dim3(kTileThreads);
  lc.dynamicSmemBytes = shared;
  lc.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = CG;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  lc.attrs = at;
  lc.numAttrs = CG == 2 ? 2 : 1;
  if (cudaLaunchKernelEx(&lc, fn, P) != cudaSuccess) {
    cudaGetLastError();
    return SEKV_ERR_CUDA;
  }
  count_launch(1);
  return SEKV_OK;
}

// A pair of CTAs shares a tile of 256 rows where there are that many
int ctas_of(int m) { return m > kRowsOfCta ? 2 : 1; }
// SEG only where a sum is longer than a segment: its tiles pass through registers as a whole, by code that is four times
// as long, which 96 x 32000 x 1024 takes 74 us for and 67 without
template <typename T, Mode MODE, bool SEG, bool AX, bool BX>
sekv_status launch_seg(TileParams& P, int32_t dtype, int sms, cudaStream_t stream) {
  return ctas_of(P.m) == 2 ? launch_tiles<T, 2, MODE, SEG, AX, BX>(P, dtype, sms, stream)
                           : launch_tiles<T, 1, MODE, SEG, AX, BX>(P, dtype, sms, stream);
}
template <typename T, Mode MODE, bool AX, bool BX>
sekv_status launch_for(TileParams& P, int32_t dtype, int sms, cudaStream_t stream) {
  int blocks = (P.k + kBlockK - 1) / kBlockK;  // of the longest sum
  if (MODE == kProduct && P.whole == 0) blocks = (blocks + P.shares - 1) / P.shares;
  if (blocks > (MODE == kProduct ? kSegmentProduct : kSegmentLogits)) return launch_seg<T, MODE, true, AX, BX>(P, dtype, sms, stream);
  return launch_seg<T, MODE, MODE == kSums, AX, BX>(P, dtype, sms, stream);
}

// Columns of a tile of the logits.  Up to 128 rows the weight's bytes bound the product, and 224
// columns are better where the tiles then fill their waves: 1 x 32000 x 4096 47.4 us for 47.9, 1 x
// 128000 160 for 167; 128 columns 55 and 180.
int width_of(int m, int64_t vocab, int sms) {
  if (ctas_of(m) == 2) return kColumns;
  auto time = [&](int w) { return ((vocab + w - 1) / w + sms - 1) / sms * w; };
  return time(224) < time(kColumns) ? 224 : kColumns;
}

// What the calls share: sizes, tensors and tokens.
struct Call {
  const void* states;
  int32_t dtype;
  int64_t rows, vocab, dim, state_stride, weight_stride;
  const void* weight;
  const void* tokens;
  int32_t tokens_64;
  int64_t token_skip, token_period;
  float scale;
  uint8_t* ws;
  size_t ws_bytes;
  int32_t flags;
  cudaStream_t stream;
};

sekv_status check_call(const Call& c, bool backward) {
  if ((c.dtype != SEKV_BF16 && c.dtype != SEKV_F16) || c.rows < 0 || c.vocab < 1 || c.dim < 1 || !c.ws || !c.weight ||
      ((!c.states || !c.tokens) && c.rows > 0))
    return SEKV_ERR_INVALID;
  if (c.dim % 8 != 0 || (c.rows > 1 && (c.state_stride % 8 != 0 || c.state_stride < c.dim)) ||
      (c.vocab > 1 && (c.weight_stride % 8 != 0 || c.weight_stride < c.dim)) || !aligned16(c.states) || !aligned16(c.weight) ||
      reinterpret_cast<uintptr_t>(c.tokens) % (c.tokens_64 ? 8 : 4) || reinterpret_cast<uintptr_t>(c.ws) % 256)
    return SEKV_ERR_INVALID;
  if (!(c.scale > 0.f) || !isfinite(c.scale * kLog2e)) return SEKV_ERR_INVALID;
  if (c.rows > INT32_MAX - 256 || c.vocab > (1 << 30) || c.dim > (1 << 24) || c.state_stride >= int64_t(1) << 38 ||
      c.weight_stride >= int64_t(1) << 38)
    return SEKV_ERR_UNSUPPORTED;
  if (c.rows > 0 && c.ws_bytes < states_ws(c.rows, c.vocab, c.dim, backward).total) return SEKV_ERR_CAPACITY;
  return SEKV_OK;
}

TileParams tile_params(const Call& c) {
  TileParams P{};
  P.status = reinterpret_cast<int32_t*>(c.ws);
  P.wait_ns = (c.flags & SEKV_FLAG_SHORT_WAITS) ? 0 : kStatesWaitNs;
  P.tokens = c.tokens;
  P.tokens_64 = c.tokens_64 != 0;
  P.token_skip = c.token_skip;
  P.token_period = c.token_period;
  P.factor = c.scale * kLog2e;
  P.vocab = int(c.vocab);
  P.k = int(c.dim);
  return P;
}

// The product of a gradient, rounded to `out` (or left in acc, where `last` is false: more pieces follow).  The
// tiles that do not fill a wave have their sums over K cut into shares: of 4096 x 4096 over 32768, 76 pairs of CTAs
// have 256 tiles, three waves and 28 more, which take a wave or, in five shares each, two fifths of one (the gradient of 4096 x
// 128000 x 4096 7.05 ms for 7.3 when it was made; 96 x 32000 x 1024, with four tiles in all, 66 us for 250).
template <typename T, bool AX, bool BX>
sekv_status product(TileParams& P, const Call& c, int sms, bool last, void* out) {
  const int cg = ctas_of(P.m), units = sms / cg, blocks = (P.k + kBlockK - 1) / kBlockK;
  const int64_t m_tiles = (P.m - 1) / (kRowsOfCta * cg) + 1, tiles = m_tiles * ((P.n - 1) / kColumns + 1);
  const int rest = int(tiles % units);
  int shares = 1;
  auto time = [&](int s) { return double((rest * s + units - 1) / units) / s + 0.002 * s; };
  for (int s = 2; s <= units && rest > 0 && rest * s * cg <= kShareCtas && blocks / s >= kSplitBlocks; ++s)
    if (time(s) < time(shares)) shares = s;
  const bool cut = shares > 1 && (time(1) - time(shares)) * blocks >= 16;  // what adding them up costs
  P.whole = int(cut ? tiles - rest : tiles);
  P.shares = cut ? shares : 1;
  P.out = last ? out : nullptr;
  P.wide_out = P.n % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 32 == 0;
  sekv_status st = launch_for<T, kProduct, AX, BX>(P, c.dtype, sms, c.stream);
  if (st != SEKV_OK || !cut) return st;
  AddParams A{};
  A.parts = P.parts;
  A.acc = P.acc;
  A.unit = P.unit;
  A.out = P.out;
  A.m = P.m;
  A.n = P.n;
  A.m_tiles = P.m_tiles;
  A.n_tiles = P.n_tiles;
  A.n_first = P.n_first;
  A.whole = P.whole;
  A.shares = shares;
  A.rows = cg * kRowsOfCta;
  A.first = P.first;
  return launch_following(add_kernel<T>, dim3(unsigned(A.rows * kColumns / 8 / kAddThreads), unsigned(rest)), kAddThreads, 0, c.stream, A);
}

template <typename T>
sekv_status forward(const Call& c, float* logprob, float* lse, bool negate) {
  const int sms = device_sm_count();
  if (sms <= 0) return SEKV_ERR_CUDA;
  const StatesWs L = states_ws(c.rows, c.vocab, c.dim, false);
  for (int64_t r0 = 0; r0 < c.rows; r0 += kRowsAtOnce) {
    TileParams P = tile_params(c);
    P.m = int(std::min(c.rows - r0, kRowsAtOnce));
    P.n = int(c.vocab);
    P.row0 = r0;
    P.at_token = reinterpret_cast<float*>(c.ws + L.at_token);
    P.sums = reinterpret_cast<float2*>(c.ws + L.sums);
    P.ld = P.m;
    P.width = width_of(P.m, c.vocab, sms);
    const int cg = ctas_of(P.m);
    const void* states = static_cast<const T*>(c.states) + r0 * c.state_stride;
    if (!map_operand(&P.a, &P.a_edge, c.dtype, false, states, c.dim, P.m, c.state_stride, kRowsOfCta) ||
        !map_operand(&P.b, &P.b_edge, c.dtype, false, c.weight, c.dim, c.vocab, c.weight_stride, P.width / cg))
      return SEKV_ERR_UNSUPPORTED;
    sekv_status st = launch_for<T, kSums, false, false>(P, c.dtype, sms, c.stream);
    if (st != SEKV_OK) return st;
    JoinParams J{};
    J.sums = reinterpret_cast<const float4*>(P.sums);
    J.at_token = P.at_token;
    J.tokens = c.tokens;
    J.logprob = logprob;
    J.lse = lse;
    J.status = P.status;
    J.ld = P.ld;
    J.token_skip = c.token_skip;
    J.token_period = c.token_period;
    J.row0 = r0;
    J.vocab = c.vocab;
    J.rows = P.m;
    J.n_tiles = P.n_tiles;
    J.tokens_64 = c.tokens_64 != 0;
    J.negate = negate;
    st = launch_following(join_kernel, dim3(unsigned((P.m + kJoinRows - 1) / kJoinRows)), kJoinRows * kJoinShares, 0, c.stream, J);
    if (st != SEKV_OK) return st;
  }
  return SEKV_OK;
}

template <typename T>
sekv_status backward(const Call& c, const float* lse, const float* grad, const float* grad_lse, void* d_states, void* d_weight) {
  const int sms = device_sm_count();
  if (sms <= 0) return SEKV_ERR_CUDA;
  const StatesWs L = states_ws(c.rows, c.vocab, c.dim, true);
  UnitParams U{};
  U.grad = grad;
  U.grad_lse = grad_lse;
  U.unit = reinterpret_cast<float*>(c.ws + L.unit);
  U.scale = c.scale;
  U.rows = c.rows;
  U.vocab = c.vocab;
  U.tokens = c.tokens;
  U.tokens_64 = c.tokens_64 != 0;
  sekv_status st = launch_following(unit_kernel, dim3(1), 1024, 0, c.stream, U);
  const int64_t piece = piece_of(c.rows, c.vocab);
  T* g = reinterpret_cast<T*>(c.ws + L.g);
  for (int64_t v0 = 0; v0 < c.vocab && st == SEKV_OK; v0 += piece) {
    const int64_t nv = std::min(piece, c.vocab - v0);
    const T* weight = static_cast<const T*>(c.weight) + v0 * c.weight_stride;
    TileParams P = tile_params(c);
    P.m = int(c.rows);
    P.n = int(nv);
    P.col0 = int(v0);
    P.lse = lse;
    P.grad = grad;
    P.grad_lse = grad_lse;
    P.unit = U.unit;
    P.g = g;
    P.ld = piece;
    P.width = width_of(P.m, nv, sms);
    if (!map_operand(&P.a, &P.a_edge, c.dtype, false, c.states, c.dim, c.rows, c.state_stride, kRowsOfCta) ||
        !map_operand(&P.b, &P.b_edge, c.dtype, false, weight, c.dim, nv, c.weight_stride, P.width / ctas_of(P.m)))
      return SEKV_ERR_UNSUPPORTED;
    st = launch_for<T, kGradient, false, false>(P, c.dtype, sms, c.stream);
    if (st == SEKV_OK && d_states) {  // G W, summed over the pieces
      TileParams Q = tile_params(c);
      Q.m = int(c.rows);
      Q.n = int(c.dim);
      Q.k = int(nv);
      Q.width = kColumns;
      Q.unit = U.unit;
      Q.acc = reinterpret_cast<float*>(c.ws + L.acc);
      Q.first = v0 == 0;
      if (!map_operand(&Q.a, &Q.a_edge, c.dtype, false, g, nv, c.rows, piece, kRowsOfCta) ||
          !map_operand(&Q.b, &Q.b_edge, c.dtype, true, weight, c.dim, nv, c.weight_stride, kBlockK))
        return SEKV_ERR_UNSUPPORTED;
      Q.parts = reinterpret_cast<float*>(c.ws + L.parts);
      st = product<T, false, true>(Q, c, sms, v0 + piece >= c.vocab, d_states);
    }
    if (st == SEKV_OK && d_weight) {  // G^T H
      TileParams Q = tile_params(c);
      Q.m = int(nv);
      Q.n = int(c.dim);
      Q.k = int(c.rows);
      Q.width = kColumns;
      Q.n_first = 1;
      Q.unit = U.unit;
      Q.first = 1;
      Q.parts = reinterpret_cast<float*>(c.ws + L.parts);
      if (!map_operand(&Q.a, &Q.a_edge, c.dtype, true, g, nv, c.rows, piece, kBlockK) ||
          !map_operand(&Q.b, &Q.b_edge, c.dtype, true, c.states, c.dim, c.rows, c.state_stride, kBlockK))
        return SEKV_ERR_UNSUPPORTED;
      st = product<T, true, true>(Q, c, sms, true, static_cast<T*>(d_weight) + v0 * c.dim);
    }
  }
  return st;
}

}  // namespace

extern "C" size_t sekv_states_workspace_size(int64_t rows, int64_t vocab, int64_t dim, int32_t backward) {
  if (rows < 0 || vocab < 1 || dim < 1 || rows > INT32_MAX - 256 || vocab > (1 << 30) || dim > (1 << 24)) return 0;
  return states_ws(rows, vocab, dim, backward != 0).total;
}

extern "C" sekv_status sekv_states_logprobs(const void* states, int32_t dtype, int64_t n_rows, int64_t dim, int64_t state_stride,
                                            const void* weight, int64_t vocab, int64_t weight_stride, const void* tokens,
                                            int32_t tokens_64, float scale, float* logprob, float* lse, int32_t flags,
                                            void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  reset_launches();
  const Call c{states, dtype, n_rows, vocab, dim, state_stride, weight_stride, weight, tokens, tokens_64, 0, 0, scale,
               static_cast<uint8_t*>(workspace), workspace_bytes, flags, stream};
  const sekv_status st = check_call(c, false);
  if (st != SEKV_OK) return st;
  if (n_rows == 0) return SEKV_OK;
  if (!logprob) return SEKV_ERR_INVALID;
  return dtype == SEKV_BF16 ? forward<__nv_bfloat16>(c, logprob, lse, false) : forward<__half>(c, logprob, lse, false);
}

extern "C" sekv_status sekv_states_surprisal(const void* states, int32_t dtype, int64_t batch, int64_t ctx_len, int64_t dim,
                                             int64_t state_stride, const void* weight, int64_t vocab, int64_t weight_stride,
                                             const void* tokens, int32_t tokens_64, float* H, int32_t flags, void* workspace,
                                             size_t workspace_bytes, cudaStream_t stream) {
  reset_launches();
  if (batch < 0 || ctx_len < 0) return SEKV_ERR_INVALID;
  if (batch > INT32_MAX || ctx_len > INT32_MAX) return SEKV_ERR_UNSUPPORTED;
  const Call c{states, dtype, batch * ctx_len, vocab, dim, state_stride, weight_stride, weight, tokens, tokens_64, 1, ctx_len, 1.f,
               static_cast<uint8_t*>(workspace), workspace_bytes, flags, stream};
  const sekv_status st = check_call(c, false);
  if (st != SEKV_OK) return st;
  if (c.rows == 0) return SEKV_OK;
  if (!H) return SEKV_ERR_INVALID;
  return dtype == SEKV_BF16 ? forward<__nv_bfloat16>(c, H, nullptr, true) : forward<__half>(c, H, nullptr, true);
}

extern "C" sekv_status sekv_states_logprobs_backward(const void* states, int32_t dtype, int64_t n_rows, int64_t dim,
                                                     int64_t state_stride, const void* weight, int64_t vocab,
                                                     int64_t weight_stride, const void* tokens, int32_t tokens_64, float scale,
                                                     const float* lse, const float* grad_logprob, const float* grad_lse,
                                                     void* d_states, void* d_weight, int32_t flags, void* workspace,
                                                     size_t workspace_bytes, cudaStream_t stream) {
  reset_launches();
  const Call c{states, dtype, n_rows, vocab, dim, state_stride, weight_stride, weight, tokens, tokens_64, 0, 0, scale,
               static_cast<uint8_t*>(workspace), workspace_bytes, flags, stream};
  const sekv_status st = check_call(c, true);
  if (st != SEKV_OK) return st;
  if (!aligned16(d_states) || !aligned16(d_weight) || (n_rows > 0 && !lse)) return SEKV_ERR_INVALID;
  if (n_rows == 0) {
    if (d_weight && cudaMemsetAsync(d_weight, 0, size_t(vocab) * dim * 2, stream) != cudaSuccess) return SEKV_ERR_CUDA;
    return SEKV_OK;
  }
  if (!d_states && !d_weight) return SEKV_OK;
  return dtype == SEKV_BF16 ? backward<__nv_bfloat16>(c, lse, grad_logprob, grad_lse, d_states, d_weight)
                            : backward<__half>(c, lse, grad_logprob, grad_lse, d_states, d_weight);
}
