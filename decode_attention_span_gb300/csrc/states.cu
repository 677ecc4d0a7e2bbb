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
// tile, the gradient a tile of G as 16-bit numbers, for one piece of the vocabulary at a time,
// which the other two products read.
#include <cuda_fp16.h>
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
constexpr int kEpilogueWarps = 4;
constexpr int kThreads = (kEpilogueWarps + 2) * 32;
constexpr uint64_t kStatesWaitNs = 2000000000ull;
constexpr int64_t kRowsAtOnce = 8192;  // rows whose tiles' sums are kept at a time
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
};

enum Mode { kSums, kGradient, kProduct };

struct TileParams {
  CUtensorMap a, b;
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
  float2* sums;             // [n_tiles][ld]: reference (log2), sum
  float* at_token;          // [rows]: the token's logit, base 2
  int64_t ld;
  // kGradient
  const float *lse, *grad, *grad_lse;
  const float* unit;        // of G
  float scale;
  int col0, vocab;          // this piece's first token
  void* g;                  // [m][ld]
  // kProduct
  float* acc;               // [m][n] sums of earlier pieces
  void* out;                // [m][n], or null: sums stay in acc
  int first;                // nothing in acc yet
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

// One tile of kSums: this thread's row.
__device__ __forceinline__ void tile_sums(const TileParams& P, uint32_t at, int row, int tile, int n0, int held) {
  float ref = -INFINITY, sum = 0.f;
  int64_t tok = -1;
  if (row < P.m) tok = token_of(P.tokens, P.tokens_64, P.token_skip, P.token_period, P.row0 + row) - n0;
  const int hit = tok >= 0 && tok < held ? int(tok) : -1;
  for (int c = 0; c < held; c += 32) {
    uint32_t r[32];
    tmem_load32(r, at + c);
    tmem_wait(r);
    if (c + 32 > held) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c + i >= held) r[i] = 0xff800000u;  // -infinity
    }
    float mx = __uint_as_float(r[0]);
#pragma unroll
    for (int i = 1; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(r[i]));
    const float up = fmaxf(ref, mx * P.factor);
    const float from = up == -INFINITY ? 0.f : up;
    sum *= ex2(ref - from);
    ref = up;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      s0 += ex2(fmaf(__uint_as_float(r[i]), P.factor, -from));
      s1 += ex2(fmaf(__uint_as_float(r[i + 1]), P.factor, -from));
    }
    sum += s0 + s1;
    if (__any_sync(~0u, hit >= c && hit < c + 32)) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (hit == c + i) x = __uint_as_float(r[i]);
      if (hit >= c && hit < c + 32) P.at_token[row] = x * P.factor;
    }
  }
  if (row < P.m) P.sums[int64_t(tile) * P.ld + row] = make_float2(ref, sum);
}

template <typename T>
__device__ __forceinline__ void tile_gradient(const TileParams& P, uint32_t at, int row, int n0) {
  const int held = min(P.width, P.n - n0);
  float on_p = 0.f, on_tok = 0.f, lse = 0.f;
  int64_t tok = -1;
  if (row < P.m) {
    tok = token_of(P.tokens, P.tokens_64, P.token_skip, P.token_period, P.row0 + row);
    const bool ok = tok >= 0 && tok < P.vocab;
    if (!ok && tok != -1) on_tok = NAN;
    if (ok && P.grad) on_tok = P.grad[row];
    on_p = (P.grad_lse ? P.grad_lse[row] : 0.f) - on_tok;
    const float up = P.scale * *P.unit;
    on_p *= up;
    on_tok *= up;
    lse = P.lse[row] * kLog2e;
    tok -= P.col0 + n0;
  }
  const bool none = on_p == 0.f && on_tok == 0.f;  // nothing of the row counts, whatever it holds
  const int hit = row < P.m && tok >= 0 && tok < held ? int(tok) : -1;
  T* g = static_cast<T*>(P.g) + int64_t(row) * P.ld + n0;
  for (int c = 0; c < P.width; c += 32) {
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
    if (c + 32 > held) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c + i >= held) x[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = pack2(x[2 * i], x[2 * i + 1], T());
    if (row < P.m) {
      store32(g + c, r);
      store32(g + c + 16, r + 8);
    }
  }
}

template <typename T>
__device__ __forceinline__ void tile_product(const TileParams& P, uint32_t at, int row, int n0) {
  const int held = min(P.width, P.n - n0);  // a multiple of 8
  const float down = P.unit ? 1.f / *P.unit : 1.f;
  float* acc = P.acc + int64_t(row) * P.n + n0;
  T* out = static_cast<T*>(P.out) + int64_t(row) * P.n + n0;
  for (int c = 0; c < held; c += 32) {
    uint32_t r[32];
    tmem_load32(r, at + c);
    tmem_wait(r);
    if (row < P.m) {
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        if (c + i < held) {
          if (!P.first) {
            const float4 u = *reinterpret_cast<const float4*>(acc + c + i), v = *reinterpret_cast<const float4*>(acc + c + i + 4);
            const float o[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i + j] = __float_as_uint(__uint_as_float(r[i + j]) + o[j]);
          }
          if (P.out) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(r[i + j]) * down;
            *reinterpret_cast<uint4*>(out + c + i) =
                make_uint4(pack2(x[0], x[1], T()), pack2(x[2], x[3], T()), pack2(x[4], x[5], T()), pack2(x[6], x[7], T()));
          } else {
            store32(acc + c + i, r + i);
          }
        }
      }
    }
  }
}

// A persistent kernel: one CTA an SM, or a pair of CTAs on two (CG 2), takes tiles of 128 CG rows and
// `width` columns in turn.  One warp copies operands, one issues the products, four turn the finished
// accumulator into results while the next one fills.
template <typename T, int CG, Mode MODE, bool AX, bool BX>
__global__ void __launch_bounds__(kThreads, 1) tile_kernel(const __grid_constant__ TileParams P) {
  extern __shared__ uint8_t smem_raw[];
  TileShared<CG>& sh = *reinterpret_cast<TileShared<CG>*>(smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023));
  constexpr int kStages = Ring<CG>::kStages;
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

  const int tiles = P.m_tiles * P.n_tiles, step = gridDim.x / CG;
  const int k_blocks = (P.k + kBlockK - 1) / kBlockK;
  auto place = [&](int t, int& mt, int& nt) {
    if (P.n_first) {
      mt = t / P.n_tiles;
      nt = t - mt * P.n_tiles;
    } else {
      nt = t / P.m_tiles;
      mt = t - nt * P.m_tiles;
    }
  };

  if (warp == kEpilogueWarps) {
    if (lane == 0) {
      const int width = P.width / CG;  // of B's columns that this CTA brings
      const uint32_t bytes = uint32_t(CG) * (kBytesA + width * kBlockK * 2);
      uint32_t done = 0;
      bool lost = false;
      for (int t = blockIdx.x / CG; t < tiles && !lost; t += step) {
        int mt, nt;
        place(t, mt, nt);
        const int m0 = mt * kRowsOfCta * CG + int(rank) * kRowsOfCta, n0 = nt * P.width + int(rank) * width;
        for (int kb = 0; kb < k_blocks; ++kb, ++done) {
          const uint32_t s = done % kStages;
          if (!mbar_wait_parked(&sh.empty[s], (done / kStages & 1) ^ 1, P.wait_ns)) {
            set_device_error(P.status, DEV_WAIT_TIMEOUT, 4);
            lost = true;
            break;
          }
          const uint32_t bar = CG == 2 ? peer_u32(&sh.full[s], 0) : smem_u32(&sh.full[s]);
          if (rank == 0) mbar_arrive_expect_tx(&sh.full[s], bytes);
          const uint32_t a = smem_u32(sh.ring[s]), b = a + kBytesA;
          if (AX) {
            for (int i = 0; i < kRowsOfCta; i += 64) tma_g2s_2d<CG == 2>(a + i * 128, &P.a, m0 + i, kb * kBlockK, bar);
          } else {
            tma_g2s_2d<CG == 2>(a, &P.a, kb * kBlockK, m0, bar);
          }
          if (BX) {
            for (int i = 0; i < width; i += 64) tma_g2s_2d<CG == 2>(b + i * 128, &P.b, n0 + i, kb * kBlockK, bar);
          } else {
            tma_g2s_2d<CG == 2>(b, &P.b, kb * kBlockK, n0, bar);
          }
        }
      }
      // no copy may be in flight when the CTA ends
      if (rank == 0)
        for (uint32_t i = done < kStages ? 0 : done - kStages; i < done; ++i)
          if (!mbar_wait_parked(&sh.full[i % kStages], i / kStages & 1, kStatesWaitNs)) break;
    }
  } else if (warp == kEpilogueWarps + 1) {
    if (rank == 0 && lane == 0) {
      uint32_t done = 0, i = 0;
      bool lost = false;
      for (int t = blockIdx.x / CG; t < tiles && !lost; t += step, ++i) {
        const uint32_t buf = i & 1;
        if (!mbar_wait_parked(&sh.acc_empty[buf], (i >> 1 & 1) ^ 1, P.wait_ns)) {
          set_device_error(P.status, DEV_WAIT_TIMEOUT, 5);
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < k_blocks; ++kb, ++done) {
          const uint32_t s = done % kStages;
          if (!mbar_wait_parked(&sh.full[s], done / kStages & 1, P.wait_ns)) {
            set_device_error(P.status, DEV_WAIT_TIMEOUT, 4);
            lost = true;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(sh.ring[s]), b = a + kBytesA;
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k)
            tc_mma<CG>(tmem + buf * kColumns, tc_operand(a + k * (AX ? 2048 : 32), AX, 64 * 128),
                       tc_operand(b + k * (BX ? 2048 : 32), BX, 64 * 128), P.shape, kb + k > 0);
          tc_commit<CG>(&sh.empty[s]);
        }
        if (!lost) tc_commit<CG>(&sh.acc_full[buf]);
      }
      // nor may a product
      tc_commit<CG>(&sh.drained);
      mbar_wait_parked(&sh.drained, 0, kStatesWaitNs);
    }
  } else {
    uint32_t i = 0;
    for (int t = blockIdx.x / CG; t < tiles; t += step, ++i) {
      const uint32_t buf = i & 1;
      const bool there = mbar_wait_parked(&sh.acc_full[buf], i >> 1 & 1, P.wait_ns);
      if (!__all_sync(~0u, there)) {
        if (lane == 0) set_device_error(P.status, DEV_WAIT_TIMEOUT, 7);
        break;
      }
      tc_fence_after();
      int mt, nt;
      place(t, mt, nt);
      const int row = (mt * CG + int(rank)) * kRowsOfCta + warp * 32 + lane, n0 = nt * P.width;
      const uint32_t at = tmem + buf * kColumns + (uint32_t(warp * 32) << 16);
      if constexpr (MODE == kSums)
        tile_sums(P, at, row, nt, n0, min(P.width, P.n - n0));
      else if constexpr (MODE == kGradient)
        tile_gradient<T>(P, at, row, n0);
      else
        tile_product<T>(P, at, row, n0);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2)
          mbar_arrive_cluster(peer_u32(&sh.acc_empty[buf], 0));
        else
          mbar_arrive(&sh.acc_empty[buf]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  tc_fence_after();
  if (warp == kEpilogueWarps) tmem_free<CG>(tmem, 2 * kColumns);
}

// Joins the tiles' sums of each row: 16 rows a block, the tiles in 32 shares.
struct JoinParams {
  const float2* sums;
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
    for (int t = share; t < P.n_tiles; t += kJoinShares) join_sums(s, P.sums[int64_t(t) * P.ld + row]);
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

// A power of two that brings the largest factor on a row of G to 2^13 .. 2^14 (f16 has 2^-24 below
// it), or 1 (bf16).
struct UnitParams {
  const float *grad, *grad_lse;
  float* unit;
  float scale;
  int64_t rows;
  int f16;
};
__global__ void __launch_bounds__(1024) unit_kernel(const UnitParams P) {
  __shared__ float part[32];
  follow_previous();
  float big = 0.f;
  if (P.f16)
    for (int64_t r = threadIdx.x; r < P.rows; r += 1024) {
      const float g = P.grad ? P.grad[r] : 0.f, e = P.grad_lse ? P.grad_lse[r] : 0.f;
      const float x = fmaxf(fabsf(g), fabsf(e - g)) * P.scale;
      if (x < INFINITY) big = fmaxf(big, x);
    }
  for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, o));
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = big;
  __syncthreads();
  if (threadIdx.x < 32) {
    big = part[threadIdx.x];
    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, o));
    if (threadIdx.x == 0) {
      float unit = 1.f;
      if (big > 0.f) {
        const int e = int(__float_as_uint(big) >> 23) - 127;
        unit = __uint_as_float(uint32_t(min(max(127 + 13 - e, 1), 253)) << 23);
      }
      *P.unit = unit;
    }
  }
}

// ---------------------------------------------------------------------- host
struct StatesWs {
  size_t unit, at_token, sums, acc, g, total;
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
  const size_t few = size_t((vocab + 127) / 128) * std::min<int64_t>(rows, kRowsOfCta) * 8;
  const size_t many = size_t((vocab + kColumns - 1) / kColumns) * at_once * 8;
  const size_t forward = L.sums + align256(std::max(few, many));
  L.total = forward;
  if (backward) {
    L.acc = 512;
    L.g = L.acc + align256(size_t(rows) * dim * 4);
    const int64_t all = rows * round_up(vocab, kColumns);
    L.total = std::max(forward, L.g + align256(size_t(std::min(all, std::max(rows * kPiece, int64_t(1) << 27))) * 2));
  }
  return L;
}

// Rows of `inner` consecutive elements, `stride` elements apart, in boxes of 64 elements and `box` rows
bool map_rows(CUtensorMap* map, int32_t dtype, const void* base, int64_t inner, int64_t rows, int64_t stride, int box) {
  return encode_rows2d(map, dtype == SEKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base,
                       uint64_t(inner), uint64_t(rows), uint64_t(rows > 1 ? stride : round_up(inner, 8)) * 2, kBlockK, uint32_t(box));
}

template <typename T, int CG, Mode MODE, bool AX, bool BX>
sekv_status launch_tiles(TileParams& P, int32_t dtype, int sms, cudaStream_t stream) {
  P.shape = tc_shape(kRowsOfCta * CG, P.width, dtype == SEKV_BF16, AX, BX);
  P.m_tiles = int((int64_t(P.m) + kRowsOfCta * CG - 1) / (kRowsOfCta * CG));
  P.n_tiles = (P.n + P.width - 1) / P.width;
  if (int64_t(P.m_tiles) * P.n_tiles > (1 << 30)) return SEKV_ERR_UNSUPPORTED;
  auto fn = tile_kernel<T, CG, MODE, AX, BX>;
  const size_t shared = sizeof(TileShared<CG>) + 1024;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(shared)) != cudaSuccess) {
    cudaGetLastError();
    return SEKV_ERR_CUDA;
  }
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(unsigned(std::min(P.m_tiles * P.n_tiles, sms / CG) * CG));
  lc.blockDim = dim3(kThreads);
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
template <typename T, Mode MODE, bool AX, bool BX>
sekv_status launch_for(TileParams& P, int32_t dtype, int sms, cudaStream_t stream) {
  return ctas_of(P.m) == 2 ? launch_tiles<T, 2, MODE, AX, BX>(P, dtype, sms, stream)
                           : launch_tiles<T, 1, MODE, AX, BX>(P, dtype, sms, stream);
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
  P.scale = c.scale;
  P.factor = c.scale * kLog2e;
  P.vocab = int(c.vocab);
  P.k = int(c.dim);
  return P;
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
    P.width = kColumns;
    const int cg = ctas_of(P.m);
    const void* states = static_cast<const T*>(c.states) + r0 * c.state_stride;
    if (!map_rows(&P.a, c.dtype, states, c.dim, P.m, c.state_stride, kRowsOfCta) ||
        !map_rows(&P.b, c.dtype, c.weight, c.dim, c.vocab, c.weight_stride, P.width / cg))
      return SEKV_ERR_UNSUPPORTED;
    sekv_status st = launch_for<T, kSums, false, false>(P, c.dtype, sms, c.stream);
    if (st != SEKV_OK) return st;
    JoinParams J{};
    J.sums = P.sums;
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
  U.f16 = c.dtype == SEKV_F16;
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
    P.width = kColumns;
    if (!map_rows(&P.a, c.dtype, c.states, c.dim, c.rows, c.state_stride, kRowsOfCta) ||
        !map_rows(&P.b, c.dtype, weight, c.dim, nv, c.weight_stride, P.width / ctas_of(P.m)))
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
      Q.out = v0 + piece >= c.vocab ? d_states : nullptr;
      if (!map_rows(&Q.a, c.dtype, g, nv, c.rows, piece, kRowsOfCta) ||
          !map_rows(&Q.b, c.dtype, weight, c.dim, nv, c.weight_stride, kBlockK))
        return SEKV_ERR_UNSUPPORTED;
      st = launch_for<T, kProduct, false, true>(Q, c.dtype, sms, c.stream);
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
      Q.out = static_cast<T*>(d_weight) + v0 * c.dim;
      if (!map_rows(&Q.a, c.dtype, g, nv, c.rows, piece, kBlockK) ||
          !map_rows(&Q.b, c.dtype, c.states, c.dim, c.rows, c.state_stride, kBlockK))
        return SEKV_ERR_UNSUPPORTED;
      st = launch_for<T, kProduct, true, true>(Q, c.dtype, sms, c.stream);
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
