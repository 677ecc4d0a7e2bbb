// sekv_kv4_append and sekv_kv4_read: tokens into the 4-bit cache and back.
//
// Bound by memory: append reads 512 bytes and writes 144 per (token, KV head),
// read the reverse.  One warp takes a tile (16 tokens of one KV head, 2304
// bytes): lanes 0-15 a token's K row, lanes 16-31 its V row, eight dimensions a
// lane; eight lanes hold a group of 64.  A tile that is written whole is put
// together in shared memory and leaves in 16-byte stores (V's codes of a token
// are 2-byte pieces 64 bytes apart, which one by one cost a memory sector each);
// of a tile written in part only the tokens' own bytes are touched.
//
// Codes: n = rint(fl((x - z) / s)) by definition.  The quotient is taken with the
// group's reciprocal and Markstein's correction (q + (a - q s) r, the residual exact in
// an fma), which rounds as a division does.
//
// Measured, 32768 tokens of 8 KV heads: append 35 us (172 MB, 25 us at the copy rate; a row is
// one chain of waits, reductions, reciprocal, codes and stores, two rows side by side: issue 74%,
// ALU 51%, DRAM 51%, half of the warps, nothing full), read 28 us (the same bytes), one after
// the other 59 us.
// Arithmetic on two floats at a time took 5 us off both.  With an approximate quotient and
// a division wherever it came near a half (39% of bf16 rows have such a value) append took
// 48 us; a warp per token with direct stores took 226 us for both.
#include "kv4.cuh"

using namespace sekv;

namespace {

constexpr int kStoreThreads = 64;  // 128: 60.2 us for 59 of both, 256: 63
constexpr int kStoreWarps = kStoreThreads / 32;
constexpr int kRowsAhead = 4;  // token rows on their way to a warp (8: 2% slower, fewer warps fit)

struct StoreParams {
  Kv4Pages pg;
  const void *k, *v;
  void *ko, *vo;
  int64_t ks[3], vs[3];
  const int32_t *first, *n_valid;
  int n_tokens;
  int tiles;         // per sequence and KV head, whatever `first` is
  int64_t items;     // warps: batch * tiles * hkv
};

// One warp's tile: tokens t0 .. t1 - 1 of the call (rows from j0 on of the tile) of
// sequence b and KV head c; false where there is nothing to do.
struct TileWork {
  uint8_t* tile;
  int b, c, t0, t1, j0;
};
__device__ __forceinline__ bool tile_work(const StoreParams& P, TileWork& W) {
  const int64_t item = int64_t(blockIdx.x) * kStoreWarps + (threadIdx.x >> 5);
  if (item >= P.items) return false;
  W.c = int(item % P.pg.hkv);
  const int64_t bt = item / P.pg.hkv;
  const int k = int(bt % P.tiles);
  W.b = int(bt / P.tiles);
  const int n = P.n_valid ? min(P.n_valid[W.b], P.n_tokens) : P.n_tokens;
  const int64_t first = P.first[W.b];
  // tile k covers positions base .. base + 15 (rounded down, also below zero)
  const int64_t base = (first - (first & (kKv4Tile - 1))) + int64_t(k) * kKv4Tile;
  const int64_t p0 = max(base, first), p1 = min(base + kKv4Tile, first + n);
  if (p0 >= p1) return false;
  if (base < 0) {
    set_device_error(P.pg.status, DEV_BAD_LIST, W.b);
    return false;
  }
  W.tile = P.pg.tile(W.b, W.c, base);
  W.t0 = int(p0 - first);
  W.t1 = int(p1 - first);
  W.j0 = int(p0 - base);
  return W.tile != nullptr;
}

// Smaller or larger of each of two pairs, NaN if either is NaN.
__device__ __forceinline__ __nv_bfloat162 min2(__nv_bfloat162 a, __nv_bfloat162 b) { return __hmin2_nan(a, b); }
__device__ __forceinline__ __half2 min2(__half2 a, __half2 b) { return __hmin2_nan(a, b); }
__device__ __forceinline__ __nv_bfloat162 max2(__nv_bfloat162 a, __nv_bfloat162 b) { return __hmax2_nan(a, b); }
__device__ __forceinline__ __half2 max2(__half2 a, __half2 b) { return __hmax2_nan(a, b); }
__device__ __forceinline__ float2 floats(uint32_t w, __nv_bfloat162) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 floats(uint32_t w, __half2) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// largest bf16 at or below x (a bf16 input is one itself)
__device__ __forceinline__ float bf16_at_or_below(float x, __nv_bfloat162) { return x; }
__device__ __forceinline__ float bf16_at_or_below(float x, __half2) {
  return __bfloat162float(__float2bfloat16_rd(x));
}

// The codes where s is below 2^-100, and a reciprocal or a quotient may be out of range.
template <typename T2>
__device__ __noinline__ uint32_t small_codes(uint4 in, float z, float s) {
  const uint32_t u[4] = {in.x, in.y, in.z, in.w};
  uint32_t word = 0;
  for (int i = 7; i >= 0; --i) {
    const float2 x = floats(u[i >> 1], T2());
    const float n = rintf(__fdiv_rn((i & 1 ? x.y : x.x) - z, s));
    word = word * 16 + uint32_t(fminf(fmaxf(n, 0.f), 15.f));
  }
  return word;
}

// Codes (eight nibbles) and bf16 s | z << 16 of this lane's eight values, whose group is
// held by eight neighbouring lanes.
template <typename T2>
__device__ __forceinline__ void quantise(const uint4& in, uint32_t& word, uint32_t& sz) {
  const uint32_t u[4] = {in.x, in.y, in.z, in.w};
  auto pair = [&](int i) { return *reinterpret_cast<const T2*>(&u[i]); };
  const T2 mn2 = min2(min2(pair(0), pair(1)), min2(pair(2), pair(3)));
  const T2 mx2 = max2(max2(pair(0), pair(1)), max2(pair(2), pair(3)));
  // (minimum, -maximum) as one pair, so that one reduction does both
  const uint32_t a = *reinterpret_cast<const uint32_t*>(&mn2);
  const uint32_t b = *reinterpret_cast<const uint32_t*>(&mx2) ^ 0x80008000u;
  const uint32_t lo = __byte_perm(a, b, 0x5410), hi = __byte_perm(a, b, 0x7632);
  T2 m = min2(*reinterpret_cast<const T2*>(&lo), *reinterpret_cast<const T2*>(&hi));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const uint32_t other = __shfl_xor_sync(~0u, *reinterpret_cast<const uint32_t*>(&m), o);
    m = min2(m, *reinterpret_cast<const T2*>(&other));
  }
  const float2 ends = floats(*reinterpret_cast<const uint32_t*>(&m), T2());
  const float mx = -ends.y;
  const float z = bf16_at_or_below(ends.x, T2());
  const __nv_bfloat16 sb = __float2bfloat16_rn((mx - z) * (1.f / 15.f));
  const float s = __bfloat162float(sb);
  sz = __byte_perm(__bfloat16_as_ushort(sb), __float_as_uint(z), 0x7610);
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number
  // one comparison of bits for kSmall <= s <= the largest number
  constexpr uint32_t kSmall = 0x0d800000u, kLargest = 0x7f7fffffu;  // 2^-100
  if (__float_as_uint(s) - kSmall <= kLargest - kSmall) {
    float r;  // 1 / s to an ulp, then by Newton's step
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    r = fmaf(fmaf(-s, r, 1.f), r, r);
    uint32_t w = 0;
    const Pair r2(r, r), s2(-s, -s);
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      const float2 x = floats(u[i], T2());
      const Pair d = add2(Pair(x.x, x.y), Pair(-z, -z)), q0 = mul2(d, r2);
      float even, odd;
      add2(fma2(fma2(q0, s2, d), r2, q0), Pair(kRound, kRound)).get(even, odd);
      w = w * 16 + __float_as_uint(odd);  // the bits of kRound come off below
      w = w * 16 + __float_as_uint(even);
    }
    word = w - __float_as_uint(kRound) * 0x11111111u;
  } else if (s > 0.f && s < 1.f) {
    word = small_codes<T2>(in, z, s);
  } else {
    // one value in the whole group (s 0); or a NaN or an infinity in it, or a range beyond
    // fp32, which leave s no number
    word = 0;
    if (s != 0.f) sz = 0x7fff7fffu;
  }
}

// Where a lane's pieces of a token row go in a tile: the codes' lower and upper half
// (K's in one word, V's four bytes apart), and the scale and zero point, at offsets linear in
// the three parts of the row number.
struct RowPlace {
  uint32_t codes, upper, odd, pair, params;
  __device__ explicit RowPlace(int lane) {
    const bool v = lane >= 16;
    codes = v ? kv4_v_half(0, lane & 15) : kv4_k_word(0, lane & 15);
    upper = v ? 4 : 2;
    odd = v ? 2 : 64;    // j % 2
    pair = v ? 16 : 128; // (j % 8) / 2
    params = kv4_param(0, (lane & 15) >> 3, v);
  }
  __device__ __forceinline__ void put(uint8_t* tile, int j, bool group_lead, uint32_t word,
                                      uint32_t sz) const {
    const uint32_t o = j & 1, u = (j >> 1) & 3, e = j >> 3;
    uint8_t* at = tile + (codes + o * odd + u * pair + e * 512);
    *reinterpret_cast<uint16_t*>(at) = uint16_t(word);
    *reinterpret_cast<uint16_t*>(at + upper) = uint16_t(word >> 16);
    if (group_lead) *reinterpret_cast<uint32_t*>(tile + (params + 8 * o + 32 * u + 16 * e)) = sz;
  }
};

template <typename T2>
__global__ void __launch_bounds__(kStoreThreads) kv4_append_kernel(const StoreParams P) {
  __shared__ __align__(16) uint8_t staged[kStoreWarps][kKv4TileBytes];
  __shared__ uint4 in[kStoreWarps][kRowsAhead][32];  // each lane copies and reads its own
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  follow_previous();
  TileWork W;
  if (!tile_work(P, W)) return;  // warp-uniform
  const bool whole = W.t1 - W.t0 == kKv4Tile;
  const int64_t step = lane < 16 ? P.ks[1] : P.vs[1];  // elements of 2 bytes
  const uint16_t* src =
      (lane < 16 ? static_cast<const uint16_t*>(P.k) + W.b * P.ks[0] + W.c * P.ks[2]
                 : static_cast<const uint16_t*>(P.v) + W.b * P.vs[0] + W.c * P.vs[2]) +
      W.t0 * step + (lane & 15) * 8;
  const int rows = W.t1 - W.t0;
  // Rows come through a ring in shared memory: kRowsAhead of them on their way without
  // holding registers.  One group of copies per row, empty past the last row.
  auto fetch = [&](int i) {
    if (i < rows)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       smem_u32(&in[warp][i % kRowsAhead][lane])),
                   "l"(src + i * step)
                   : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto row = [&](int i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kRowsAhead - 1) : "memory");
    return in[warp][i % kRowsAhead][lane];
  };  // the slot is filled again once the row has been used
  for (int i = 0; i < kRowsAhead; ++i) fetch(i);
  const RowPlace place(lane);
  const bool lead = (lane & 7) == 0;
  if (!whole) {
    for (int i = 0; i < rows; ++i) {
      uint32_t word, sz;
      quantise<T2>(row(i), word, sz);
      place.put(W.tile, W.j0 + i, lead, word, sz);
      fetch(i + kRowsAhead);
    }
    return;
  }
#pragma unroll 2
  for (int j = 0; j < kKv4Tile; ++j) {
    uint32_t word, sz;
    quantise<T2>(row(j), word, sz);
    place.put(staged[warp], j, lead, word, sz);
    fetch(j + kRowsAhead);
  }
  __syncwarp();
  for (int i = lane; i < kKv4TileBytes / 16; i += 32)
    reinterpret_cast<uint4*>(W.tile)[i] = reinterpret_cast<const uint4*>(staged[warp])[i];
}

__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                 pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])));
}
__device__ __forceinline__ void store8(__half* p, const float (&x)[8]) {
  __half2 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
  __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<uint4*>(h));
}

template <typename T>
__global__ void __launch_bounds__(kStoreThreads) kv4_read_kernel(const StoreParams P) {
  __shared__ __align__(16) uint8_t staged[kStoreWarps][kKv4TileBytes];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  follow_previous();
  TileWork W;
  if (!tile_work(P, W)) return;  // warp-uniform
  const uint8_t* tile = W.tile;
  if (W.t1 - W.t0 > 2) {  // more than a few rows: bring the whole tile
    uint4 in[5];
#pragma unroll
    for (int i = 0; i < 5; ++i)
      if (lane + 32 * i < kKv4TileBytes / 16) in[i] = __ldcs(reinterpret_cast<const uint4*>(W.tile) + lane + 32 * i);
#pragma unroll
    for (int i = 0; i < 5; ++i)
      if (lane + 32 * i < kKv4TileBytes / 16) reinterpret_cast<uint4*>(staged[warp])[lane + 32 * i] = in[i];
    __syncwarp();
    tile = staged[warp];
  }
  const int oct = lane & 15;
  T* dst = static_cast<T*>(lane < 16 ? P.ko : P.vo) +
           ((int64_t(W.b) * P.pg.hkv + W.c) * P.n_tokens + W.t0) * kHeadDim + oct * 8;
  const int rows = W.t1 - W.t0;
#pragma unroll 8
  for (int i = 0; i < rows; ++i) {
    const int j = W.j0 + i;
    uint32_t word;
    if (lane < 16) {
      word = *reinterpret_cast<const uint32_t*>(tile + kv4_k_word(j, oct));
    } else {
      word = *reinterpret_cast<const uint16_t*>(tile + kv4_v_half(j, oct)) |
             uint32_t(*reinterpret_cast<const uint16_t*>(tile + kv4_v_half(j, oct) + 4)) << 16;
    }
    const uint32_t sz = *reinterpret_cast<const uint32_t*>(tile + kv4_param(j, oct >> 3, lane >= 16));
    const float s = __uint_as_float(sz << 16), z = __uint_as_float(sz & 0xffff0000u);
    float x[8];
    // a byte under the exponent of 2^23 is 2^23 + n
    const uint32_t even = word & 0x0f0f0f0fu, odd = word >> 4 & 0x0f0f0f0fu;
#pragma unroll
    for (int d = 0; d < 8; d += 2) {
      const Pair n = add2(Pair(__uint_as_float(__byte_perm(even, 0x4b000000u, 0x7440 + d / 2)),
                               __uint_as_float(__byte_perm(odd, 0x4b000000u, 0x7440 + d / 2))),
                          Pair(-8388608.f, -8388608.f));
      fma2(Pair(s, s), n, Pair(z, z)).get(x[d], x[d + 1]);
    }
    store8(dst + int64_t(i) * kHeadDim, x);
  }
}

StoreParams store_params(const sekv_config* cfg, const sekv_kv4_cache* cache, int32_t n_tokens,
                         const int32_t* first, const int32_t* n_valid, void* workspace) {
  StoreParams P{};
  P.pg.pages = static_cast<uint8_t*>(cache->pages);
  P.pg.table = cache->page_table;
  P.pg.status = static_cast<int32_t*>(workspace);
  P.pg.n_pages = cache->n_pages;
  P.pg.max_pages = cache->max_pages;
  P.pg.hkv = cfg->n_kv_heads;
  P.first = first;
  P.n_valid = n_valid;
  P.n_tokens = n_tokens;
  P.tiles = (n_tokens + kKv4Tile - 2) / kKv4Tile + 1;  // `first` may stand anywhere in a tile
  P.items = int64_t(cfg->batch) * P.tiles * cfg->n_kv_heads;
  return P;
}

constexpr int64_t kStoreItemsMax = int64_t(INT32_MAX) * kStoreWarps;

}  // namespace

extern "C" sekv_status sekv_kv4_append(const sekv_config* cfg, const sekv_kv4_cache* cache,
                                       int32_t dtype, const void* k, const int64_t k_stride[3],
                                       const void* v, const int64_t v_stride[3],
                                       int32_t n_tokens, const int32_t* first,
                                       const int32_t* n_valid, void* workspace,
                                       size_t workspace_bytes, cudaStream_t stream) {
  reset_launches();
  sekv_status st = kv4_check(cfg, cache, 1, workspace);
  if (st != SEKV_OK) return st;
  if (dtype != SEKV_BF16 && dtype != SEKV_F16) return SEKV_ERR_INVALID;
  if (((!k || !v) && n_tokens != 0) || !k_stride || !v_stride || !first || n_tokens < 0 ||
      !aligned16(k) || !aligned16(v))
    return SEKV_ERR_INVALID;
  StoreParams P = store_params(cfg, cache, n_tokens, first, n_valid, workspace);
  P.k = k;
  P.v = v;
  const int64_t size[3] = {cfg->batch, n_tokens, cfg->n_kv_heads};
  for (int i = 0; i < 3; ++i) {
    if (size[i] <= 1) continue;  // the stride of a single row means nothing
    if (k_stride[i] % 8 != 0 || v_stride[i] % 8 != 0) return SEKV_ERR_INVALID;
    P.ks[i] = k_stride[i];
    P.vs[i] = v_stride[i];
  }
  if (n_tokens == 0) return SEKV_OK;
  if (n_tokens > (1 << 30)) return SEKV_ERR_UNSUPPORTED;
  if (P.items > kStoreItemsMax) return SEKV_ERR_UNSUPPORTED;
  st = kv4_check_ws(cfg, 1, workspace_bytes);
  if (st != SEKV_OK) return st;
  const unsigned blocks = unsigned((P.items + kStoreWarps - 1) / kStoreWarps);
  return launch_following(dtype == SEKV_BF16 ? kv4_append_kernel<__nv_bfloat162> : kv4_append_kernel<__half2>,
                          dim3(blocks), kStoreThreads, 0, stream, P);
}

extern "C" sekv_status sekv_kv4_read(const sekv_config* cfg, const sekv_kv4_cache* cache,
                                     int32_t dtype, void* k_out, void* v_out, int32_t n_tokens,
                                     const int32_t* first, const int32_t* n_valid,
                                     void* workspace, size_t workspace_bytes,
                                     cudaStream_t stream) {
  reset_launches();
  sekv_status st = kv4_check(cfg, cache, 1, workspace);
  if (st != SEKV_OK) return st;
  if (dtype < SEKV_BF16 || dtype > SEKV_F32) return SEKV_ERR_INVALID;
  if (((!k_out || !v_out) && n_tokens != 0) || !first || n_tokens < 0 || !aligned16(k_out) || !aligned16(v_out))
    return SEKV_ERR_INVALID;
  StoreParams P = store_params(cfg, cache, n_tokens, first, n_valid, workspace);
  P.ko = k_out;
  P.vo = v_out;
  if (n_tokens == 0) return SEKV_OK;
  if (n_tokens > (1 << 30)) return SEKV_ERR_UNSUPPORTED;
  if (P.items > kStoreItemsMax) return SEKV_ERR_UNSUPPORTED;
  st = kv4_check_ws(cfg, 1, workspace_bytes);
  if (st != SEKV_OK) return st;
  const unsigned blocks = unsigned((P.items + kStoreWarps - 1) / kStoreWarps);
  return launch_following(dtype == SEKV_BF16  ? kv4_read_kernel<__nv_bfloat16>
                          : dtype == SEKV_F16 ? kv4_read_kernel<__half>
                                              : kv4_read_kernel<float>,
                          dim3(blocks), kStoreThreads, 0, stream, P);
}
