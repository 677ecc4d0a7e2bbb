// sekv_kv4_append and sekv_kv4_read: tokens into the 4-bit cache and back.
//
// Bound by memory: append reads 512 bytes and writes 144 per (token, KV head).
// One warp takes a (token, KV head): lanes 0-15 its K row, lanes 16-31 its V
// row, eight dimensions a lane.  Eight lanes hold a group of 64, so its minimum and
// maximum take three shuffles; the lane's eight codes are one 32-bit word.
#include "kv4.cuh"

using namespace sekv;

namespace {

constexpr int kStoreThreads = 256;

struct StoreParams {
  Kv4Pages pg;
  const void *k, *v;
  void *ko, *vo;
  int64_t ks[3], vs[3];
  const int32_t *first, *n_valid;
  int n_tokens;
  int64_t items;  // batch * n_tokens * hkv
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8], __nv_bfloat16) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8], __half) {
  const __half2* h = reinterpret_cast<const __half2*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <typename T>
__global__ void __launch_bounds__(kStoreThreads) kv4_append_kernel(const StoreParams P) {
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * (kStoreThreads / 32) + (threadIdx.x >> 5);
  if (item >= P.items) return;  // warp-uniform
  const int c = int(item % P.pg.hkv);
  const int64_t bt = item / P.pg.hkv;
  const int t = int(bt % P.n_tokens), b = int(bt / P.n_tokens);
  if (P.n_valid && t >= P.n_valid[b]) return;
  const int64_t pos = int64_t(P.first[b]) + t;
  uint8_t* tile = pos >= 0 ? P.pg.tile(b, c, pos) : nullptr;
  if (!tile) {
    if (pos < 0) set_device_error(P.pg.status, DEV_BAD_LIST, b);
    return;
  }
  const int j = int(pos % kKv4Tile);
  const bool is_v = lane >= 16;
  const int oct = lane & 15;
  const T* src = is_v ? static_cast<const T*>(P.v) + b * P.vs[0] + t * P.vs[1] + c * P.vs[2]
                      : static_cast<const T*>(P.k) + b * P.ks[0] + t * P.ks[1] + c * P.ks[2];
  float x[8];
  unpack8(reinterpret_cast<const uint4*>(src)[oct], x, T());
  float mn = x[0], mx = x[0];
  bool fin = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mn = fminf(mn, x[i]);
    mx = fmaxf(mx, x[i]);
    fin &= fabsf(x[i]) <= 3.4028235e38f;  // false for NaN too
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    mn = fminf(mn, __shfl_xor_sync(~0u, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
  }
  const uint32_t ok = __ballot_sync(~0u, fin) >> (lane & 24) & 0xffu;
  __nv_bfloat16 zb = __float2bfloat16_rd(mn);
  const float z = __bfloat162float(zb);
  __nv_bfloat16 sb = __float2bfloat16_rn((mx - z) * (1.f / 15.f));
  const float s = __bfloat162float(sb);
  if (ok != 0xffu || !(fabsf(s) <= 3.4028235e38f) || !(fabsf(z) <= 3.4028235e38f))
    sb = zb = __ushort_as_bfloat16(0x7fffu);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float n = s > 0.f ? rintf(__fdiv_rn(x[i] - z, s)) : 0.f;
    word |= uint32_t(fminf(fmaxf(n, 0.f), 15.f)) << (4 * i);
  }
  if (!is_v) {
    *reinterpret_cast<uint32_t*>(tile + kv4_k_word(j, oct)) = word;
  } else {
    *reinterpret_cast<uint16_t*>(tile + kv4_v_half(j, oct)) = uint16_t(word);
    *reinterpret_cast<uint16_t*>(tile + kv4_v_half(j, oct) + 4) = uint16_t(word >> 16);
  }
  if ((lane & 7) == 0) {
    const uint32_t sz = uint32_t(__bfloat16_as_ushort(sb)) | uint32_t(__bfloat16_as_ushort(zb)) << 16;
    *reinterpret_cast<uint32_t*>(tile + kv4_param(j, oct >> 3, is_v)) = sz;
  }
}

__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                            pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(__half* p, const float (&x)[8]) {
  __half2 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(h);
}

template <typename T>
__global__ void __launch_bounds__(kStoreThreads) kv4_read_kernel(const StoreParams P) {
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * (kStoreThreads / 32) + (threadIdx.x >> 5);
  if (item >= P.items) return;
  const int t = int(item % P.n_tokens);
  const int64_t bc = item / P.n_tokens;
  const int c = int(bc % P.pg.hkv), b = int(bc / P.pg.hkv);
  if (P.n_valid && t >= P.n_valid[b]) return;
  const int64_t pos = int64_t(P.first[b]) + t;
  const uint8_t* tile = pos >= 0 ? P.pg.tile(b, c, pos) : nullptr;
  if (!tile) {
    if (pos < 0) set_device_error(P.pg.status, DEV_BAD_LIST, b);
    return;
  }
  const int j = int(pos % kKv4Tile);
  const bool is_v = lane >= 16;
  const int oct = lane & 15;
  uint32_t word;
  if (!is_v) {
    word = *reinterpret_cast<const uint32_t*>(tile + kv4_k_word(j, oct));
  } else {
    word = *reinterpret_cast<const uint16_t*>(tile + kv4_v_half(j, oct)) |
           uint32_t(*reinterpret_cast<const uint16_t*>(tile + kv4_v_half(j, oct) + 4)) << 16;
  }
  const uint32_t sz = *reinterpret_cast<const uint32_t*>(tile + kv4_param(j, oct >> 3, is_v));
  const float s = __uint_as_float(sz << 16), z = __uint_as_float(sz & 0xffff0000u);
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf(s, float((word >> (4 * i)) & 15u), z);
  T* dst = static_cast<T*>(is_v ? P.vo : P.ko) + item * kHeadDim + oct * 8;
  store8(dst, x);
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
  P.items = int64_t(cfg->batch) * n_tokens * cfg->n_kv_heads;
  return P;
}

constexpr int64_t kStoreItemsMax = int64_t(INT32_MAX) * (kStoreThreads / 32);

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
  if (!k || !v || !k_stride || !v_stride || !first || n_tokens < 0 || !aligned16(k) ||
      !aligned16(v))
    return SEKV_ERR_INVALID;
  StoreParams P = store_params(cfg, cache, n_tokens, first, n_valid, workspace);
  P.k = k;
  P.v = v;
  for (int i = 0; i < 3; ++i) {
    if (k_stride[i] % 8 != 0 || v_stride[i] % 8 != 0) return SEKV_ERR_INVALID;
    P.ks[i] = k_stride[i];
    P.vs[i] = v_stride[i];
  }
  if (n_tokens == 0) return SEKV_OK;
  if (P.items > kStoreItemsMax) return SEKV_ERR_UNSUPPORTED;
  st = kv4_check_ws(cfg, 1, workspace_bytes);
  if (st != SEKV_OK) return st;
  const unsigned blocks = unsigned((P.items + kStoreThreads / 32 - 1) / (kStoreThreads / 32));
  if (dtype == SEKV_BF16)
    kv4_append_kernel<__nv_bfloat16><<<blocks, kStoreThreads, 0, stream>>>(P);
  else
    kv4_append_kernel<__half><<<blocks, kStoreThreads, 0, stream>>>(P);
  if (cudaGetLastError() != cudaSuccess) return SEKV_ERR_CUDA;
  count_launch(1);
  return SEKV_OK;
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
  if (!k_out || !v_out || !first || n_tokens < 0 || !aligned16(k_out) || !aligned16(v_out))
    return SEKV_ERR_INVALID;
  StoreParams P = store_params(cfg, cache, n_tokens, first, n_valid, workspace);
  P.ko = k_out;
  P.vo = v_out;
  if (n_tokens == 0) return SEKV_OK;
  if (P.items > kStoreItemsMax) return SEKV_ERR_UNSUPPORTED;
  st = kv4_check_ws(cfg, 1, workspace_bytes);
  if (st != SEKV_OK) return st;
  const unsigned blocks = unsigned((P.items + kStoreThreads / 32 - 1) / (kStoreThreads / 32));
  if (dtype == SEKV_BF16)
    kv4_read_kernel<__nv_bfloat16><<<blocks, kStoreThreads, 0, stream>>>(P);
  else if (dtype == SEKV_F16)
    kv4_read_kernel<__half><<<blocks, kStoreThreads, 0, stream>>>(P);
  else
    kv4_read_kernel<float><<<blocks, kStoreThreads, 0, stream>>>(P);
  if (cudaGetLastError() != cudaSuccess) return SEKV_ERR_CUDA;
  count_launch(1);
  return SEKV_OK;
}
