// The 4-bit cache's layout (include/sekv.h) as the kernels use it.
#pragma once

#include <cuda_fp16.h>

#include "decode_host.h"
#include "host_common.h"

namespace sekv {

constexpr int kKv4Page = SEKV_KV4_PAGE_TOKENS;
constexpr int kKv4PageBytes = SEKV_KV4_PAGE_BYTES;
constexpr int kKv4Tile = 16;          // tokens
constexpr int kKv4TileBytes = 2304;   // K codes, V codes, K and V scales and zeros
constexpr int kKv4V = 1024;           // V codes
constexpr int kKv4Params = 2048;      // K scales and zeros; V's 128 bytes further

// Eight neighbouring dimensions 8*oct .. 8*oct+7 of token row j of a tile: K
// keeps them in one 32-bit word, V in the same half of two neighbouring words
// (the other half is the token next to it).
__host__ __device__ inline int kv4_k_word(int j, int oct) {
  const int d = oct * 8;
  return 64 * j + 16 * ((d & 63) >> 4) + 8 * (d >> 6) + 4 * (oct & 1);
}
__host__ __device__ inline int kv4_v_half(int j, int oct) {
  return kKv4V + 512 * (j >> 3) + 64 * (oct & 7) + 16 * ((j & 7) >> 1) + 8 * (oct >> 3) + 2 * (j & 1);
}
// (s, z) of group g of token row j
__host__ __device__ inline int kv4_param(int j, int g, bool v) {
  return kKv4Params + (v ? 128 : 0) + 32 * ((j & 7) >> 1) + 16 * (j >> 3) + 8 * (j & 1) + 4 * g;
}

struct Kv4Pages {
  uint8_t* pages;
  const int32_t* table;
  int32_t* status;
  int n_pages, max_pages, hkv;

  // Tile of token t of sequence b (KV head c), or null after flagging a bad
  // page or a position past the table.
  __device__ __forceinline__ uint8_t* tile(int b, int c, int64_t t) const {
    const int64_t p = t / kKv4Page;
    int id = -1;
    if (p < max_pages) id = table[int64_t(b) * max_pages + p];
    if (id < 0 || id >= n_pages) {
      set_device_error(status, DEV_BAD_LIST, b);
      return nullptr;
    }
    return pages + (int64_t(id) * hkv + c) * kKv4PageBytes +
           int(t % kKv4Page) / kKv4Tile * kKv4TileBytes;
  }
};

// cfg and cache of a kv4 call, and whether the workspace is large enough for n_q
// query tokens.
sekv_status kv4_check(const sekv_config* cfg, const sekv_kv4_cache* cache, int n_q,
                      const void* workspace);
sekv_status kv4_check_ws(const sekv_config* cfg, int n_q, size_t workspace_bytes);

}  // namespace sekv
