// Host-side helpers shared by the C-ABI translation units.
#pragma once

#include <cuda.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/sekv.h"
#include "sekv_common.cuh"

namespace sekv {

int device_sm_count();
int decode_cg(const sekv_config* cfg, int sms);
int route_chunks(const sekv_config* cfg);
WsLayout ws_layout(const sekv_config* cfg, int sms);
size_t ws_cta_bytes(const WsLayout& L);
void count_launch(int n);
void reset_launches();

// Rows of row_elems elements ([groups][rows][row_elems], dense) seen as
// (x: half a row, row, half, group): a box of box_rows rows brings both
// 128-byte halves of each row in one copy, 128-byte swizzle.
bool encode_rows4d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base,
                   uint64_t row_elems, uint64_t rows, uint64_t groups, int elem_bytes,
                   uint32_t box_rows);

// Rows of `inner` 16-bit elements, `stride` bytes apart, in boxes of box_inner elements by
// box_rows rows, 128-byte swizzle, zeros beyond the ends.
bool encode_rows2d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, uint64_t inner,
                   uint64_t rows, uint64_t stride, uint32_t box_inner, uint32_t box_rows);

// Launches a kernel that begins with follow_previous(): its blocks may be on their way
// while the kernel before it on the stream still runs.
template <typename Params>
inline sekv_status launch_following(void (*kernel)(Params), dim3 grid, int threads, size_t shared,
                                    cudaStream_t stream, Params P) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = grid;
  lc.blockDim = dim3(threads);
  lc.dynamicSmemBytes = shared;
  lc.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, kernel, P) != cudaSuccess) {
    cudaGetLastError();
    return SEKV_ERR_CUDA;
  }
  count_launch(1);
  return SEKV_OK;
}
// Waits for the kernel before this one and what it wrote; only then may the next one's blocks
// be on their way, so that a kernel never runs beside any but the one before it.
__device__ __forceinline__ void follow_previous() {
  pdl_wait();
  pdl_launch_dependents();
}

size_t build_workspace_size(const sekv_config* cfg, int64_t ctx_len);
size_t kv4_workspace_size(const sekv_config* cfg, int64_t n_q);

}  // namespace sekv
