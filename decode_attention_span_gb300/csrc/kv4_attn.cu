// sekv_kv4_attention: attention of a few query tokens over the 4-bit cache.
//
// Bound by memory: 144 bytes per (token, KV head) are read once for all query
// heads of the group.  The cache's layout is the tensor cores' operand
// layout, so a lane's codes come from shared memory as 16-byte words and become
// bf16 operands with one shift and one lop3 per pair (0x4300 | n is 128 + n
// exactly); no value is rebuilt.  With K^ = z + s n for each group of 64
// dimensions,
//   q . K^ = sum over groups of  s (sum_d q_d n_d) + z (sum_d q_d)
// and the 128 is taken off by starting the product's accumulators at
// -128 sum_d q_d.  For V, sum_j p_j V^_j = sum_j (p_j s_j) (n_j - 8) + sum_j
// p_j (z_j + 8 s_j): the weights p_j s_j enter the product as the sum of two bf16
// numbers (16 significant bits), the upper one in rows 0-7 of the A operand and
// the lower in rows 8-15, which the eight (token, head) columns leave free; so
// the result keeps fp32's usefulness at no further matrix instruction.
//
// Work: the cache is a line of chunks of 32 tokens (sequence by sequence, in
// it KV head by KV head), cut into equal pieces, one per CTA.  The warps of a CTA
// share a piece chunk by chunk, each with its own ring of bulk copies.  A CTA
// joins its warps' softmax states per (sequence, KV head) and, where that
// group spans several CTAs, leaves a partial; the last of them to finish joins
// the partials in order.
#include <math.h>

#include <type_traits>

#include "kv4.cuh"

using namespace sekv;

namespace {

constexpr int kAttnWarps = 12;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kStages = 3;
constexpr int kChunkTokens = 32;
constexpr int kChunkBytes = 2 * kKv4TileBytes;
constexpr int kCols = 8;                         // (token, head) pairs of a block
constexpr int kStateFloats = kCols * (kHeadDim + 2);  // o, m, l
constexpr uint64_t kWaitNs = 2000000000ull;

struct AttnShared {
  uint8_t ring[kAttnWarps][kStages][kChunkBytes];
  float o[kAttnWarps][kCols][kHeadDim];
  float m[kAttnWarps][kCols];
  float l[kAttnWarps][kCols];
  float w[kAttnWarps][kCols];
  float mx[kCols], sum[kCols];
  uint64_t bar[kAttnWarps][kStages];
  int64_t before[SEKV_KV4_MAX_BATCH + 1];  // chunks before each sequence
  int last;
};

struct AttnParams {
  Kv4Pages pg;
  const void* q;
  const int32_t* seq_len;
  float *out, *lse;
  float* partials;   // [CTA][2][kStateFloats]
  int32_t* arrived;  // per group; zero between calls
  int batch, hpg, n_q, tpb, n_blk;
  float scale_log2;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// codes i and i + 4 of a word as a bf16 pair 128 + n
__device__ __forceinline__ uint32_t codes(uint32_t w, int i) {
  return ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
}
// the same, n - 8 (exact)
__device__ __forceinline__ uint32_t centred(uint32_t w, int i) {
  const uint32_t c = codes(w, i);
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&c),
                                   __nv_bfloat162(__ushort_as_bfloat16(0x4308),
                                                  __ushort_as_bfloat16(0x4308)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 2^x, to 2^-22 of its value; 0 for -infinity
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float q_value(const __nv_bfloat16* q) { return __bfloat162float(*q); }
__device__ __forceinline__ float q_value(const __half* q) { return __half2float(*q); }

// A warp's softmax state of one group: columns g = lane / 4, and of the values
// the dimensions that the matrix product's accumulators give this lane.
struct WarpState {
  float o[16][4];
  float m, l;     // of column g; l over this lane's tokens
  float c[2];     // sum of p (z + 8 s) over this lane's tokens, per group of dimensions
};

template <typename T>
__global__ void __launch_bounds__(kAttnThreads, 1) kv4_attn_kernel(const AttnParams P) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  AttnShared& sh = *reinterpret_cast<AttnShared*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int per_seq = P.pg.hkv * P.n_blk;  // groups of a sequence

  if (lane == 0)
    for (int s = 0; s < kStages; ++s) mbar_init(&sh.bar[warp][s], 1);
  fence_mbar_init();
  // chunks of each sequence (at least one, so that every group has a CTA)
  const int64_t cap = int64_t(P.pg.max_pages) * kKv4Page;
  if (warp == 0) {
    int64_t run = 0;
    for (int b0 = 0; b0 < P.batch; b0 += 32) {
      const int b = b0 + lane;
      int64_t n = 0;
      if (b < P.batch) {
        int64_t len = P.seq_len[b];
        if (len < 0 || len > cap) {
          if (blockIdx.x == 0) set_device_error(P.pg.status, DEV_BAD_LIST, b);
          len = len < 0 ? 0 : cap;
        }
        n = max(int64_t(1), (len + kChunkTokens - 1) / kChunkTokens) * per_seq;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(~0u, n, o);
        if (lane >= o) n += up;
      }
      if (b < P.batch) sh.before[b + 1] = run + n;
      run += __shfl_sync(~0u, n, 31);
    }
    if (lane == 0) sh.before[0] = 0;
  }
  __syncthreads();
  const int64_t total = sh.before[P.batch];
  const int n_cta = int(min(int64_t(gridDim.x), total));
  const int cta = blockIdx.x;
  if (cta >= n_cta) return;
  const int64_t u0 = total * cta / n_cta, u1 = total * (cta + 1) / n_cta;

  uint32_t done = 0;  // chunks this warp has taken off its ring, over all segments
  bool lost = false;  // a copy of this warp did not land in time
  int64_t u = u0;
  while (u < u1) {
    int b = 0;
    for (int step = 512; step > 0; step >>= 1)
      if (b + step < P.batch && sh.before[b + step] <= u) b += step;
    const int64_t len = max(int64_t(0), min(int64_t(P.seq_len[b]), cap));
    const int n_chunks = int((sh.before[b + 1] - sh.before[b]) / per_seq);
    const int64_t rel = u - sh.before[b];
    const int gi = int(rel / n_chunks);
    const int c0 = int(rel - int64_t(gi) * n_chunks);
    const int c1 = int(min(int64_t(n_chunks), c0 + (u1 - u)));
    const int blk = gi / P.pg.hkv, head = gi - blk * P.pg.hkv;
    const int cols = min(P.tpb, P.n_q - blk * P.tpb) * P.hpg;
    const int tok_g = blk * P.tpb + g / P.hpg;  // query token of column g
    const int64_t see = g < cols ? len - (P.n_q - 1 - tok_g) : 0;  // tokens column g sees

    // ring: this warp's k-th chunk of the segment is c0 + warp + 12 k
    const int mine = c1 - c0 > warp ? (c1 - c0 - warp + kAttnWarps - 1) / kAttnWarps : 0;
    auto issue = [&](int k) {  // lane 0
      const int ch = c0 + warp + k * kAttnWarps;
      const uint32_t st = (done + k) % kStages;
      const int64_t pos = int64_t(ch) * kChunkTokens;
      const uint8_t* src = pos < len && !lost ? P.pg.tile(b, head, pos) : nullptr;
      if (src) {
        mbar_arrive_expect_tx(&sh.bar[warp][st], kChunkBytes);
        bulk_g2s(sh.ring[warp][st], src, kChunkBytes, &sh.bar[warp][st]);
      } else {
        mbar_arrive(&sh.bar[warp][st]);  // nothing to copy: no token of the chunk counts
      }
      return src != nullptr;
    };
    uint32_t present = 0;  // bit k % 32: chunk k has a page
    if (lane == 0)
      for (int k = 0; k < min(mine, kStages); ++k)
        if (issue(k)) present |= 1u << (k & 31);

    // queries: A operand of the eight 16-dimension steps, upper half (rows 0-7) and,
    // for f16 input, what bf16 leaves of it (rows 8-15)
    uint32_t qa[8][2], ql[8][2];
    float qs[2] = {0.f, 0.f}, qsl[2] = {0.f, 0.f};
    constexpr bool kSplit = !std::is_same<T, __nv_bfloat16>::value;
    {
      const int h = head * P.hpg + g % P.hpg;
      const T* q = static_cast<const T*>(P.q) +
                   ((int64_t(b) * P.n_q + tok_g) * P.pg.hkv * P.hpg + h) * kHeadDim;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = (ks >> 2) * 64 + t * 16 + ((ks >> 1) & 1) * 8 + (ks & 1) * 2 + e;
          const float x0 = g < cols ? q_value(q + d) : 0.f;
          const float x1 = g < cols ? q_value(q + d + 4) : 0.f;
          const uint32_t w = pack_bf16(x0, x1);
          qa[ks][e] = w;
          qs[ks >> 2] += lo16(w) + hi16(w);
          if (kSplit) {
            const uint32_t wl = pack_bf16(x0 - lo16(w), x1 - hi16(w));
            ql[ks][e] = wl;
            qsl[ks >> 2] += lo16(wl) + hi16(wl);
          } else {
            ql[ks][e] = 0;
          }
        }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          qs[i] += __shfl_xor_sync(~0u, qs[i], o);
          qsl[i] += __shfl_xor_sync(~0u, qsl[i], o);
        }
    }

    WarpState S;
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) S.o[j][i] = 0.f;
    S.m = -INFINITY;
    S.l = S.c[0] = S.c[1] = 0.f;

    for (int k = 0; k < mine; ++k) {
      const uint32_t st = (done + k) % kStages;
      bool have = __shfl_sync(~0u, present, 0) >> (k & 31) & 1u;
      if (have && !lost &&
          !__all_sync(~0u, mbar_wait_parked(&sh.bar[warp][st], ((done + k) / kStages) & 1, kWaitNs))) {
        // a copy did not land: nothing more is copied or waited for by this warp, and
        // what is still in flight gets its time to land before the CTA may end
        if (lane == 0) set_device_error(P.pg.status, DEV_WAIT_TIMEOUT, 4);
        for (int j = k; j < min(mine, k + kStages); ++j)
          mbar_wait_parked(&sh.bar[warp][(done + j) % kStages], ((done + j) / kStages) & 1, kWaitNs);
        lost = true;
      }
      have = have && !lost;
      const int64_t pos = int64_t(c0 + warp + k * kAttnWarps) * kChunkTokens;
      const int seen = have ? int(min(int64_t(kChunkTokens), see - pos)) : 0;  // this column's
      const uint8_t* chunk = sh.ring[warp][st];

      float x[2][4];
#pragma unroll
      for (int ti = 0; ti < 2; ++ti) {
        const uint8_t* tile = chunk + ti * kKv4TileBytes;
        uint32_t kp[4][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(tile + kKv4Params + 32 * t + 16 * i);
          kp[2 * i][0] = w.x; kp[2 * i][1] = w.y; kp[2 * i + 1][0] = w.z; kp[2 * i + 1][1] = w.w;
        }
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          const uint4 kw = *reinterpret_cast<const uint4*>(tile + sub * 512 + lane * 16);
          const uint32_t w[4] = {kw.x, kw.y, kw.z, kw.w};
          float y[2] = {0.f, 0.f};
#pragma unroll
          for (int gr = 0; gr < 2; ++gr) {
            float acc[4] = {-128.f * qs[gr], -128.f * qs[gr], -128.f * qsl[gr], -128.f * qsl[gr]};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const int ks = gr * 4 + s;
              mma_bf16(acc, qa[ks][0], ql[ks][0], qa[ks][1], ql[ks][1],
                       codes(w[ks >> 1], (ks & 1) * 2), codes(w[ks >> 1], (ks & 1) * 2 + 1));
            }
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const uint32_t sz = kp[sub * 2 + o][gr];
              const float dot = kSplit ? acc[o] + acc[2 + o] : acc[o];
              y[o] += lo16(sz) * dot + hi16(sz) * (kSplit ? qs[gr] + qsl[gr] : qs[gr]);
            }
          }
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int row = ti * 16 + sub * 8 + 2 * t + o;
            x[ti][sub * 2 + o] = row < seen ? y[o] * P.scale_log2 : -INFINITY;
          }
        }
      }

      float mx = -INFINITY;
#pragma unroll
      for (int ti = 0; ti < 2; ++ti)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, x[ti][i]);
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
      if (__any_sync(~0u, mx > S.m)) {
        const float m1 = fmaxf(S.m, mx);
        const float f = S.m == -INFINITY ? 0.f : ex2(S.m - m1);
        S.m = m1;
        S.l *= f;
        S.c[0] *= f;
        S.c[1] *= f;
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) S.o[j][i] *= f;
      }
      const float m0 = S.m == -INFINITY ? 0.f : S.m;

#pragma unroll
      for (int ti = 0; ti < 2; ++ti) {
        const uint8_t* tile = chunk + ti * kKv4TileBytes;
        uint32_t a[2][4];  // per group of dimensions: upper and lower parts of p s
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          const uint4 w = *reinterpret_cast<const uint4*>(tile + kKv4Params + 128 + 32 * t + 16 * sub);
          const uint32_t vp[2][2] = {{w.x, w.y}, {w.z, w.w}};
          float ps[2][2];
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const float p = ex2(x[ti][sub * 2 + o] - m0);
            S.l += p;
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
              // a row that the column does not see may hold anything: take it as zero
              const uint32_t sz = ti * 16 + sub * 8 + 2 * t + o < seen ? vp[o][gr] : 0u;
              const float s = lo16(sz), z = hi16(sz);
              ps[gr][o] = p * s;
              S.c[gr] = fmaf(p, fmaf(8.f, s, z), S.c[gr]);
            }
          }
#pragma unroll
          for (int gr = 0; gr < 2; ++gr) {
            const uint32_t h = pack_bf16(ps[gr][0], ps[gr][1]);
            a[gr][2 * sub] = h;
            a[gr][2 * sub + 1] = pack_bf16(ps[gr][0] - lo16(h), ps[gr][1] - hi16(h));
          }
        }
        const uint4 v0 = *reinterpret_cast<const uint4*>(tile + kKv4V + lane * 16);
        const uint4 v1 = *reinterpret_cast<const uint4*>(tile + kKv4V + 512 + lane * 16);
        const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int j = 0; j < 16; ++j)
          mma_bf16(S.o[j], a[j >> 3][0], a[j >> 3][1], a[j >> 3][2], a[j >> 3][3],
                   centred(w0[j >> 2], j & 3), centred(w1[j >> 2], j & 3));
      }
      __syncwarp();
      if (lane == 0 && k + kStages < mine) {
        const bool ok = issue(k + kStages);
        const uint32_t bit = 1u << ((k + kStages) & 31);
        present = ok ? present | bit : present & ~bit;
      }
    }
    done += mine;

    // the warps' states into shared memory
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      S.l += __shfl_xor_sync(~0u, S.l, o);
      S.c[0] += __shfl_xor_sync(~0u, S.c[0], o);
      S.c[1] += __shfl_xor_sync(~0u, S.c[1], o);
    }
    if (t == 0) {
      sh.m[warp][g] = S.m;
      sh.l[warp][g] = S.l;
    }
#pragma unroll
    for (int gr = 0; gr < 2; ++gr)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const int j = gr * 8 + i;
          *reinterpret_cast<float4*>(&sh.o[warp][g][gr * 64 + t * 16 + e * 8 + i]) = make_float4(
              S.o[j][e] + S.o[j][2 + e] + S.c[gr], S.o[j + 1][e] + S.o[j + 1][2 + e] + S.c[gr],
              S.o[j + 2][e] + S.o[j + 2][2 + e] + S.c[gr],
              S.o[j + 3][e] + S.o[j + 3][2 + e] + S.c[gr]);
        }
    __syncthreads();
    if (tid < kCols) {
      float mx = -INFINITY, sum = 0.f;
      for (int w = 0; w < kAttnWarps; ++w) mx = fmaxf(mx, sh.m[w][tid]);
      for (int w = 0; w < kAttnWarps; ++w) {
        const float f = sh.m[w][tid] == -INFINITY ? 0.f : ex2(sh.m[w][tid] - mx);
        sh.w[w][tid] = f;
        sum += f * sh.l[w][tid];
      }
      sh.mx[tid] = mx;
      sh.sum[tid] = sum;
    }
    __syncthreads();

    const int64_t gs = sh.before[b] + int64_t(gi) * n_chunks, ge = gs + n_chunks;
    const bool whole = u0 <= gs && ge <= u1;
    const int64_t group = int64_t(b) * per_seq + gi;
    auto write_out = [&](int col, int d, float4 v, float mx, float sum) {
      const int tk = blk * P.tpb + col / P.hpg;
      const int64_t row = (int64_t(b) * P.n_q + tk) * P.pg.hkv * P.hpg + head * P.hpg + col % P.hpg;
      const float inv = sum != 0.f ? 1.f / sum : 0.f;
      *reinterpret_cast<float4*>(P.out + row * kHeadDim + d) =
          sum != 0.f ? make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
      if (d == 0 && P.lse) P.lse[row] = sum != 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
    };
    float* part = P.partials + (int64_t(cta) * 2 + (gs > u0 ? 1 : 0)) * kStateFloats;
    if (tid < kCols * kHeadDim / 4) {
      const int col = tid / (kHeadDim / 4), d = tid % (kHeadDim / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < kAttnWarps; ++w) {
        const float f = sh.w[w][col];
        const float4 x = *reinterpret_cast<const float4*>(&sh.o[w][col][d]);
        v.x += f * x.x; v.y += f * x.y; v.z += f * x.z; v.w += f * x.w;
      }
      if (whole) {
        if (col < cols) write_out(col, d, v, sh.mx[col], sh.sum[col]);
      } else {
        *reinterpret_cast<float4*>(part + col * kHeadDim + d) = v;
        if (d == 0) {
          part[kCols * kHeadDim + col] = sh.mx[col];
          part[kCols * kHeadDim + kCols + col] = sh.sum[col];
        }
      }
    }
    if (!whole) {
      // the CTAs of this group, in order of their pieces
      const int first = int(((gs + 1) * n_cta - 1) / total), last = int((ge * n_cta - 1) / total);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int n = atomicAdd(P.arrived + group, 1) + 1;
        sh.last = n == last - first + 1;
        if (sh.last) P.arrived[group] = 0;  // ready for the next call
      }
      __syncthreads();
      if (sh.last && tid < kCols * kHeadDim / 4) {
        __threadfence();
        const int col = tid / (kHeadDim / 4), d = tid % (kHeadDim / 4) * 4;
        auto slot = [&](int c) {
          return P.partials + (int64_t(c) * 2 + (gs > total * c / n_cta ? 1 : 0)) * kStateFloats;
        };
        float mx = -INFINITY, sum = 0.f;
        for (int c = first; c <= last; ++c) mx = fmaxf(mx, __ldcg(slot(c) + kCols * kHeadDim + col));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = first; c <= last; ++c) {
          const float* p = slot(c);
          const float m = __ldcg(p + kCols * kHeadDim + col);
          const float f = m == -INFINITY ? 0.f : ex2(m - mx);
          sum += f * __ldcg(p + kCols * kHeadDim + kCols + col);
          const float4 x = __ldcg(reinterpret_cast<const float4*>(p + col * kHeadDim + d));
          v.x += f * x.x; v.y += f * x.y; v.z += f * x.z; v.w += f * x.w;
        }
        if (col < cols) write_out(col, d, v, mx, sum);
      }
    }
    __syncthreads();  // the shared states are free again
    u += c1 - c0;
  }
}

int blocks_of(const sekv_config* cfg, int64_t n_q) {
  const int tpb = kCols / (cfg->n_q_heads / cfg->n_kv_heads);
  return int((n_q + tpb - 1) / tpb);
}

struct Kv4Ws {
  size_t arrived, partials, total;
};
Kv4Ws kv4_ws(const sekv_config* cfg, int64_t n_q, int sms) {
  Kv4Ws L{};
  L.arrived = 256;
  L.partials = L.arrived + align256(size_t(cfg->batch) * cfg->n_kv_heads * blocks_of(cfg, n_q) * 4);
  L.total = L.partials + align256(size_t(sms) * 2 * kStateFloats * 4);
  return L;
}

}  // namespace

namespace sekv {

size_t kv4_workspace_size(const sekv_config* cfg, int64_t n_q) {
  const int sms = device_sm_count();
  if (sms <= 0 || n_q < 1 || n_q > SEKV_MAX_QUERY_TOKENS || cfg->batch > SEKV_KV4_MAX_BATCH) return 0;
  return kv4_ws(cfg, n_q, sms).total;
}

sekv_status kv4_check(const sekv_config* cfg, const sekv_kv4_cache* cache, int n_q,
                      const void* workspace) {
  sekv_status why;
  if (!config_ok(cfg, &why)) return why;
  if (cfg->batch > SEKV_KV4_MAX_BATCH) return SEKV_ERR_UNSUPPORTED;
  if (n_q < 1 || n_q > SEKV_MAX_QUERY_TOKENS) return SEKV_ERR_UNSUPPORTED;
  if (!cache || !cache->pages || !cache->page_table || !workspace || cache->n_pages < 1 ||
      cache->max_pages < 1 || !aligned16(cache->pages) || !aligned16(workspace))
    return SEKV_ERR_INVALID;
  return SEKV_OK;
}

sekv_status kv4_check_ws(const sekv_config* cfg, int n_q, size_t workspace_bytes) {
  const int sms = device_sm_count();
  if (sms <= 0) return SEKV_ERR_CUDA;
  if (workspace_bytes < kv4_ws(cfg, n_q, sms).total) return SEKV_ERR_CAPACITY;
  return SEKV_OK;
}

}  // namespace sekv

extern "C" sekv_status sekv_kv4_attention(const sekv_config* cfg, const sekv_kv4_cache* cache,
                                          int32_t dtype, const void* q, int32_t n_q,
                                          const int32_t* seq_len, float scale, float* out,
                                          float* lse, void* workspace, size_t workspace_bytes,
                                          cudaStream_t stream) {
  reset_launches();
  sekv_status st = kv4_check(cfg, cache, n_q, workspace);
  if (st != SEKV_OK) return st;
  if (dtype != SEKV_BF16 && dtype != SEKV_F16) return SEKV_ERR_INVALID;
  if (!q || !seq_len || !out || !aligned16(q) || !aligned16(out) || !isfinite(scale))
    return SEKV_ERR_INVALID;
  st = kv4_check_ws(cfg, n_q, workspace_bytes);
  if (st != SEKV_OK) return st;
  const int sms = device_sm_count();
  const Kv4Ws L = kv4_ws(cfg, n_q, sms);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  AttnParams P{};
  P.pg.pages = static_cast<uint8_t*>(cache->pages);
  P.pg.table = cache->page_table;
  P.pg.status = reinterpret_cast<int32_t*>(w);
  P.pg.n_pages = cache->n_pages;
  P.pg.max_pages = cache->max_pages;
  P.pg.hkv = cfg->n_kv_heads;
  P.q = q;
  P.seq_len = seq_len;
  P.out = out;
  P.lse = lse;
  P.arrived = reinterpret_cast<int32_t*>(w + L.arrived);
  P.partials = reinterpret_cast<float*>(w + L.partials);
  P.batch = cfg->batch;
  P.hpg = cfg->n_q_heads / cfg->n_kv_heads;
  P.n_q = n_q;
  P.tpb = kCols / P.hpg;
  P.n_blk = blocks_of(cfg, n_q);
  P.scale_log2 = scale * kLog2e;
  const void* fn = dtype == SEKV_BF16 ? reinterpret_cast<const void*>(kv4_attn_kernel<__nv_bfloat16>)
                                      : reinterpret_cast<const void*>(kv4_attn_kernel<__half>);
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(AttnShared)) !=
      cudaSuccess) {
    cudaGetLastError();
    return SEKV_ERR_CUDA;
  }
  void* args[] = {&P};
  if (cudaLaunchKernel(fn, dim3(sms), dim3(kAttnThreads), args, sizeof(AttnShared), stream) !=
      cudaSuccess) {
    cudaGetLastError();
    return SEKV_ERR_CUDA;
  }
  count_launch(1);
  return SEKV_OK;
}
