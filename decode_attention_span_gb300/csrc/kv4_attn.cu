// sekv_kv4_attention: attention of a few query tokens over the 4-bit cache.
//
// 144 bytes per (token, KV head) are read once for all query heads of the group.
// The cache's layout is the matrix instructions' operand layout: a lane's codes come from
// shared memory as 16-byte words and become the A operand (tokens or dimensions in its 16 rows,
// the eight (token, head) columns in B) with one or two instructions per pair; no K or V value
// is rebuilt.  With
// K^ = z + s n for each group of 64 dimensions,
//   q . K^ = sum over groups of  s (sum_d q_d n_d) + z (sum_d q_d).
// Queries enter as f16, scaled by a power of two per column (exact for bf16 but for
// elements below 2^-23 of the column's largest).  Codes masked out of a word are f16 numbers
// below the normal ones as they stand: n 2^-24 from the low nibbles, n 2^-20 from the high ones
// (K's low ones are multiplied up to n 2^-14, for queries 2^-6 of the high ones').  For V,
//   sum_j p_j V^_j = sum_j +-(p_j s_j) n'_j + sum_j p_j z'_j,
// an even token with n' = n, z' = z and +, an odd one with n' = 15 - n, z' = z + 15 s and -:
// the mask's instruction inverts the odd tokens' codes too, and the sum of many tokens stays
// as small as it would with codes around zero.  The weight p_j s_j enters as the sum of two f16
// numbers (22 significant bits: one alone would cost the fp32 result 13 of its bits), scaled by
// a power of two, the unit of a column and a group of dimensions.  It follows the largest weight
// p_j s_j of that column and group, not the largest s: a token of large scale and no weight, or with
// weight in another column, takes no bits from the others.
//
// The matrix instructions take a number below the normal ones as if it were as large as those
// when they line their addends up, and cut off 25 bits under the largest.  So the place of
// a code in its f16 costs bits: shifted up by two, V's give an error of 2.4e-7 where n 2^-24
// gives 1.1e-6 (4 x 2000), and a query element counts in steps of 2^-19 of the column's largest
// (n 2^-24 for all of K: 2^-15, for 3% less time at 16 x 65536; K's high nibbles as normal
// numbers too: 3% more).
//
// Work: the cache is a line of chunks of 32 tokens (sequence by sequence, in
// it KV head by KV head), cut into equal pieces, one per CTA.  The warps of a CTA
// share a piece chunk by chunk, each with its own ring of bulk copies.  A CTA
// joins its warps' softmax states per (sequence, KV head) and, where that
// group spans several CTAs, leaves a partial; the last of them to finish joins
// the partials in order.
//
// What bounds it is waits for results, not memory and no single unit: a chunk takes a warp
// about 600 instructions (208 of them turn codes into operands), most of them in chains of fixed
// latency, and registers allow three warps per SM quarter, too few to hide those (issue 55%, ALU
// 46%, tensor 34%, DRAM 55% busy).  Measured, 16 sequences of up to 65536 tokens, 28 query
// and 4 KV heads (463 MB): 102.5 us, copies alone 76 us; one sequence of 131072, 32 and 8
// heads (151 MB): 39.5 us, copies alone 31 us, of which about 9 us move no data.  128-row
// tcgen05 tiles with these eight columns alone, and f16 operands by way of shared memory,
// would write and read 16 KB a chunk again at 128 bytes a clock: 256 clocks where a chunk now
// takes about 265 in all.
// e4m3 operands (a code's four bits in a byte are n 2^-9) need no arithmetic to make, but
// mma.sync converts them to f16 again: 53 us where f16 took 44.
#include <math.h>

#include <algorithm>

#include "kv4.cuh"

using namespace sekv;

namespace {

constexpr int kAttnWarps = 12;  // 168 registers; 8: 118 us where 12 take 102 and 15 (128 registers) 109
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kStages = 2;       // 3 are no faster: the copies are not what is waited for
constexpr int kChunkTokens = 32;
constexpr int kChunkBytes = 2 * kKv4TileBytes;
constexpr int kMaxCtas = 256;                    // of a launch
constexpr int kCols = 8;                         // (token, head) pairs of a block
constexpr int kStateFloats = kCols * (kHeadDim + 2);  // o, m, l
// What a second group costs a CTA (its plan, queries, first copies and join, about 6 us), in chunks
constexpr int kGroupCost = 40;
constexpr float kNone = -3e38f;
constexpr float kGrowth = 8.f;                   // log2 by which a weight may outgrow the reference
constexpr float kMaxScale = 128.f;               // of V with the unit: 2^8 times it fits f16
// A unit brings V's largest scale to 2^5 .. 2^6 unless the column's largest weight is then below
// kLeast, of which f16 takes 2^-25; it brings that weight to 2^5 .. 2^6 then.
constexpr float kLeast = 1.f, kMost = 4096.f;
constexpr int kUnitTop = 5;
constexpr uint32_t kUnitMax = 127 + 118;         // exponent: a weight of 2^8 fits fp32 with it
constexpr int kFlush = 16;                       // chunks between two flushes: 1% of the time
constexpr int kCodeBits = 20;                    // K's sums of q n are in units of 2^-20
constexpr uint64_t kWaitNs = 2000000000ull;

struct AttnShared {
  uint8_t ring[kAttnWarps][kStages][kChunkBytes];
  float o[kAttnWarps][kCols][kHeadDim];
  float4 par[kAttnWarps][2][kChunkTokens];  // a chunk's scales and zeros, K's and V's, as floats
  float m[kAttnWarps][kCols];
  float l[kAttnWarps][kCols];
  float4 units[kAttnWarps][32];    // powers of two on the weights: group 0 of a lane's columns, group 1
  float4 weights[kAttnWarps][32];  // the columns' largest weights, once they have units of their own
  float mx[kCols], sum[kCols];
  // the segment's queries: B operand, two 16-dimension steps a vector; per group of dimensions
  // the sums of q; from a column's units to log2 of its weights
  uint4 qb[4][32];
  float q_sum[2][kCols], q_scale[kCols];
  uint64_t bar[kAttnWarps][kStages];
  int before[SEKV_KV4_MAX_BATCH + 1];  // chunks (or pieces) before each sequence
  int len[SEKV_KV4_MAX_BATCH];         // tokens of each sequence
  int piece;                           // chunks of a piece, 0: pieces cross groups
  int last;
};
// The join of partials: kJoinParts sets of threads take every kJoinParts-th partial each.
constexpr int kJoinThreads = kCols * kHeadDim / 4 / 2;  // two float4 a thread
constexpr int kJoinParts = kAttnThreads / kJoinThreads;
constexpr int kFewPartials = 4;  // joined without shared memory
// scratch of the last CTA of a group, over the warps' values
struct JoinShared {
  float w[kMaxCtas][kCols];   // maxima, then weights
  float l[kMaxCtas][kCols];
  float4 part[kJoinParts - 1][2][kJoinThreads];
};
static_assert(sizeof(JoinShared) <= sizeof(AttnShared::o), "the join's scratch lies over the warps' values");

struct AttnParams {
  Kv4Pages pg;
  const void* q;
  const int32_t* seq_len;
  float *out, *lse;
  float* partials;   // [CTA][2][kStateFloats]
  int32_t* arrived;  // per group; zero between calls
  uint64_t wait_ns;  // of a warp for its next chunk
  int batch, hpg, n_q, tpb, n_blk;
  float scale_log2;
};

// D = A B + C in f16, 16 x 8 = 16 x 16 * 16 x 8 + 16 x 8
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
        "f"(c3));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  mma_f16(d, a, b0, b1, d[0], d[1], d[2], d[3]);
}
// (w & MASK) ^ bits in one instruction: the compiler makes two of the plain form, whose
// two constants do not fit one; `bits` stays in a register
template <uint32_t MASK>
__device__ __forceinline__ uint32_t mask_xor(uint32_t w, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(w), "n"(MASK), "r"(bits));
  return r;
}

// What h, a rounded pair, lacks of (w0, w1)
__device__ __forceinline__ __half2 rest(__half2 h, float w0, float w1) {
  float d0, d1;
  asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; sub.rn.f32.f16 %0, a, %3; sub.rn.f32.f16 %1, b, %4;}"
      : "=f"(d0), "=f"(d1)
      : "r"(*reinterpret_cast<const uint32_t*>(&h)), "f"(w0), "f"(w1));
  return __floats2half2_rn(-d0, -d1);
}

// 8x8 matrix of 16-bit values over the warp, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// The four pairs of a word of K's codes (pair i: codes i and i + 4) as f16 numbers: n 2^-14
// from the low nibbles of each byte (pairs 0 and 2), n 2^-20 from the high ones.
__device__ __forceinline__ void k_pairs(uint32_t w, uint32_t (&r)[4]) {
  const uint32_t w8 = w >> 8;
  r[0] = w & 0x000f000fu;
  r[1] = w & 0x00f000f0u;
  r[2] = w8 & 0x000f000fu;
  r[3] = w8 & 0x00f000f0u;
  const __half2 up = __half2half2(__ushort_as_half(0x6400));  // 2^10
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&r[i]), up);
    r[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
}
// V's: n 2^-22 and n 2^-18, the upper code of each pair, an odd token's, as 15 - n.
__device__ __forceinline__ void v_pairs(uint32_t w, uint32_t (&r)[4]) {
  const uint32_t w2 = w << 2, w6 = w >> 6;
  r[0] = mask_xor<0x003c003cu>(w2, 0x003c0000u);
  r[1] = mask_xor<0x03c003c0u>(w2, 0x03c00000u);
  r[2] = mask_xor<0x003c003cu>(w6, 0x003c0000u);
  r[3] = mask_xor<0x03c003c0u>(w6, 0x03c00000u);
}

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 2^x, to 2^-22 of its value; 0 for -infinity
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float q_value(__nv_bfloat16 q) { return __bfloat162float(q); }
__device__ __forceinline__ float q_value(__half q) { return __half2float(q); }

__device__ __forceinline__ int chunks_of(int len) {
  return max(1, (len + kChunkTokens - 1) / kChunkTokens);
}

// A warp's softmax state of one group.  A lane holds columns 2t and 2t + 1, and of
// the values dimensions 8g .. 8g + 7 of both groups of dimensions; l and c are sums
// over its own tokens (rows g and g + 8 of each tile).
struct WarpState {
  float o[8][4];   // [4 dims apiece: word m, i][rows g, g + 8 x columns], in units of 1 / unit
  float m[2], l[2];  // the weights' reference, log2: within 2^8 of the largest; kNone: no token yet
  float c[2][2];   // sum of p z': [column][group of dimensions]
  float most;      // the largest unit of any column and group of dimensions
  float least;     // what every column's largest weight with its unit is at least
  bool split;      // the columns and groups have units of their own
};

// The power of two that brings the number with these exponent bits to 2^kUnitTop .. twice that
__device__ __forceinline__ float unit_of(uint32_t exponent) {
  return __uint_as_float(uint32_t(min(max(2 * 127 + kUnitTop - int(exponent), 1), int(kUnitMax))) << 23);
}

// B operand, sums and scale of column `col` into shared memory, by one warp: q is this
// lane's four dimensions, 4 lane .. 4 lane + 3.
template <typename T>
__device__ __forceinline__ void put_queries(AttnShared& sh, const T (&q)[4], int col, int lane,
                                            float scale_log2) {
  float x[4], big = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = q_value(q[i]);
    big = fmaxf(big, fabsf(x[i]));
  }
  // 2^-7 of the sum, which large queries do not take past fp32 (exact for every bf16 and f16 number)
  float sum = (x[0] * 0.0078125f + x[2] * 0.0078125f) + (x[1] * 0.0078125f + x[3] * 0.0078125f);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    big = fmaxf(big, __shfl_xor_sync(~0u, big, o));
    if (o < 16) sum += __shfl_xor_sync(~0u, sum, o);  // the lower lanes: the first group
  }
  // power of two that brings the largest element to 2^13 .. 2^14 (less where it is below 2^-114)
  const int e = min(max(int(__float_as_uint(big) >> 23) - 127, -114), 127);
  const float up = __uint_as_float(uint32_t(127 + 13 - e) << 23);
  if ((lane & 15) == 0) {
    // an infinity among the queries makes the column NaN, as NaN does
    sh.q_sum[lane >> 4][col] = big < INFINITY ? sum * up / (1 << (kCodeBits - 7)) : NAN;
    const int f = 127 - 13 + kCodeBits + e, over = max(f - 254, 0);
    sh.q_scale[col] = scale_log2 * float(1 << over) * __uint_as_float(uint32_t(f - over) << 23);
  }
  // dimension d = 64 gr + 16 t + 8 w + i is in vector 2 gr + w of lane 4 col + t, half i / 4
  // of word i % 4; even dimensions meet low nibbles
  __half* dst = reinterpret_cast<__half*>(&sh.qb[(lane >> 4) * 2 + (lane >> 1 & 1)][col * 4 + (lane >> 2 & 3)]);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    dst[2 * i + (lane & 1)] = __float2half_rn(x[i] * (i & 1 ? up : up * 0.015625f));
}

// The segment's queries as a lane uses them: its columns are 2t and 2t + 1.  The B operand
// stays in shared memory: its sixteen registers are worth more to the rest (3% at 16 sequences of
// 65536).
struct Query {
  const uint4* b;      // [4][32], this lane's element of each
  float sum[2][2];     // [column][group]
  float scale_log2[2];
};

// The matrix instructions cut their sums off towards zero, which over hundreds of them adds
// up to more than fp32's rounding (16 x 65536: 3.5e-7 of
// the result, with flushes 1.8e-7; more where odd tokens weigh more than even ones or less).  So
// every kFlush chunks a warp adds its values to a second set in shared memory, rounded
// properly; eight 16-byte words a lane.
__device__ __forceinline__ void flush(WarpState& S, float4* kept, int lane, bool first) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float4 v = make_float4(S.o[j][0], S.o[j][1], S.o[j][2], S.o[j][3]);
    if (!first) {
      const float4 x = kept[j * 32 + lane];
      v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
    kept[j * 32 + lane] = v;
    S.o[j][0] = S.o[j][1] = S.o[j][2] = S.o[j][3] = 0.f;
  }
}
// k: on the values, of group 0 of the lane's columns, then of group 1
__device__ __noinline__ void rescale_kept(float4* kept, int lane, float4 k) {
  for (int j = 0; j < 8; ++j) {
    if (j == 4) k.x = k.z, k.y = k.w;
    float4 v = kept[j * 32 + lane];
    v.x *= k.x; v.y *= k.y; v.z *= k.x; v.w *= k.y;
    kept[j * 32 + lane] = v;
  }
}

// Units of their own for the columns and groups of dimensions, where scales lie far apart: by the
// chunk's largest scale as long as the column's largest weight is kLeast or more with that, and
// by that weight otherwise.  f: on the sums, as the reference moves; k: on the values.
__device__ __forceinline__ void split_units(WarpState& S, const Query& Q, const float (&x)[2][2][2],
                                            const float4* par, float by_scale,
                                            const float (&f)[2], float (&k)[2][2], float4& units,
                                            float4& weights, int g) {
  float* un = reinterpret_cast<float*>(&units);
  float* largest = reinterpret_cast<float*>(&weights);
  float w[2][2] = {{0.f, 0.f}, {0.f, 0.f}}, most = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = par[i * 8 + g];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float p = ex2(fmaf(x[i >> 1][i & 1][c], Q.scale_log2[c], -S.m[c]));
      w[0][c] = fmaxf(w[0][c], p * fabsf(v.x));  // NaN does not count
      w[1][c] = fmaxf(w[1][c], p * fabsf(v.z));
    }
  }
#pragma unroll
  for (int gr = 0; gr < 2; ++gr) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float old = un[2 * gr + c];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) w[gr][c] = fmaxf(w[gr][c], __shfl_xor_sync(~0u, w[gr][c], o));
      const float all = fmaxf(w[gr][c], f[c] * (S.split ? largest[2 * gr + c] : kLeast / old));
      float unit = fminf(old, by_scale);
      if (!(all * unit >= kLeast && all * unit < kMost)) unit = unit_of(__float_as_uint(all) >> 23);
      un[2 * gr + c] = unit;
      largest[2 * gr + c] = all;
      k[gr][c] = unit >= 1.f ? f[c] * unit / old : f[c] * (unit / old);  // in range in between, too
      most = fmaxf(most, unit);
    }
  }
  most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
  S.most = fmaxf(most, __shfl_xor_sync(~0u, most, 2));
  S.split = true;
}

// EDGE: some token of the chunk is not seen by some column (seen: per column of the
// lane; held: tokens of the chunk that the sequence has).  PACK: only four columns are in
// use; columns 4-7 hold the same queries again, and their lanes put the weights' lower
// parts in, so that one product does for both.
template <bool EDGE, bool PACK>
__device__ __forceinline__ void chunk_step(WarpState& S, const Query& Q, const uint8_t* chunk,
                                           float4 (&par)[2][kChunkTokens], float4* kept,
                                           float4* units, float4* weights, bool any_kept, int lane,
                                           int held, const int (&seen)[2]) {
  const int g = lane >> 2;
  // a lane turns one token's scales and zeros into floats for all
  const uint8_t* sz = chunk + (lane >> 4) * kKv4TileBytes + kv4_param(lane & 15, 0, false);
  const uint2 kp = *reinterpret_cast<const uint2*>(sz);
  uint2 vp = *reinterpret_cast<const uint2*>(sz + 128);
  if (EDGE && lane >= held) vp = make_uint2(0u, 0u);  // behind the end: may hold anything
  par[0][lane] = make_float4(lo16(kp.x), hi16(kp.x), lo16(kp.y), hi16(kp.y));
  const float s0 = lo16(vp.x), s1 = lo16(vp.y);
  __syncwarp();
  float x[2][2][2];  // tile, row half, column
#pragma unroll
  for (int ti = 0; ti < 2; ++ti) {
    const uint8_t* tile = chunk + ti * kKv4TileBytes;
    float acc[2][4];
    const uint4 k0 = *reinterpret_cast<const uint4*>(tile + lane * 16);
    const uint4 k1 = *reinterpret_cast<const uint4*>(tile + 512 + lane * 16);
    const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
    // the groups' chains of products take turns
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t r0[2][4], r1[2][4];
#pragma unroll
      for (int gr = 0; gr < 2; ++gr) {
        k_pairs(w0[2 * gr + i], r0[gr]);
        k_pairs(w1[2 * gr + i], r1[gr]);
      }
#pragma unroll
      for (int gr = 0; gr < 2; ++gr) {
        const uint32_t a[4] = {r0[gr][0], r1[gr][0], r0[gr][1], r1[gr][1]};
        const uint4 q = Q.b[(2 * gr + i) * 32];
        if (i == 0)
          mma_f16(acc[gr], a, q.x, q.y, 0.f, 0.f, 0.f, 0.f);
        else
          mma_f16(acc[gr], a, q.x, q.y);
      }
#pragma unroll
      for (int gr = 0; gr < 2; ++gr) {
        const uint32_t a[4] = {r0[gr][2], r1[gr][2], r0[gr][3], r1[gr][3]};
        const uint4 q = Q.b[(2 * gr + i) * 32];
        mma_f16(acc[gr], a, q.z, q.w);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float4 k = par[0][ti * 16 + e * 8 + g];  // s, z of both groups
      // both columns at once (2% at 16 sequences of 65536)
      Pair y = mul2(Pair(k.x, k.x), Pair(acc[0][2 * e], acc[0][2 * e + 1]));
      y = fma2(Pair(k.y, k.y), Pair(Q.sum[0][0], Q.sum[1][0]), y);
      y = fma2(Pair(k.z, k.z), Pair(acc[1][2 * e], acc[1][2 * e + 1]), y);
      y = fma2(Pair(k.w, k.w), Pair(Q.sum[0][1], Q.sum[1][1]), y);
      y.get(x[ti][e][0], x[ti][e][1]);
      if (EDGE)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (ti * 16 + e * 8 + g >= seen[c]) x[ti][e][c] = -INFINITY;
    }
  }

  {  // s, signed, and z'
    const float odd = lane & 1 ? 15.f : 0.f, sign = lane & 1 ? -1.f : 1.f;
    par[1][lane] = make_float4(s0 * sign, fmaf(odd, s0, hi16(vp.x)), s1 * sign, fmaf(odd, s1, hi16(vp.y)));
  }
  __syncwarp();
  // A new reference, or new units, only where the old ones may no longer do.
  float mx[2];
#pragma unroll
  for (int c = 0; c < 2; ++c)
    mx[c] = Q.scale_log2[c] * fmaxf(fmaxf(x[0][0][c], x[0][1][c]), fmaxf(x[1][0][c], x[1][1][c]));
  const bool over = mx[0] > S.m[0] + kGrowth || mx[1] > S.m[1] + kGrowth ||
                    fmaxf(s0, s1) * S.most >= kMaxScale;
  if (__any_sync(~0u, over)) {
    float f[2], k[2][2];  // k: on the values, [group][column]
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(~0u, mx[c], o));
      const float m1 = fmaxf(S.m[c], mx[c]);
      f[c] = ex2(S.m[c] - m1);
      S.m[c] = m1;
      S.l[c] *= f[c];
      S.c[c][0] *= f[c];
      S.c[c][1] *= f[c];
    }
    // One unit for all while that serves them: where a column's reference moves, a token of this
    // chunk has weight 1 in it, and so at least the chunk's smallest scale.
    const uint32_t t0 = vp.x & 0x7fffu, t1 = vp.y & 0x7fffu;
    const uint32_t top = __reduce_max_sync(~0u, max(t0 < 0x7f80u ? t0 : 0u, t1 < 0x7f80u ? t1 : 0u));
    const uint32_t low = __reduce_min_sync(~0u, EDGE && lane >= held ? 0x7f80u : min(t0, t1));
    const float by_scale = unit_of(top >> 7), unit = fminf(S.most, by_scale), ratio = unit / S.most;
    S.least = fminf(S.least * ratio, __uint_as_float(low << 16) * unit);
    if (!S.split && S.least >= kLeast) {
      S.most = unit;
      *units = make_float4(unit, unit, unit, unit);
      k[0][0] = k[1][0] = f[0] * ratio;
      k[0][1] = k[1][1] = f[1] * ratio;
    } else {
      split_units(S, Q, x, par[1], by_scale, f, k, *units, *weights, g);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) S.o[j][i] *= k[j >> 2][i & 1];
    if (any_kept) rescale_kept(kept, lane, make_float4(k[0][0], k[0][1], k[1][0], k[1][1]));
  }

  const float4 un = *units;
#pragma unroll
  for (int ti = 0; ti < 2; ++ti) {
    const uint8_t* tile = chunk + ti * kKv4TileBytes;
    uint32_t bh[2][2], bl[2][2];  // [group of dimensions][row half]: B operands, upper and lower part
    const float low = lane & 2 ? -1.f : 0.f;  // PACK: this lane's columns take the lower parts
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float4 v = par[1][ti * 16 + e * 8 + g];  // of both groups
      float p[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        p[c] = ex2(fmaf(x[ti][e][c], Q.scale_log2[c], -S.m[c]));
        S.l[c] += p[c];
      }
#pragma unroll
      for (int gr = 0; gr < 2; ++gr) {
        const float sv = gr ? v.z : v.x, z = gr ? v.w : v.y;
        float w[2];
        // in this order: a large s with the unit of a column without weight on it may overflow
        const Pair u(gr ? un.z : un.x, gr ? un.w : un.y);
        mul2(mul2(Pair(p[0], p[1]), u), Pair(sv, sv)).get(w[0], w[1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          // a token that the column does not see has p 0, but may hold NaN
          const bool ok = !EDGE || ti * 16 + e * 8 + g < seen[c];
          if (!ok) w[c] = 0.f;
          S.c[c][gr] = ok ? fmaf(p[c], z, S.c[c][gr]) : S.c[c][gr];
        }
        const __half2 h = __floats2half2_rn(w[0], w[1]);
        if (PACK) {
          const float2 hf = __half22float2(h);
          const __half2 part = __floats2half2_rn(fmaf(low, hf.x, w[0]), fmaf(low, hf.y, w[1]));
          bh[gr][e] = transpose8(*reinterpret_cast<const uint32_t*>(&part));
        } else {
          const __half2 l = rest(h, w[0], w[1]);
          bh[gr][e] = transpose8(*reinterpret_cast<const uint32_t*>(&h));
          bl[gr][e] = transpose8(*reinterpret_cast<const uint32_t*>(&l));
        }
      }
    }
    const uint4 v0 = *reinterpret_cast<const uint4*>(tile + kKv4V + lane * 16);
    const uint4 v1 = *reinterpret_cast<const uint4*>(tile + kKv4V + 512 + lane * 16);
    const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      uint32_t r0[4], r1[4];
      v_pairs(w0[m], r0);
      v_pairs(w1[m], r1);
      const uint32_t a0[4] = {r0[0], r0[2], r1[0], r1[2]}, a1[4] = {r0[1], r0[3], r1[1], r1[3]};
      mma_f16(S.o[2 * m], a0, bh[m >> 1][0], bh[m >> 1][1]);
      mma_f16(S.o[2 * m + 1], a1, bh[m >> 1][0], bh[m >> 1][1]);
      if (!PACK) {
        mma_f16(S.o[2 * m], a0, bl[m >> 1][0], bl[m >> 1][1]);
        mma_f16(S.o[2 * m + 1], a1, bl[m >> 1][0], bl[m >> 1][1]);
      }
    }
  }
}

template <typename T, bool PACK>
__global__ void __launch_bounds__(kAttnThreads, 1) kv4_attn_kernel(const AttnParams P) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  AttnShared& sh = *reinterpret_cast<AttnShared*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int per_seq = P.pg.hkv * P.n_blk;  // groups of a sequence

  if (lane == 0)
    for (int s = 0; s < kStages; ++s) mbar_init(&sh.bar[warp][s], 1);
  fence_mbar_init();
  follow_previous();
  // The plan, by one warp.  Chunks of each sequence (at least one, so that every group
  // has a CTA), then either every group cut into pieces of at most `piece` chunks, a CTA
  // each, or the line of all groups' chunks cut into equal pieces.
  const int cap = P.pg.max_pages * kKv4Page;
  if (warp == 0) {
    int sum = 0, longest = 1;
    for (int b = lane; b < P.batch; b += 32) {
      const int given = P.seq_len[b];
      const int len = min(max(given, 0), cap);
      if (given != len && blockIdx.x == 0) set_device_error(P.pg.status, DEV_BAD_LIST, b);
      sh.len[b] = len;
      sum += chunks_of(len);
      longest = max(longest, chunks_of(len));
    }
    sum = __reduce_add_sync(~0u, sum);
    longest = __reduce_max_sync(~0u, longest);
    __syncwarp();
    // as many CTAs for each group, if there are enough and its longest piece is not much
    // more than the line's share
    const int n_cta = int(gridDim.x), groups = P.batch * per_seq;
    int piece = 0;
    if (groups <= n_cta) {
      const int k = n_cta / groups, share = (sum * per_seq + n_cta - 1) / n_cta;
      piece = (longest + k - 1) / k;
      if (piece > share + kGroupCost) piece = 0;
    }
    int run = 0;
    for (int b0 = 0; b0 < P.batch; b0 += 32) {
      const int b = b0 + lane;
      int n = 0;
      if (b < P.batch) {
        n = chunks_of(sh.len[b]);
        if (piece > 0) n = (n + piece - 1) / piece;
        n *= per_seq;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(~0u, n, o);
        if (lane >= o) n += up;
      }
      if (b < P.batch) sh.before[b + 1] = run + n;
      run += __shfl_sync(~0u, n, 31);
    }
    if (lane == 0) {
      sh.before[0] = 0;
      sh.piece = piece;
    }
  }
  __syncthreads();
  const bool by_piece = sh.piece > 0;
  const int total = sh.before[P.batch];
  const int n_cta = min(int(gridDim.x), total);
  const int cta = blockIdx.x;
  if (cta >= n_cta) return;
  // CTA c's share of the line: [start(c), start(c + 1)), start(c) = total * c / n_cta (by
  // piece: total == n_cta, and the units of the line are the pieces)
  const int each = total / n_cta, over = total - each * n_cta;
  auto start = [&](int c) { return each * c + over * c / n_cta; };
  const int u0 = start(cta), u1 = start(cta + 1);
  auto cta_of = [&](int u) {  // whose share unit u is in: an estimate, and its correction
    int c = max(0, min(n_cta - 1, int(float(u) * (float(n_cta) / float(total)))));
    while (start(c) > u) --c;
    while (start(c + 1) <= u) ++c;
    return c;
  };

  uint32_t done = 0;  // chunks this warp has taken off its ring, over all segments
  bool lost = false;  // a copy of this warp did not land in time
  int u = u0, b = 0;
  while (u < u1) {
    for (;;) {  // the sequence of chunk u: the last one that starts at or before it
      const int i = b + 1 + lane;
      const int n = __popc(__ballot_sync(~0u, i < P.batch && sh.before[i] <= u));
      b += n;
      if (n < 32) break;
    }
    const int len = sh.len[b];
    const int n_units = (sh.before[b + 1] - sh.before[b]) / per_seq;  // of a group
    const int rel = u - sh.before[b];
    const int gi = rel / n_units;
    const int i0 = rel - gi * n_units, i1 = min(n_units, i0 + (u1 - u));
    // this segment's chunks of the group
    int c0 = i0, c1 = i1;
    if (by_piece) {  // n_units is at most the number of CTAs: no product overflows
      const int n = chunks_of(len), q = n / n_units, r = n - q * n_units;
      c0 = q * i0 + r * i0 / n_units;
      c1 = q * i1 + r * i1 / n_units;
    }
    const int blk = gi / P.pg.hkv, head = gi - blk * P.pg.hkv;
    const int cols = min(P.tpb, P.n_q - blk * P.tpb) * P.hpg;

    // The queries: warp w brings column w.
    union {
      uint2 w;
      T e[4];
    } qv;
    qv.w = make_uint2(0, 0);
    const int qcol = PACK ? warp & 3 : warp;
    if (warp < kCols && qcol < cols) {
      const int tok = blk * P.tpb + qcol / P.hpg;
      const T* q = static_cast<const T*>(P.q) +
                   ((int64_t(b) * P.n_q + tok) * P.pg.hkv * P.hpg + head * P.hpg + qcol % P.hpg) *
                       kHeadDim;
      // volatile: the compiler would move a plain load down to its use, behind the copies; not
      // .nc: this grid may be resident while the kernel before it still writes the queries
      asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(qv.w.x), "=r"(qv.w.y) : "l"(q + 4 * lane));
    }

    // This warp's k-th chunk of the segment is c0 + warp + kAttnWarps k.  Lane i
    // looks up the page of chunk 32 j + i; -1 where there is none to copy.
    const int mine = c1 - c0 > warp ? (c1 - c0 - warp + kAttnWarps - 1) / kAttnWarps : 0;
    auto lookup = [&](int k) {
      const int pos = (c0 + warp + k * kAttnWarps) * kChunkTokens;
      if (k >= mine || pos >= len) return -1;
      const int id = P.pg.table[int64_t(b) * P.pg.max_pages + pos / kKv4Page];
      if (id >= 0 && id < P.pg.n_pages) return id;
      set_device_error(P.pg.status, DEV_BAD_LIST, b);
      return -1;
    };
    int ids = lookup(lane), ids_next = lookup(32 + lane);
    uint32_t present = 0;  // bit k % 32: chunk k is in the ring
    auto issue = [&](int k) {
      if (k > 0 && (k & 31) == 0) {
        ids = ids_next;
        ids_next = lookup(k + 32 + lane);
      }
      const int id = lost ? -1 : __shfl_sync(~0u, ids, k & 31);
      const uint32_t bit = 1u << (k & 31);
      present = id >= 0 ? present | bit : present & ~bit;
      if (lane == 0) {
        const uint32_t st = (done + k) % kStages;
        if (id >= 0) {
          const int ch = c0 + warp + k * kAttnWarps;
          mbar_arrive_expect_tx(&sh.bar[warp][st], kChunkBytes);
          bulk_g2s(sh.ring[warp][st],
                   P.pg.pages + (int64_t(id) * P.pg.hkv + head) * kKv4PageBytes +
                       (ch & (kKv4Page / kChunkTokens - 1)) * kChunkBytes,
                   kChunkBytes, &sh.bar[warp][st]);
        } else {
          mbar_arrive(&sh.bar[warp][st]);  // nothing to copy: no token of the chunk counts
        }
      }
    };

    if (warp < kCols) put_queries<T>(sh, qv.e, warp, lane, P.scale_log2);
    __syncthreads();
    Query Q;
    int see[2];  // tokens that columns 2t and 2t + 1 see
    Q.b = &sh.qb[0][lane];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = 2 * t + c;
#pragma unroll
      for (int gr = 0; gr < 2; ++gr) {
        Q.sum[c][gr] = sh.q_sum[gr][col];
      }
      Q.scale_log2[c] = sh.q_scale[col];
      const int real = PACK ? col & 3 : col;
      see[c] = real < cols ? len - (P.n_q - 1 - (blk * P.tpb + real / P.hpg)) : 0;
    }
    // up to here no token is hidden from any column in use
    const int open = len - (P.n_q - 1 - blk * P.tpb);

    // the first copies; the queries' shuffles above do not wait behind them
    for (int k = 0; k < min(mine, kStages); ++k) issue(k);

    WarpState S;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) S.o[j][i] = 0.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      S.m[c] = kNone;
      S.l[c] = S.c[c][0] = S.c[c][1] = 0.f;
    }
    S.most = __uint_as_float(kUnitMax << 23);
    S.least = INFINITY;
    S.split = false;
    sh.units[warp][lane] = make_float4(S.most, S.most, S.most, S.most);

    float4* kept = reinterpret_cast<float4*>(&sh.o[warp][0][0]);
    for (int k = 0; k < mine; ++k) {
      const uint32_t st = (done + k) % kStages;
      if ((present >> (k & 31) & 1u) && !lost) {
        if (__all_sync(~0u, mbar_wait_parked(&sh.bar[warp][st], ((done + k) / kStages) & 1, P.wait_ns))) {
          const int pos = (c0 + warp + k * kAttnWarps) * kChunkTokens;
          const int held = len - pos;
          const int seen[2] = {see[0] - pos, see[1] - pos};
          float4 *un = &sh.units[warp][lane], *wt = &sh.weights[warp][lane];
          if (pos + kChunkTokens <= open)
            chunk_step<false, PACK>(S, Q, sh.ring[warp][st], sh.par[warp], kept, un, wt, k >= kFlush, lane, held, seen);
          else
            chunk_step<true, PACK>(S, Q, sh.ring[warp][st], sh.par[warp], kept, un, wt, k >= kFlush, lane, held, seen);
        } else {
          // a copy did not land: nothing more is copied or waited for by this warp, and
          // what is still in flight gets its time to land before the CTA may end
          if (lane == 0) set_device_error(P.pg.status, DEV_WAIT_TIMEOUT, 4);
          for (int j = k; j < min(mine, k + kStages); ++j)
            mbar_wait_parked(&sh.bar[warp][(done + j) % kStages], ((done + j) / kStages) & 1, kWaitNs);
          lost = true;
        }
      }
      __syncwarp();
      if (k + kStages < mine) issue(k + kStages);
      if (k % kFlush == kFlush - 1) flush(S, kept, lane, k < kFlush);
    }
    done += mine;
    if (mine >= kFlush) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 x = kept[j * 32 + lane];
        S.o[j][0] += x.x; S.o[j][1] += x.y; S.o[j][2] += x.z; S.o[j][3] += x.w;
      }
      __syncwarp();  // the state goes where the kept values were
    }

    // the warps' states into shared memory (PACK: the lower parts' sums as columns 4-7)
    const float* un = reinterpret_cast<const float*>(&sh.units[warp][lane]);
    const float low = float(1 << 22), high = float(1 << 18);
#pragma unroll 1
    for (int o = 4; o < 32; o <<= 1)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        S.l[c] += __shfl_xor_sync(~0u, S.l[c], o);
        S.c[c][0] += __shfl_xor_sync(~0u, S.c[c][0], o);
        S.c[c][1] += __shfl_xor_sync(~0u, S.c[c][1], o);
      }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (g == 0) {
        sh.m[warp][2 * t + c] = S.m[c];
        sh.l[warp][2 * t + c] = S.l[c];
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float add = PACK && t >= 2 ? 0.f : S.c[c][m >> 1], inv_unit = 1.f / un[(m >> 1) * 2 + c];
        *reinterpret_cast<float4*>(&sh.o[warp][2 * t + c][(m >> 1) * 64 + g * 8 + (m & 1) * 4]) =
            make_float4(fmaf(S.o[2 * m][c] * low, inv_unit, add), fmaf(S.o[2 * m + 1][c] * high, inv_unit, add),
                        fmaf(S.o[2 * m][2 + c] * low, inv_unit, add),
                        fmaf(S.o[2 * m + 1][2 + c] * high, inv_unit, add));
      }
    }
    __syncthreads();

    const int gs = sh.before[b] + gi * n_units, ge = gs + n_units;
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
    if (warp < (PACK ? kCols / 2 : kCols)) {  // warp: a column, lane: four of its dimensions
      const int col = warp, d = 4 * lane;
      const float m = lane < kAttnWarps ? sh.m[lane][col] : kNone;
      float mx = m;
#pragma unroll 1
      for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
      mx = __shfl_sync(~0u, mx, 0);
      const float f = ex2(m - mx);
      float sum = lane < kAttnWarps ? f * sh.l[lane][col] : 0.f;
#pragma unroll 1
      for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
      sum = __shfl_sync(~0u, sum, 0);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int w = 0; w < kAttnWarps; ++w) {
        const float fw = __shfl_sync(~0u, f, w);
        float4 x = *reinterpret_cast<const float4*>(&sh.o[w][col][d]);
        if (PACK) {
          const float4 y = *reinterpret_cast<const float4*>(&sh.o[w][col + kCols / 2][d]);
          x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
        }
        v.x = fmaf(fw, x.x, v.x); v.y = fmaf(fw, x.y, v.y);
        v.z = fmaf(fw, x.z, v.z); v.w = fmaf(fw, x.w, v.w);
      }
      if (col < cols) {
        if (whole) {
          write_out(col, d, v, mx, sum);
        } else {
          *reinterpret_cast<float4*>(part + col * kHeadDim + d) = v;
          if (lane == 0) {
            part[kCols * kHeadDim + col] = mx;
            part[kCols * kHeadDim + kCols + col] = sum;
          }
        }
      }
    }
    if (!whole) {
      // the CTAs of this group, in order of their pieces
      const int first = cta_of(gs), n = cta_of(ge - 1) - first + 1;
      __syncthreads();
      if (tid == 0) {
        // releases the CTA's partial (ordered before by the barrier), acquires the others'
        int before;
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                     : "=r"(before)
                     : "l"(P.arrived + group)
                     : "memory");
        sh.last = before == n - 1;
        if (sh.last) P.arrived[group] = 0;  // ready for the next call
      }
      __syncthreads();
      auto slot = [&](int i) {
        return P.partials + (int64_t(first + i) * 2 + (gs > start(first + i) ? 1 : 0)) * kStateFloats;
      };
      if (sh.last && n <= kFewPartials) {
        // each thread on its own: two loads deep and no barrier
        if (tid < cols * kHeadDim / 4) {
          const int col = tid / (kHeadDim / 4);
          float m[kFewPartials], l[kFewPartials];
          float4 x[kFewPartials];
#pragma unroll
          for (int i = 0; i < kFewPartials; ++i) {
            m[i] = kNone;
            if (i < n) {
              const float* p = slot(i);
              m[i] = __ldcg(p + kCols * kHeadDim + col);
              l[i] = __ldcg(p + kCols * kHeadDim + kCols + col);
              x[i] = __ldcg(reinterpret_cast<const float4*>(p) + tid);
            }
          }
          float mx = m[0], sum = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int i = 1; i < kFewPartials; ++i) mx = fmaxf(mx, m[i]);
#pragma unroll
          for (int i = 0; i < kFewPartials; ++i)
            if (i < n) {
              const float f = ex2(m[i] - mx);
              sum = fmaf(f, l[i], sum);
              v.x = fmaf(f, x[i].x, v.x); v.y = fmaf(f, x[i].y, v.y);
              v.z = fmaf(f, x[i].z, v.z); v.w = fmaf(f, x[i].w, v.w);
            }
          write_out(col, tid % (kHeadDim / 4) * 4, v, mx, sum);
        }
      } else if (sh.last) {
        JoinShared& jn = *reinterpret_cast<JoinShared*>(&sh.o[0][0][0]);
        for (int i = tid; i < n * kCols; i += kAttnThreads) {
          const float* p = slot(i / kCols) + kCols * kHeadDim + i % kCols;
          jn.w[i / kCols][i % kCols] = __ldcg(p);
          jn.l[i / kCols][i % kCols] = __ldcg(p + kCols);
        }
        __syncthreads();
        static_assert(kAttnWarps >= kCols, "a warp per column");
        if (warp < kCols) {
          float mx = kNone, sum = 0.f;
          for (int i = lane; i < n; i += 32) mx = fmaxf(mx, jn.w[i][warp]);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
          for (int i = lane; i < n; i += 32) {
            const float f = ex2(jn.w[i][warp] - mx);
            jn.w[i][warp] = f;
            sum += f * jn.l[i][warp];
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
          if (lane == 0) {
            sh.mx[warp] = mx;
            sh.sum[warp] = sum;
          }
        }
        __syncthreads();
        const int at = tid % kJoinThreads, set = tid / kJoinThreads;
        float4 v[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 4
        for (int i = set; i < n; i += kJoinParts) {
          const float4* p = reinterpret_cast<const float4*>(slot(i));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float f = jn.w[i][(at + h * kJoinThreads) / (kHeadDim / 4)];
            const float4 x = __ldcg(p + at + h * kJoinThreads);
            v[h].x = fmaf(f, x.x, v[h].x); v[h].y = fmaf(f, x.y, v[h].y);
            v[h].z = fmaf(f, x.z, v[h].z); v[h].w = fmaf(f, x.w, v[h].w);
          }
        }
        if (set > 0)
          for (int h = 0; h < 2; ++h) jn.part[set - 1][h][at] = v[h];
        __syncthreads();
        if (set == 0) {
          for (int h = 0; h < 2; ++h) {
            for (int k = 0; k < kJoinParts - 1; ++k) {
              const float4 x = jn.part[k][h][at];
              v[h].x += x.x; v[h].y += x.y; v[h].z += x.z; v[h].w += x.w;
            }
            const int f4 = at + h * kJoinThreads, col = f4 / (kHeadDim / 4);
            if (col < cols) write_out(col, f4 % (kHeadDim / 4) * 4, v[h], sh.mx[col], sh.sum[col]);
          }
        }
      }
    }
    __syncthreads();  // the shared states are free again
    u += i1 - i0;
  }
}

int blocks_of(const sekv_config* cfg, int64_t n_q) {
  const int tpb = kCols / (cfg->n_q_heads / cfg->n_kv_heads);
  return int((n_q + tpb - 1) / tpb);
}

int attn_ctas() { return std::min(device_sm_count(), kMaxCtas); }  // one per SM

struct Kv4Ws {
  size_t partials, arrived, total;
};
Kv4Ws kv4_ws(const sekv_config* cfg, int64_t n_q, int sms) {
  // the counters last: where they begin is the same whatever batch and n_q a call has, so
  // that calls of different sizes can take turns on a workspace
  Kv4Ws L{};
  L.partials = 256;
  L.arrived = L.partials + align256(size_t(sms) * 2 * kStateFloats * 4);
  L.total = L.arrived + align256(size_t(cfg->batch) * cfg->n_kv_heads * blocks_of(cfg, n_q) * 4);
  return L;
}

}  // namespace

namespace sekv {

size_t kv4_workspace_size(const sekv_config* cfg, int64_t n_q) {
  const int sms = attn_ctas();
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
  const int sms = attn_ctas();
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
  if (!q || !seq_len || !out || !aligned16(q) || !aligned16(out) ||
      !isfinite(scale * kLog2e) || !(scale > 0.f))
    return SEKV_ERR_INVALID;
  // the kernel numbers tokens and chunks in 32 bits
  if (cache->max_pages >= 1 << 24 ||
      int64_t(cfg->batch) * cfg->n_kv_heads * blocks_of(cfg, n_q) * cache->max_pages >= 1 << 29)
    return SEKV_ERR_UNSUPPORTED;
  st = kv4_check_ws(cfg, n_q, workspace_bytes);
  if (st != SEKV_OK) return st;
  const int sms = attn_ctas();
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
  P.wait_ns = (cfg->flags & SEKV_FLAG_SHORT_WAITS) ? 0 : kWaitNs;
  P.batch = cfg->batch;
  P.hpg = cfg->n_q_heads / cfg->n_kv_heads;
  P.n_q = n_q;
  P.tpb = kCols / P.hpg;
  P.n_blk = blocks_of(cfg, n_q);
  P.scale_log2 = scale * kLog2e;
  const bool pack = n_q * P.hpg <= kCols / 2;
  void (*const fns[4])(AttnParams) = {
      kv4_attn_kernel<__nv_bfloat16, false>, kv4_attn_kernel<__half, false>,
      kv4_attn_kernel<__nv_bfloat16, true>, kv4_attn_kernel<__half, true>};
  void (*const fn)(AttnParams) = fns[(dtype == SEKV_BF16 ? 0 : 1) + (pack ? 2 : 0)];
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(AttnShared)) !=
      cudaSuccess) {
    cudaGetLastError();
    return SEKV_ERR_CUDA;
  }
  return launch_following(fn, dim3(sms), kAttnThreads, sizeof(AttnShared), stream, P);
}
