// sekv_kv4_tree_attention for many (token, head) columns: 128 of them side by side on the fifth
// generation's tensor cores, one pass over the cache for all.
//
// Mathematics.  A group's values z + s n (n 0 .. 15) are z' + s n' with n' = n - 8 and z' = z + 8 s.  s has
// eight significant bits and n' three (or is -8), so s n' is an f16 number exactly, up to a power of two:
//   q . K^ = g_t (sum_d q_d k'_d) + sum over groups of z' (sum_d q_d),    k' = s n' / g_t
//   sum_t p_t V^_t = sum_t (p_t f_t) v'_t + sum_t p_t z'_t,               v' = s n' / f_t
// with g_t and f_t powers of two that bring a token's larger scale to 2^kTop .. twice that (the smaller one
// stays exact down to 2^-25 of it).  The weights p_t f_t u enter as the sum of two f16 numbers (22
// bits); u is a power of two for each column, moved where its largest weight would leave f16's range: no token
// takes bits from the others by the size of its values alone.
//
// Sixteen warps.  Two streams take every other page each: four softmax warps (a lane quadrant of tensor memory
// each, both halves of a page in turn) and one that issues the stream's products; the tensor cores work for one
// stream while the other's weights are made.  Four warps turn codes into operands, one a page's scales into floats, one
// copies pages.  The logits of two pages a stream are multiplied ahead.  A softmax thread has four rows and eight
// tokens of a half page: a scale read from shared memory
// serves four weights.
//
// What bounds it is taken to be the softmax warps' chains of dependent instructions, two such warps to an SM
// quarter (issue 49% of active cycles, tensor pipe 23%, DRAM 11%: 65536 tokens, 32 drafted).
// 131072 tokens, 32 and 8 heads, 64 drafted tokens (two blocks of columns): 331 us; 8 sequences of up to
// 16384, 28 and 4 heads, 26 drafted: 158 us.  Leaving parts out of copies of it that gave wrong results (when the whole took
// 326 to 352 us): code expansion 315 us, expansion and scales 306, softmax 271, softmax and expansion 195; none hides the
// others entirely.  Steps: logits kept in registers 715 us, in tensor memory 426; half pages in turn and
// products issued by whole warps 352; scales folded into the operands 339; a warp for the scales 326.  The
// flushes cost 308 -> 331.
#include <math.h>

#include <algorithm>

#include "kv4.cuh"
#include "kv4_tree.h"
#include "tc.cuh"

using namespace sekv;

namespace {

constexpr int kRaw = 4;         // pages on their way
constexpr int kKeys = 3;        // pages' keys as operands, and values
constexpr int kVals = 5;
constexpr int kSoftWarps = 8;   // two streams of four
constexpr int kCodeWarps = 4;
constexpr int kTreeThreads = (kSoftWarps + kCodeWarps + 4) * 32;  // and copies, scales, a stream's products each
constexpr int kGroupBytes = kKv4Page * 128;      // an operand of one group: 64 tokens x 64 dimensions f16
constexpr int kOpBytes = 2 * kGroupBytes;
constexpr int kTop = 8;
constexpr int kHalfPage = 32;                    // tokens that a stream takes at a time
constexpr int kStreamColumns = 256;              // tensor memory of a stream: two pages' logits or weights, 64 columns each, and the values
constexpr int kValues = 128;                     // from here on
// Pages of a stream between two flushes, of 128 additions in tensor memory.  Those cut off towards zero: values that
// all point one way were off by 2^-17.6 of their size after 32 pages and 2^-13.6 after 500, with flushes 2^-18.7 after
// any number.  A flush takes some 3 us, its wait for the products among them (131072 tokens 308 -> 332 us).
constexpr int kFlush = 16;
constexpr int kItemCost = 8;                     // what an item costs beyond its pages, in pages
constexpr float kNone = -3e38f;
constexpr float kGrowth = 8.f;
constexpr float kMaxScale = 128.f;      // of V with the unit: 2^8 times it fits f16
constexpr float kLeast = 1.f, kMost = 4096.f;
constexpr int kUnitTop = 5;             // a unit brings what it is made for to 2^5 .. 2^6
constexpr uint32_t kUnitMax = 127 + 118;
constexpr uint64_t kTreeWaitNs = 2000000000ull;

// Of tokens 2 i and 2 i + 1, keys (k) and values (v): the powers of two and z' of the first group (a), z' of
// the second (b)
struct PageParams {
  float4 ka[kKv4Page / 2], va[kKv4Page / 2];
  float2 kb[kKv4Page / 2], vb[kKv4Page / 2];
  int top[2], low[2];  // exponents of the largest and the smallest f of 32 tokens
  int held;            // tokens of the page that the sequence has
};

struct __align__(1024) TreeShared {
  uint8_t q[2][kTreeRows * 128];  // the columns' queries: a group of dimensions each
  uint8_t key[kKeys][kOpBytes];
  uint8_t val[kVals][kOpBytes];
  uint8_t raw[kRaw][kKv4PageBytes];
  uint4 scale[kRaw][kKv4Page];  // of a token: K's two groups, V's two, each twice as f16
  PageParams par[kVals];
  float4 q_sum[kTreeRows];  // of the two groups, each twice
  float q_scale[kTreeRows];
  float m[2][kTreeRows], l[2][kTreeRows];  // the streams'
  uint64_t raw_full[kRaw], raw_empty[kRaw], scaled[kRaw], k_full[kKeys], k_empty[kKeys], v_full[kVals], v_empty[kVals];
  uint64_t s_full[2][2], p_full[2][2][2], v_done[2][2][2], o_full, drained[2];
  uint32_t tmem;
  int raw_held[kRaw];
  TreePlan plan;
};
static_assert(sizeof(TreeShared) + 1024 <= 227 * 1024, "shared memory of a CTA");
static_assert(kVals * kOpBytes >= kTreeRows * kHeadDim * 4, "the streams' values lie over the operands");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float q_value(__nv_bfloat16 q) { return __bfloat162float(q); }
__device__ __forceinline__ float q_value(__half q) { return __half2float(q); }
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// What h, a rounded pair, lacks of (w0, w1)
__device__ __forceinline__ uint32_t rest(__half2 h, float w0, float w1) {
  float d0, d1;
  asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; add.rn.f32.f16 %0, a, %3; add.rn.f32.f16 %1, b, %4;}"
      : "=f"(d0), "=f"(d1)
      : "r"(bits(h) ^ 0x80008000u), "f"(w0), "f"(w1));
  return bits(__floats2half2_rn(d0, d1));
}

// (w & MASK) | bits in one instruction: the compiler makes two of it, for its two constants
template <uint32_t MASK>
__device__ __forceinline__ __half2 mask_or(uint32_t w, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "n"(MASK), "r"(bits));
  return *reinterpret_cast<const __half2*>(&r);
}
// Eight codes of a word as f16 numbers (n - 8) s, in the order 0, 4, 1, 5, 2, 6, 3, 7
__device__ __forceinline__ uint4 codes(uint32_t w, uint32_t scale) {
  const uint32_t magic = 0x64006400u;  // 1024: a code in the lowest bits adds itself, one above 16 times
  const uint32_t w8 = w >> 8;
  const __half2 less = __float2half2_rn(-1032.f), sixteenth = __float2half2_rn(0.0625f), less16 = __float2half2_rn(-72.f);
  const __half2 s = *reinterpret_cast<const __half2*>(&scale);
  return make_uint4(bits(__hmul2(__hadd2(mask_or<0x000f000fu>(w, magic), less), s)),
                    bits(__hmul2(__hfma2(mask_or<0x00f000f0u>(w, magic), sixteenth, less16), s)),
                    bits(__hmul2(__hadd2(mask_or<0x000f000fu>(w8, magic), less), s)),
                    bits(__hmul2(__hfma2(mask_or<0x00f000f0u>(w8, magic), sixteenth, less16), s)));
}
// A token's scales (bf16 s, z of both groups) over a power of two, whose exponent is returned (1 .. 253).  What
// is not finite, or not there, counts as 0: its z' is not finite either.
__device__ __forceinline__ int scales(uint2 w, bool there, uint32_t& s0, uint32_t& s1) {
  uint32_t b0 = w.x & 0xffffu, b1 = w.y & 0xffffu;
  if (!there || (b0 & 0x7fffu) >= 0x7f80u) b0 = 0;
  if (!there || (b1 & 0x7fffu) >= 0x7f80u) b1 = 0;
  const int up = min(254 + kTop - int(max(b0 & 0x7fffu, b1 & 0x7fffu) >> 7), 253);
  const float by = __uint_as_float(uint32_t(up) << 23);
  s0 = bits(__float2half2_rn(__uint_as_float(b0 << 16) * by));
  s1 = bits(__float2half2_rn(__uint_as_float(b1 << 16) * by));
  return 254 - up;
}
// Byte of 16-byte piece c of row r in an operand
__device__ __forceinline__ uint32_t piece_at(int r, int c) { return uint32_t(r * 128 + ((c ^ (r & 7)) << 4)); }

// One page's scales, by a warp: `held`, its tokens
__device__ __forceinline__ void expand_scales(const uint8_t* raw, uint4* scale, PageParams& par, int held, int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = i * 32 + lane;
    const uint8_t* sz = raw + j / 16 * kKv4TileBytes + kv4_param(j % 16, 0, false);
    uint2 k = *reinterpret_cast<const uint2*>(sz), v = *reinterpret_cast<const uint2*>(sz + 128);
    const bool there = j < held;
    if (!there) k = v = make_uint2(0u, 0u);  // behind the end: may hold anything
    uint4 s;
    auto put = [&](float4* a, float2* b, uint2 w, int e) {
      float *pa = reinterpret_cast<float*>(a + j / 2) + j % 2, *pb = reinterpret_cast<float*>(b + j / 2) + j % 2;
      pa[0] = __uint_as_float(uint32_t(e) << 23);
      pa[2] = fmaf(8.f, lo16(w.x), hi16(w.x));
      pb[0] = fmaf(8.f, lo16(w.y), hi16(w.y));
    };
    put(par.ka, par.kb, k, scales(k, there, s.x, s.y));
    const int e = scales(v, there, s.z, s.w);
    put(par.va, par.vb, v, e);
    scale[j] = s;
    const int top = __reduce_max_sync(~0u, there ? e : 1), low = __reduce_min_sync(~0u, there ? e : 254);
    if (lane == 0) {
      par.top[i] = top;
      par.low[i] = low;
    }
  }
  if (lane == 0) par.held = held;
}
// One page's keys (or values) as an operand, by the kCodeWarps
__device__ __forceinline__ void expand_keys(const uint8_t* raw, const uint4* scale, uint8_t* op, int tid) {
#pragma unroll
  for (int i = 0; i < 256 / (kCodeWarps * 32); ++i) {
    // 16 bytes: dimensions 16 q .. 16 q + 15 of both groups of a token
    const int at = tid + i * kCodeWarps * 32, r = at / 4, q = at % 4;
    const uint4 w = *reinterpret_cast<const uint4*>(raw + at / 64 * kKv4TileBytes + at % 64 * 16);
    const uint2 s = *reinterpret_cast<const uint2*>(&scale[r].x);
    *reinterpret_cast<uint4*>(op + piece_at(r, 2 * q)) = codes(w.x, s.x);
    *reinterpret_cast<uint4*>(op + piece_at(r, 2 * q + 1)) = codes(w.y, s.x);
    *reinterpret_cast<uint4*>(op + kGroupBytes + piece_at(r, 2 * q)) = codes(w.z, s.y);
    *reinterpret_cast<uint4*>(op + kGroupBytes + piece_at(r, 2 * q + 1)) = codes(w.w, s.y);
  }
}
__device__ __forceinline__ void expand_values(const uint8_t* raw, const uint4* scale, uint8_t* op, int tid) {
#pragma unroll
  for (int i = 0; i < 256 / (kCodeWarps * 32); ++i) {
    // 16 bytes: eight dimensions of two neighbouring tokens and both groups
    const int at = tid + i * kCodeWarps * 32, r = at / 64 * 16 + at % 64 / 32 * 8 + at % 4 * 2, oct = at % 32 / 4;
    const uint4 w = *reinterpret_cast<const uint4*>(raw + at / 64 * kKv4TileBytes + kKv4V + at % 64 * 16);
    const uint2 s = *reinterpret_cast<const uint2*>(&scale[r].z), s1 = *reinterpret_cast<const uint2*>(&scale[r + 1].z);
    *reinterpret_cast<uint4*>(op + piece_at(r, oct)) = codes(__byte_perm(w.x, w.y, 0x5410), s.x);
    *reinterpret_cast<uint4*>(op + kGroupBytes + piece_at(r, oct)) = codes(__byte_perm(w.z, w.w, 0x5410), s.y);
    *reinterpret_cast<uint4*>(op + piece_at(r + 1, oct)) = codes(__byte_perm(w.x, w.y, 0x7632), s1.x);
    *reinterpret_cast<uint4*>(op + kGroupBytes + piece_at(r + 1, oct)) = codes(__byte_perm(w.z, w.w, 0x7632), s1.y);
  }
}

// The power of two that brings the number with these exponent bits to 2^kUnitTop .. twice that
__device__ __forceinline__ float unit_of(int exponent) {
  return __uint_as_float(uint32_t(min(max(2 * 127 + kUnitTop - exponent, 1), int(kUnitMax))) << 23);
}
// Bounded wait.  A warp that polls takes the softmax warps' issue slots (2000 of 9000 instructions a page without
// the sleep), so those that run ahead sleep between two looks.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, uint64_t limit_ns, uint32_t sleep_ns) {
  auto look = [&]() {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
  };
  if (limit_ns == 0) return mbar_test_wait(bar, parity);
  if (look()) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 0;; ++i) {
    if (sleep_ns > 0) __nanosleep(sleep_ns);
    if (look()) return true;
    if ((i & 63u) == 63u && globaltimer_ns() - t0 > limit_ns) return false;
  }
}
__device__ __forceinline__ int pages_of(int len) { return max(1, (len + kKv4Page - 1) / kKv4Page); }

// The plan, by one warp: the number of pieces that the longest group is cut into, for which the waves
// of items take least.
__device__ __forceinline__ void make_plan(TreePlan& plan, const TreeCall& P, int ctas, bool report, int lane) {
  const int cap = P.pg.max_pages * kKv4Page, per_seq = P.pg.hkv * P.n_blk;
  int longest = 1;
  for (int b = lane; b < P.batch; b += 32) {
    int given = P.first[b];
    if (given >= 0) given = given < INT32_MAX - P.n_q ? given + P.n_q : INT32_MAX;
    const int len = min(max(given, 0), cap);
    if (report && given != len) set_device_error(P.pg.status, DEV_BAD_LIST, b);
    plan.len[b] = len;
    longest = max(longest, pages_of(len));
  }
  longest = __reduce_max_sync(~0u, longest);
  __syncwarp();
  const int groups = P.batch * per_seq;
  int piece = longest;
  if (groups * 2 <= kTreeItems) {  // lane: lane + 1 pieces
    const int each = (longest + lane) / (lane + 1);
    int items = 0;
    for (int b = 0; b < P.batch; ++b) items += (pages_of(plan.len[b]) + each - 1) / each;
    items *= per_seq;
    uint32_t cost = ~0u;
    if (items <= kTreeItems || lane == 0) cost = min(uint32_t((items + ctas - 1) / ctas) * uint32_t(each + kItemCost), 0x03ffffffu);
    const uint32_t best = __reduce_min_sync(~0u, cost == ~0u ? ~0u : cost << 5 | uint32_t(lane));
    piece = __shfl_sync(~0u, each, best & 31u);
  }
  int run = 0;
  for (int b0 = 0; b0 < P.batch; b0 += 32) {
    const int b = b0 + lane;
    int n = b < P.batch ? (pages_of(plan.len[b]) + piece - 1) / piece * per_seq : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(~0u, n, o);
      if (lane >= o) n += up;
    }
    if (b < P.batch) plan.before[b + 1] = run + n;
    run += __shfl_sync(~0u, n, 31);
  }
  if (lane == 0) {
    plan.before[0] = 0;
    plan.piece = piece;
  }
}

// An item: pages [page0, page1) of group `group` of sequence b; all of them where `pieces` is 1.
struct Item {
  int b, group, pieces, page0, page1, len;
  __device__ __forceinline__ Item(const TreePlan& plan, const TreeCall& P, int item, int lane) {
    b = 0;
    for (;;) {  // the last sequence whose items start at or before it
      const int i = b + 1 + lane;
      const int n = __popc(__ballot_sync(~0u, i < P.batch && plan.before[i] <= item));
      b += n;
      if (n < 32) break;
    }
    const int per_seq = P.pg.hkv * P.n_blk;
    pieces = (plan.before[b + 1] - plan.before[b]) / per_seq;
    const int rel = item - plan.before[b];
    group = rel / pieces;
    const int i = rel - group * pieces;
    len = plan.len[b];
    const int n = pages_of(len), q = n / pieces, r = n - q * pieces;
    page0 = q * i + r * i / pieces;
    page1 = q * (i + 1) + r * (i + 1) / pieces;
  }
};

// The 64 tokens of the page at `pos` that a drafted token sees: those before the first drafted one, then
// those of its mask, of what the sequence has.
__device__ __forceinline__ uint64_t seen_of(uint64_t tree, int prefix, int pos, int held) {
  const int ahead = prefix - pos;
  const uint64_t b = ahead >= 64 ? ~0ull : ahead > 0 ? tree << ahead | ((1ull << ahead) - 1) : -ahead < 64 ? tree >> -ahead : 0ull;
  return held >= 64 ? b : b & ((1ull << max(held, 0)) - 1);
}

// A softmax thread's part: rows lane / 4 + 8 i (i 0 .. 3) of its warp's 32, and of half a page the tokens
// 8 b + 2 (lane % 4) and the next (b 0 .. 3).
struct Soft {
  float m[4];        // reference of the weights, log2: within 2^8 of the largest; kNone: no token yet
  Pair u2[4];        // units, twice
  float largest[4];  // the rows' largest weights p f times 2^-9, once they have units of their own
  Pair qs2[4], less[4];  // the queries' scales, twice; -m, twice
  float most;        // the largest unit of the warp's rows
  float least;       // what every row's largest weight with its unit is at least
  bool split;        // the rows have units of their own
  __device__ __forceinline__ float u(int row) const { return first(u2[row]); }
  __device__ __forceinline__ float qs(int row) const { return first(qs2[row]); }
  static __device__ __forceinline__ float first(const Pair& p) {
    float a, b;
    p.get(a, b);
    return a;
  }
  __device__ __forceinline__ Soft(const float* q_scale)
      : u2{top(), top(), top(), top()},
        qs2{twice(q_scale[0]), twice(q_scale[8]), twice(q_scale[16]), twice(q_scale[24])},
        less{twice(-kNone), twice(-kNone), twice(-kNone), twice(-kNone)} {
    most = __uint_as_float(kUnitMax << 23);
    least = INFINITY;
    split = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = kNone;
      largest[i] = 0.f;
    }
  }
  static __device__ __forceinline__ Pair twice(float x) { return Pair(x, x); }
  static __device__ __forceinline__ Pair top() { return twice(__uint_as_float(kUnitMax << 23)); }
};

// Values of this warp's rows times f[row]
__device__ __forceinline__ void rescale_values(uint32_t at, const float (&f)[4]) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t r[16];
      const uint32_t a = at + c * 32 + (uint32_t(h * 16) << 16);
      tmem_load_16x32(r, a);
      tmem_wait_loads();
      tie(r);
#pragma unroll
      for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f[2 * h + (i >> 1 & 1)]);
      tmem_store_16x32(a, r);
    }
  tmem_wait_stores();
}

// Maximum and sum over the four threads of a row
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
  return fmaxf(x, __shfl_xor_sync(~0u, x, 2));
}
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor_sync(~0u, x, 1);
  return x + __shfl_xor_sync(~0u, x, 2);
}

// Units of their own for the rows, where scales lie far apart: by the half page's largest as long as the
// row's largest weight is kLeast or more with that, and by that weight otherwise.  x: the logits; f: on the
// sums, as the reference moves; k: on the values.
template <bool EDGE>
__device__ __forceinline__ void split_units(Soft& S, const uint32_t (&x)[2][16], const float4* va, float by_scale, const float (&f)[4],
                                            float (&k)[4], const uint32_t (&seen)[4], int t) {
  float most = 0.f;
#pragma unroll
  for (int row = 0; row < 4; ++row) {
    const int h = row >> 1, e = row & 1;
    float w = 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const float4 v = va[4 * b + t];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // 2^-9: finite with any f
        const float p = ex2(fmaf(__uint_as_float(x[h][4 * b + 2 * e + j]), S.qs(row), -S.m[row])) * 0.001953125f;
        if (!EDGE || (seen[row] >> (8 * b + 2 * t + j) & 1)) w = fmaxf(w, p * (j ? v.y : v.x));
      }
    }
    const float old = S.u(row);
    const float all = fmaxf(row_max(w), f[row] * (S.split ? S.largest[row] : kLeast * 0.001953125f / old));
    float unit = fminf(old, by_scale);
    if (!(all * unit >= kLeast * 0.001953125f && all * unit < kMost * 0.001953125f)) unit = unit_of(int(__float_as_uint(all) >> 23) + 9);
    S.u2[row] = Soft::twice(unit);
    S.largest[row] = all;
    k[row] = unit >= 1.f ? f[row] * unit / old : f[row] * (unit / old);  // in range in between, too
    most = fmaxf(most, unit);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
  S.most = most;
  S.split = true;
}

// Half a page of a stream: its sums of q k' in 32 columns of tensor memory at `at` become the weights'
// upper and lower parts there, 16 columns each.  l, c: sums of the weights and of their products with z', over
// this thread's even and odd tokens.  settle(): waits until no product writes the values.
template <bool EDGE, typename F>
__device__ __forceinline__ void soft_half(Soft& S, Pair (&l)[4], Pair (&c)[4][2], const PageParams& par, int half, uint32_t at,
                                          uint32_t values, bool any, const uint32_t (&seen)[4], int t, const float4* q_sum, F settle) {
  const float4 *ka = par.ka + half * (kHalfPage / 2), *va = par.va + half * (kHalfPage / 2);
  const float2 *kb = par.kb + half * (kHalfPage / 2), *vb = par.vb + half * (kHalfPage / 2);
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  uint32_t s[2][16];  // [row half]: sums, then logits
#pragma unroll
  for (int h = 0; h < 2; ++h) tmem_load_16x32(s[h], at + (uint32_t(h * 16) << 16));
  {
    const float4 sum[4] = {q_sum[0], q_sum[8], q_sum[16], q_sum[24]};
    tmem_wait_loads();
    tie(s[0]);
    tie(s[1]);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const float4 a4 = ka[4 * b + t];
      const float2 b2 = kb[4 * b + t];
#pragma unroll
      for (int row = 0; row < 4; ++row) {
        const int h = row >> 1, i = 4 * b + 2 * (row & 1);
        Pair y = mul2(Pair(b2.x, b2.y), Pair(sum[row].z, sum[row].w));
        y = fma2(Pair(a4.z, a4.w), Pair(sum[row].x, sum[row].y), y);
        y = fma2(Pair(a4.x, a4.y), Pair(__uint_as_float(s[h][i]), __uint_as_float(s[h][i + 1])), y);
        float x[2];
        y.get(x[0], x[1]);
        if (EDGE)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (!(seen[row] >> (8 * b + 2 * t + j) & 1)) x[j] = -INFINITY;
        mx[row] = fmaxf(mx[row], fmaxf(x[0], x[1]));
        s[h][i] = __float_as_uint(x[0]);
        s[h][i + 1] = __float_as_uint(x[1]);
      }
    }
  }
  // A new reference, or new units, only where the old ones may no longer do.
  bool over = __uint_as_float(uint32_t(par.top[half]) << 23) * S.most >= kMaxScale;
#pragma unroll
  for (int row = 0; row < 4; ++row) {
    mx[row] *= S.qs(row);
    over |= mx[row] > S.m[row] + kGrowth;
  }
  if (__any_sync(~0u, over)) {
    float f[4], k[4];
#pragma unroll
    for (int row = 0; row < 4; ++row) {
      const float m1 = fmaxf(S.m[row], row_max(mx[row]));
      f[row] = ex2(S.m[row] - m1);
      S.m[row] = m1;
      S.less[row] = Soft::twice(-m1);
      const Pair f2(f[row], f[row]);
      l[row] = mul2(l[row], f2);
      c[row][0] = mul2(c[row][0], f2);
      c[row][1] = mul2(c[row][1], f2);
    }
    // One unit for all while that serves them: where a row's reference moves, a token of this half page
    // has p = 1 in it, and so at least its smallest f.
    const float low = __uint_as_float(uint32_t(par.low[half]) << 23);
    const float by_scale = unit_of(par.top[half]), unit = fminf(S.most, by_scale), ratio = unit / S.most;
    S.least = fminf(S.least * ratio, low * unit);
    if (!S.split && S.least >= kLeast) {
      S.most = unit;
#pragma unroll
      for (int row = 0; row < 4; ++row) {
        S.u2[row] = Soft::twice(unit);
        k[row] = f[row] * ratio;
      }
    } else {
      split_units<EDGE>(S, s, va, by_scale, f, k, seen, t);
    }
    if (any) {
      settle();
      rescale_values(values, k);
    }
  }
#pragma unroll
  for (int ch = 0; ch < 2; ++ch) {
    uint32_t part[2][2][4];  // [row half][part]
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int b = ch * 2 + j;
      const float4 a4 = va[4 * b + t];
      const float2 b2 = vb[4 * b + t];
#pragma unroll
      for (int row = 0; row < 4; ++row) {
        const int h = row >> 1, e = row & 1, i = 4 * b + 2 * e;
        float p[2];
        fma2(Pair(__uint_as_float(s[h][i]), __uint_as_float(s[h][i + 1])), S.qs2[row], S.less[row])
            .get(p[0], p[1]);
        float z[4] = {a4.z, a4.w, b2.x, b2.y};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          p[n] = ex2(p[n]);
          if (EDGE && !(seen[row] >> (8 * b + 2 * t + n) & 1)) p[n] = z[n] = z[2 + n] = 0.f;  // z' may be NaN there
        }
        const Pair pp(p[0], p[1]);
        l[row] = add2(l[row], pp);
        c[row][0] = fma2(pp, Pair(z[0], z[1]), c[row][0]);
        c[row][1] = fma2(pp, Pair(z[2], z[3]), c[row][1]);
        float w[2];
        // in this order: a large f with the unit of a row without weight on it may overflow
        mul2(mul2(pp, S.u2[row]), Pair(a4.x, a4.y)).get(w[0], w[1]);
        const __half2 hi = __floats2half2_rn(w[0], w[1]);
        part[h][0][2 * j + e] = bits(hi);
        part[h][1][2 * j + e] = rest(hi, w[0], w[1]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < 2; ++n) tmem_store_16x8(at + n * 16 + ch * 8 + (uint32_t(h * 16) << 16), part[h][n]);
  }
  tmem_wait_stores();
}

// What a thread has flushed, in memory: it alone writes and reads it
__device__ __forceinline__ float4 load_kept(const float4* p) {
  float4 x;
  asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(p) : "memory");
  return x;
}
__device__ __forceinline__ void store_kept(float4* p, float4 x) {
  asm volatile("st.relaxed.gpu.global.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w) : "memory");
}
// A thread's place there: values, then for each of its rows the sums of the weights and of those times z', and the
// reference that all of them are of
constexpr int kKeptSums = kTreeRows * kHeadDim / 4;
__device__ __forceinline__ float4* kept_of(const TreeCall& P, int stream) {
  return reinterpret_cast<float4*>(P.kept + (int64_t(blockIdx.x) * 2 + stream) * kTreeKeptFloats) + threadIdx.x % kTreeRows;
}
// A stream's sums since the last flush join those before it (`first`: none), rounded properly, there or, of the
// `last` pages, in tensor memory.  done(): waits for the products.
template <typename F>
__device__ __forceinline__ void flush(const TreeCall& P, const Soft& S, Pair (&l)[4], Pair (&c)[4][2], int stream, uint32_t values, bool first,
                                      bool last, F done) {
  float4* kept = kept_of(P, stream);
  float4 was[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) was[i] = first ? make_float4(0.f, 0.f, 0.f, kNone) : load_kept(kept + kKeptSums + i * kTreeRows);
  done();
  float old[4], now[4];  // factors on what was there and on what joins it
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = ex2(was[i].w - S.m[i]);
    old[i] = last ? f * S.u(i) : f;
    now[i] = last ? 1.f : 1.f / S.u(i);
    float l0, l1, z0, z1, z2, z3;
    l[i].get(l0, l1);
    c[i][0].get(z0, z1);
    c[i][1].get(z2, z3);
    const float4 x = make_float4(fmaf(was[i].x, f, l0 + l1), fmaf(was[i].y, f, z0 + z1), fmaf(was[i].z, f, z2 + z3), S.m[i]);
    if (!last) store_kept(kept + kKeptSums + i * kTreeRows, x);
    l[i] = Pair(last ? x.x : 0.f, 0.f);
    c[i][0] = Pair(last ? x.y : 0.f, 0.f);
    c[i][1] = Pair(last ? x.z : 0.f, 0.f);
  }
#pragma unroll 2
  for (int n = 0; n < 4; ++n, kept += 8 * kTreeRows, values += 32) {
    uint32_t r[2][16];
    float4 y[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) tmem_load_16x32(r[h], values + (uint32_t(h * 16) << 16));
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = first ? make_float4(0.f, 0.f, 0.f, 0.f) : load_kept(kept + j * kTreeRows);
    tmem_wait_loads();
    tie(r[0]);
    tie(r[1]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t* v = &r[j / 4][j % 4 * 4];
      auto join = [&](float x, uint32_t w, int row) { return fmaf(x, old[row], __uint_as_float(w) * now[row]); };
      const int row = j / 4 * 2;
      y[j] = make_float4(join(y[j].x, v[0], row), join(y[j].y, v[1], row), join(y[j].z, v[2], row + 1), join(y[j].w, v[3], row + 1));
      v[0] = __float_as_uint(y[j].x), v[1] = __float_as_uint(y[j].y), v[2] = __float_as_uint(y[j].z), v[3] = __float_as_uint(y[j].w);
    }
    if (last) {
#pragma unroll
      for (int h = 0; h < 2; ++h) tmem_store_16x32(values + (uint32_t(h * 16) << 16), r[h]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) store_kept(kept + j * kTreeRows, y[j]);
    }
  }
  tmem_wait_stores();
}

template <typename T>
__global__ void __launch_bounds__(kTreeThreads, 1) kv4_tree_kernel(const __grid_constant__ TreeCall P) {
  extern __shared__ uint8_t smem_raw[];
  TreeShared& sh = *reinterpret_cast<TreeShared*>(smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kCopy = kSoftWarps + kCodeWarps, kScale = kCopy + 1, kMma = kScale + 1;  // and kMma + 1
  if (tid == 0) {
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_empty[i], kCodeWarps);
      mbar_init(&sh.scaled[i], 1);
    }
    for (int i = 0; i < kKeys; ++i) {
      mbar_init(&sh.k_full[i], kCodeWarps);
      mbar_init(&sh.k_empty[i], 1);
    }
    for (int i = 0; i < kVals; ++i) {
      mbar_init(&sh.v_full[i], kCodeWarps);
      mbar_init(&sh.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < 2; ++j) {
        mbar_init(&sh.s_full[i][j], 1);
        for (int h = 0; h < 2; ++h) {
          mbar_init(&sh.p_full[i][j][h], 4);
          mbar_init(&sh.v_done[i][j][h], 1);
        }
      }
    }
    mbar_init(&sh.o_full, 2);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.drained[i], 1);
    fence_mbar_init();
  }
  if (warp == kMma) tmem_alloc<1>(&sh.tmem, 512);
  follow_previous();
  if (warp == kCopy) make_plan(sh.plan, P, gridDim.x, blockIdx.x == 0, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int items = sh.plan.before[P.batch], cap = P.pg.max_pages * kKv4Page;
  bool lost = false;       // a wait of this warp ran out: it waits and works no more
  uint32_t pages = 0;      // before this item
  uint32_t issued = 0;     // pages that the copying warp has brought: all of them, unless it is lost
  auto wait = [&](uint64_t* bar, uint32_t parity, int which, uint32_t sleep_ns = 0) {
    if (!lost && !wait_for(bar, parity, P.wait_ns, sleep_ns)) {
      set_device_error(P.pg.status, DEV_WAIT_TIMEOUT, which);
      lost = true;
    }
    return !lost;
  };
  // Between items all warps meet; the softmax warps and those of the products once the queries are there
  auto ready = [&]() {
    __syncwarp();
    tc_fence_before();
    named_bar(3, (kSoftWarps + 2) * 32);
    tc_fence_after();
  };
  auto meet = [&]() {
    __syncwarp();
    tc_fence_before();
    named_bar(2, kTreeThreads);
    tc_fence_after();
  };

  // Each role goes through the items on its own: the softmax threads have 184 registers, the others 72
  // (256 x 184 + 256 x 72 = 512 x 128, what the CTA was launched with).
  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    uint32_t of_stream = 0, n_items = 0;  // pages of the stream, items
    for (int item = blockIdx.x; item < items; item += gridDim.x, ++n_items) {
      const Item I(sh.plan, P, item, lane);
      const int blk = I.group / P.pg.hkv, head = I.group - blk * P.pg.hkv;
      const int col0 = blk * kTreeRows, cols = min(kTreeRows, P.n_q * P.hpg - col0);
      const int n = I.page1 - I.page0;
      const int prefix = min(max(P.first[I.b], 0), cap);
      // the queries, two rows at a time: a lane has dimensions 8 (lane % 16) .. + 7 of one, a piece of its operand
      constexpr int kEach = kTreeRows / kSoftWarps;
#pragma unroll 1
      for (int i0 = 0; i0 < kEach; i0 += 8) {
        uint4 in[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = warp * kEach + i0 + 2 * i + (lane >> 4), col = col0 + r, tok = col / P.hpg;
          in[i] = make_uint4(0, 0, 0, 0);
          if (r < cols) {
            const T* q = static_cast<const T*>(P.q) +
                         ((int64_t(I.b) * P.n_q + tok) * P.pg.hkv * P.hpg + head * P.hpg + col - tok * P.hpg) * kHeadDim + 8 * (lane & 15);
            asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(in[i].x), "=r"(in[i].y), "=r"(in[i].z), "=r"(in[i].w) : "l"(q));
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = warp * kEach + i0 + 2 * i + (lane >> 4);
          const T* e8 = reinterpret_cast<const T*>(&in[i]);
          float x[8], big = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] = q_value(e8[j]);
            big = fmaxf(big, fabsf(x[j]));
          }
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, o));
          // power of two that brings the largest element to 2^13 .. 2^14
          const int e = min(max(int(__float_as_uint(big) >> 23) - 127, -113), 127);
          const float up = __uint_as_float(uint32_t(127 + 13 - e) << 23);
          float sum = 0.f;
          uint32_t w[4];  // in the order of codes(): 0, 4, 1, 5, 2, 6, 3, 7
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __half2 v = __floats2half2_rn(x[j] * up, x[j + 4] * up);
            const float2 f = __half22float2(v);
            sum += f.x + f.y;
            w[j] = bits(v);
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
          const int g = lane >> 3 & 1;
          *reinterpret_cast<uint4*>(&sh.q[g][piece_at(r, lane & 7)]) = make_uint4(w[0], w[1], w[2], w[3]);
          if ((lane & 7) == 0) {
            const float v = big < INFINITY ? sum : NAN;
            reinterpret_cast<float2*>(&sh.q_sum[r])[g] = make_float2(v, v);
          }
          if ((lane & 15) == 0) sh.q_scale[r] = P.scale_log2 * __uint_as_float(uint32_t(127 - 13 + e) << 23);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      ready();
      const int stream = warp >> 2, g4 = lane >> 2, t = lane & 3, row0 = warp % 4 * 32 + g4;
      const uint32_t at = tmem + stream * kStreamColumns + (uint32_t(warp % 4 * 32) << 16);
      Soft S(&sh.q_scale[row0]);
      const Pair none(0.f, 0.f);
      Pair l2[4] = {none, none, none, none}, c2[4][2] = {{none, none}, {none, none}, {none, none}, {none, none}};
      bool any = false;
#pragma unroll 1
      for (int k0 = stream; k0 < n && !lost; k0 += 2 * kFlush) {
        const int k1 = k0 + 2 * kFlush;
#pragma unroll 1
        for (int k = k0; k < min(n, k1); k += 2, ++of_stream) {
          const uint32_t buf = (pages + k) % kVals, place = of_stream & 1;
          wait(&sh.v_full[buf], (pages + k) / kVals & 1, 4);
          wait(&sh.s_full[stream][place], of_stream >> 1 & 1, 5);
          if (__any_sync(~0u, lost)) lost = true;
          if (lost) break;
          tc_fence_after();
          const PageParams& par = sh.par[buf];
          const int pos = (I.page0 + k) * kKv4Page;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            // The products with the weights of the half page before.  They may lag behind by three halves, no more
            // (the logits of this page were multiplied after those of the page before the last), so each place and
            // half has a barrier of its own, which no two phases can pass unseen.
            auto settle = [&]() {
              const uint32_t of = half ? of_stream : of_stream - 1;
              wait(&sh.v_done[stream][of & 1][half ^ 1], of >> 1 & 1, 6);
              tc_fence_after();
              __syncwarp();
            };
            uint32_t seen[4] = {};
            const uint32_t a = at + place * kKv4Page + half * kHalfPage;
            if (pos + (half + 1) * kHalfPage > prefix || par.held < (half + 1) * kHalfPage) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = row0 + 8 * i;
                const uint64_t tree = r < cols ? uint64_t(P.tree[I.b * P.tree_stride + (col0 + r) / P.hpg]) : 0;
                seen[i] = uint32_t(seen_of(tree, prefix, pos, par.held) >> (half * kHalfPage));
              }
              soft_half<true>(S, l2, c2, par, half, a, at + kValues, any, seen, t, &sh.q_sum[row0], settle);
            } else {
              soft_half<false>(S, l2, c2, par, half, a, at + kValues, any, seen, t, &sh.q_sum[row0], settle);
            }
            any = true;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[stream][place][half]);
          }
        }
        const bool first = k0 < 2, last = k1 >= n;
        lost = __any_sync(~0u, lost);
        if (!(first && last) && !lost) {  // the products of the pages that follow are a new sum
          flush(P, S, l2, c2, stream, at + kValues, first, last, [&]() {
            wait(&sh.v_done[stream][(of_stream - 1) & 1][1], (of_stream - 1) >> 1 & 1, 6);
            tc_fence_after();
            __syncwarp();
          });
          any = last;
          lost = __any_sync(~0u, lost);
        }
      }
      wait(&sh.o_full, n_items & 1, 6);
      lost = __any_sync(~0u, lost);
      tc_fence_after();
      float l[4], m[4], c[4][2], inv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x, y;
        l2[i].get(x, y);
        l[i] = row_sum(x + y);
        m[i] = S.m[i];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          c2[i][g].get(x, y);
          c[i][g] = row_sum(x + y);
        }
        inv[i] = 1.f / S.u(i);
      }
      // a stream's values, four rows and 32 columns at a time
      auto values = [&](int c32, float (&v)[2][16]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) tmem_load_16x32(reinterpret_cast<uint32_t(&)[16]>(v[h]), at + kValues + c32 * 32 + (uint32_t(h * 16) << 16));
        tmem_wait_loads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tie(reinterpret_cast<uint32_t(&)[16]>(v[h]));
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int row = 2 * h + (i >> 1 & 1);
            v[h][i] = any ? fmaf(v[h][i], inv[row], c32 < 2 ? c[row][0] : c[row][1]) : 0.f;
          }
        }
      };
      // Each stream writes one group of dimensions; the other's values of it come through shared memory, over
      // the operands, whose products are done.
      float* shared = reinterpret_cast<float*>(&sh.val[0][0]) + tid % 128;
      auto slot = [&](int group, int c, int h, int i) { return (group * 64 + c * 32 + h * 16 + i) * 128; };
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        float v[2][16];
        values(2 * (1 - stream) + c, v);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 16; ++i) shared[slot(1 - stream, c, h, i)] = v[h][i];
      }
      if (t == 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sh.m[stream][row0 + 8 * i] = m[i];
          sh.l[stream][row0 + 8 * i] = l[i];
        }
      named_bar(1, kSoftWarps * 32);
      const bool whole = I.pieces == 1;
      float f0[4], f1[4];
      float* to[4];  // dimension t of the rows
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = row0 + 8 * i, col = col0 + r, tok = col / P.hpg;
        const int64_t o = (int64_t(I.b) * P.n_q + tok) * P.pg.hkv * P.hpg + head * P.hpg + col - tok * P.hpg;
        const float om = sh.m[1 - stream][r], all = fmaxf(m[i], om);
        f0[i] = ex2(m[i] - all);
        f1[i] = ex2(om - all);
        // in the order of the streams, so that both have the same sum
        const float own = f0[i] * l[i], else_ = f1[i] * sh.l[1 - stream][r];
        l[i] = stream == 0 ? own + else_ : else_ + own;
        to[i] = whole ? P.out + o * kHeadDim : P.partials + int64_t(item) * kTreePartialFloats + r * kHeadDim;
        if (stream == 0 && t == 0 && r < cols) {
          if (!whole) {
            float* ml = P.partials + int64_t(item) * kTreePartialFloats + kTreeRows * kHeadDim;
            ml[r] = all;
            ml[kTreeRows + r] = l[i];
          } else if (P.lse) {
            P.lse[o] = l[i] != 0.f ? (all + log2f(l[i])) * kLn2 : -INFINITY;
          }
        }
        if (whole) {  // a row without a token is 0
          const float by = l[i] != 0.f ? 1.f / l[i] : 0.f;
          f0[i] *= by;
          f1[i] *= by;
        }
        to[i] = r < cols ? to[i] + stream * 64 + t : nullptr;
      }
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        float v[2][16];
        values(2 * stream + c, v);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int row = 2 * h + (i >> 1 & 1);
            // position 2 t + i % 2 of a piece of eight: dimension t or t + 4
            if (to[row]) to[row][c * 32 + (i >> 2) * 8 + (i & 1) * 4] = f0[row] * v[h][i] + f1[row] * shared[slot(stream, c, h, i)];
          }
      }
      pages += n;
      meet();  // queries, operands and values are free again
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp < kCopy) {
      for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const Item I(sh.plan, P, item, lane);
        const int n = I.page1 - I.page0;
        for (int k = 0; k < n; ++k) {
          const uint32_t at = pages + k, raw = at % kRaw, key = at % kKeys, val = at % kVals;
          wait(&sh.scaled[raw], at / kRaw & 1, 4, 50);
          wait(&sh.k_empty[key], (at / kKeys & 1) ^ 1, 5, 50);
          if (__any_sync(~0u, lost)) {
            lost = true;
            break;
          }
          const int me = tid - kSoftWarps * 32;
          expand_keys(sh.raw[raw], sh.scale[raw], sh.key[key], me);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.k_full[key]);
          expand_values(sh.raw[raw], sh.scale[raw], sh.val[val], me);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.raw_empty[raw]);
            mbar_arrive(&sh.v_full[val]);
          }
        }
        pages += n;
        meet();  // queries, operands and values are free again
      }
    } else if (warp == kCopy) {
      for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const Item I(sh.plan, P, item, lane);
        const int n = I.page1 - I.page0;
        const int head = I.group % P.pg.hkv;
        for (int k0 = 0; k0 < n && !lost; k0 += 32) {
          int id = -1;
          if (k0 + lane < n && (I.page0 + k0 + lane) * kKv4Page < I.len) {
            id = P.pg.table[int64_t(I.b) * P.pg.max_pages + I.page0 + k0 + lane];
            if (id < 0 || id >= P.pg.n_pages) {
              set_device_error(P.pg.status, DEV_BAD_LIST, I.b);
              id = -1;
            }
          }
          for (int k = k0; k < min(n, k0 + 32); ++k) {
            const uint32_t at = pages + k, raw = at % kRaw;
            wait(&sh.raw_empty[raw], (at / kRaw & 1) ^ 1, 4, 200);
            lost = __any_sync(~0u, lost);
            if (lost) break;
            const int page = __shfl_sync(~0u, id, k - k0);
            if (lane == 0) {
              // a page that is not there has no tokens; what lies in its place is finite whatever it is
              sh.raw_held[raw] = page >= 0 ? min(kKv4Page, I.len - (I.page0 + k) * kKv4Page) : 0;
              if (page >= 0) {
                mbar_arrive_expect_tx(&sh.raw_full[raw], kKv4PageBytes);
                bulk_g2s(sh.raw[raw], P.pg.pages + (int64_t(page) * P.pg.hkv + head) * kKv4PageBytes, kKv4PageBytes, &sh.raw_full[raw]);
              } else {
                mbar_arrive(&sh.raw_full[raw]);
              }
            }
            ++issued;
            __syncwarp();
          }
        }
        pages += n;
        meet();  // queries, operands and values are free again
      }
    } else if (warp == kScale) {
      for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const Item I(sh.plan, P, item, lane);
        const int n = I.page1 - I.page0;
        for (int k = 0; k < n; ++k) {
          const uint32_t at = pages + k, raw = at % kRaw, val = at % kVals;
          wait(&sh.raw_full[raw], at / kRaw & 1, 4, 50);
          wait(&sh.v_empty[val], (at / kVals & 1) ^ 1, 5, 50);
          if (__any_sync(~0u, lost)) {
            lost = true;
            break;
          }
          expand_scales(sh.raw[raw], sh.scale[raw], sh.par[val], sh.raw_held[raw], lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.scaled[raw]);
        }
        pages += n;
        meet();  // queries, operands and values are free again
      }
    } else {
      // the whole warp, with operands that are the same in all its threads (tc_mma_warp)
      auto same = [](uint32_t x) { return __shfl_sync(~0u, x, 0); };
      auto wait_warp = [&](uint64_t* bar, uint32_t parity, int which, uint32_t sleep_ns) {
        wait(bar, parity, which, sleep_ns);
        lost = __any_sync(~0u, lost);
        return !lost;
      };
      const uint32_t by_key = tc_shape(kTreeRows, kKv4Page, false, false, false), by_value = tc_shape(kTreeRows, kHeadDim, false, false, true);
      const uint32_t tmem0 = same(tmem), q0 = same(smem_u32(sh.q[0])), k0 = same(smem_u32(sh.key[0])), v0 = same(smem_u32(sh.val[0]));
      const uint64_t q_desc = tc_operand(q0, false, 0), k_desc = tc_operand(k0, false, 0), v_desc = tc_operand(v0, true, kGroupBytes);
      const int stream = same(warp - kMma) & 1;
      const uint32_t d0 = tmem0 + stream * kStreamColumns;
      uint32_t done = 0;  // pages of the stream
      for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const Item I(sh.plan, P, item, lane);
        const int n = same(I.page1 - I.page0);
        const uint32_t base = same(pages);
        ready();
        {
          auto logits = [&](int k, uint32_t count) {  // page k, the stream's count-th
            const uint32_t key = (base + k) % kKeys, place = count & 1;
            if (!wait_warp(&sh.k_full[key], (base + k) / kKeys & 1, 4, 50)) return;
            tc_fence_after();
            const uint64_t b = k_desc + key * (kOpBytes / 16);
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tc_mma_warp(d0 + place * kKv4Page, q_desc + g * (kTreeRows * 128 / 16) + j * 2, b + g * (kGroupBytes / 16) + j * 2, by_key,
                            g + j > 0);
            tc_commit_warp(&sh.s_full[stream][place]);
            tc_commit_warp(&sh.k_empty[key]);
          };
          if (stream < n) logits(stream, done);
          if (stream + 2 < n && !lost) logits(stream + 2, done + 1);
          for (int k = stream; k < n && !lost; k += 2, ++done) {
            const uint32_t val = (base + k) % kVals, place = done & 1;
            const bool more = (k >> 1) % kFlush > 0;
            if (!wait_warp(&sh.v_full[val], (base + k) / kVals & 1, 4, 50)) break;
            const uint64_t b = v_desc + val * (kOpBytes / 16);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (lost || !wait_warp(&sh.p_full[stream][place][half], done >> 1 & 1, 7, 20)) break;
              tc_fence_after();
              const uint32_t a = d0 + place * kKv4Page + half * kHalfPage;
#pragma unroll
              for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  tc_mma_tmem_warp(d0 + kValues, a + part * 16 + j * 8, b + (2 * half + j) * 128, by_value,
                                   more || half + part + j > 0);
              tc_commit_warp(&sh.v_done[stream][place][half]);
            }
            tc_commit_warp(&sh.v_empty[val]);
            if (k + 4 < n && !lost) logits(k + 4, done + 2);
          }
          tc_commit_warp(&sh.o_full);
        }
        pages += n;
        meet();  // queries, operands and values are free again
      }
    }
  }

  // no copy or product may be in flight when the CTA ends
  if (warp == kCopy && lane == 0) {
    for (uint32_t i = issued < kRaw ? 0 : issued - kRaw; i < issued; ++i)
      if (!mbar_wait_parked(&sh.raw_full[i % kRaw], i / kRaw & 1, kTreeWaitNs)) break;
  }
  if (warp == kMma || warp == kMma + 1) {
    tc_commit_warp(&sh.drained[warp - kMma]);
    mbar_wait_parked(&sh.drained[warp - kMma], 0, kTreeWaitNs);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_free<1>(tmem, 512);
}

// Joins the pieces of the groups that were cut: eight rows a block, a warp each.
constexpr int kTreeJoinRows = 8;
struct TreeJoin {
  TreeCall call;
  int ctas;  // of the kernel before
};
__global__ void __launch_bounds__(kTreeJoinRows * 32) kv4_tree_join_kernel(const __grid_constant__ TreeJoin J) {
  __shared__ TreePlan plan;
  const TreeCall& P = J.call;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  follow_previous();
  if (warp == 0) make_plan(plan, P, J.ctas, false, lane);
  __syncthreads();
  const int per_seq = P.pg.hkv * P.n_blk, b = blockIdx.x / per_seq, group = blockIdx.x % per_seq;
  const int pieces = (plan.before[b + 1] - plan.before[b]) / per_seq;
  if (pieces == 1) return;
  const int blk = group / P.pg.hkv, head = group - blk * P.pg.hkv, r = blockIdx.y * kTreeJoinRows + warp, col = blk * kTreeRows + r;
  if (col >= P.n_q * P.hpg) return;
  const float* part = P.partials + int64_t(plan.before[b] + group * pieces) * kTreePartialFloats;
  float mx = kNone;
  for (int i = lane; i < pieces; i += 32) mx = fmaxf(mx, part[i * kTreePartialFloats + kTreeRows * kHeadDim + r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
  float sum = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < pieces; ++i) {
    const float* p = part + i * kTreePartialFloats;
    const float f = ex2(p[kTreeRows * kHeadDim + r] - mx);
    const float4 x = *reinterpret_cast<const float4*>(p + r * kHeadDim + lane * 4);
    sum = fmaf(f, p[kTreeRows * kHeadDim + kTreeRows + r], sum);
    v.x = fmaf(f, x.x, v.x);
    v.y = fmaf(f, x.y, v.y);
    v.z = fmaf(f, x.z, v.z);
    v.w = fmaf(f, x.w, v.w);
  }
  const int tok = col / P.hpg;
  const int64_t o = (int64_t(b) * P.n_q + tok) * P.pg.hkv * P.hpg + head * P.hpg + col - tok * P.hpg;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  *reinterpret_cast<float4*>(P.out + o * kHeadDim + lane * 4) =
      sum != 0.f ? make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
  if (lane == 0 && P.lse) P.lse[o] = sum != 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

}  // namespace

namespace sekv {

sekv_status tree_attention(const TreeCall& call, int sms, cudaStream_t stream) {
  void (*const fn)(TreeCall) = call.bf16 ? kv4_tree_kernel<__nv_bfloat16> : kv4_tree_kernel<__half>;
  const size_t shared = sizeof(TreeShared) + 1024;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(shared)) != cudaSuccess) {
    cudaGetLastError();
    return SEKV_ERR_CUDA;
  }
  const sekv_status st = launch_following(fn, dim3(unsigned(sms)), kTreeThreads, shared, stream, call);
  const int64_t groups = int64_t(call.batch) * call.pg.hkv * call.n_blk;
  if (st != SEKV_OK || groups * 2 > kTreeItems) return st;  // no group is cut
  const TreeJoin J{call, sms};
  return launch_following(kv4_tree_join_kernel, dim3(unsigned(groups), kTreeRows / kTreeJoinRows), kTreeJoinRows * 32, 0, stream, J);
}

}  // namespace sekv
