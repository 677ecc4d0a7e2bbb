// sekv_token_logprobs and sekv_surprisal: log-probabilities of given tokens,
// entropies and the likeliest alternatives, in one pass over the logits.
//
// Bound by memory: rows * vocab elements are read once (surprisal of 4096 rows of 128000
// in bf16: 163 us, 95% of the copy rate; few rows: launch and joins, 5.7 us for one row of
// 32000 with five alternatives).  A row is cut into
// 16-byte vectors; a cluster of 1 to 8 CTAs takes one row (as many as it takes
// to fill the GPU when there are few rows), and each thread keeps a running
// maximum m, S = sum e^(x-m) and A = sum e^(x-m) (x-m) of its own vectors, joined
// over the CTA by shuffles and over the cluster through distributed shared
// memory.  entropy = ln S - A/S has no cancellation (both terms are >= 0).
//
// The alternatives need no second pass over the row.  The n-th largest of the
// maxima of every four threads is a bound that at least n elements reach; only the
// vectors of threads whose own maximum reaches it are read again (out of L2), a warp
// per thread, and what reaches the bound -- little more than n elements as a rule --
// is sorted by (value, lowest index first).  Where that is too many -- ties, or rows
// so short that the n-th of the maxima is one of the lowest of them -- the bound is found
// again among exact keys of value and index, which no two elements share.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "decode_host.h"
#include "host_common.h"

namespace cg = cooperative_groups;
using namespace sekv;

namespace {

constexpr int kLpUnroll = 4;      // vectors of a thread in flight
constexpr int kLpMaxCluster = 8;
// exponents below this count as this, without weight; times 2^30 elements it is an fp32 number
constexpr float kFar = -1e28f;

struct LpParams {
  const void* logits;
  const void* tokens;
  float *logprob, *lse, *entropy, *top_lp;
  int32_t* top_ids;
  int32_t* status;
  int64_t stride_b, stride_t, token_stride_b;
  int64_t out_stride_b;    // rows of a sequence in the outputs
  int64_t n_tokens;        // rows of a sequence that are computed
  int64_t vocab;
  float scale;
  int tokens64, n_top, negate;  // negate: surprisal (and its H[b][0] = 0)
};

struct Stat {
  float m, s, a;  // maximum; sums in units of e^(scale (x - m)); a in log2 units
};

// 2^x, to 2^-22 of its value; 0 for -infinity
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// c (x - m), finite differences first: with x and m at the type's lowest value the product would
// overflow, the difference is 0; of halves, because with x and m at its two ends the difference would
__device__ __forceinline__ float scaled(float x, float m, float c) {
  return (x * 0.5f - m * 0.5f) * c * 2.f;
}
// exponent scale (x - m) in log2 units
__device__ __forceinline__ float exp_arg(float x, float m, float c) {
  return scaled(x, m == -INFINITY ? 0.f : m, c);
}

// (s, a) of the smaller maximum p.m in units of the larger one, m
__device__ __forceinline__ void rescale(Stat& p, float m, float c) {
  // a term without weight has no share (0 * finite), whatever its distance
  const float d = fmaxf(exp_arg(p.m, m, c), kFar), f = ex2(d);
  p.a = f * (p.a + p.s * d);
  p.s *= f;
  p.m = m;
}

__device__ __forceinline__ Stat join(Stat p, Stat q, float c) {
  const float m = fmaxf(p.m, q.m);
  rescale(p, m, c);
  rescale(q, m, c);
  return {m, p.s + q.s, p.a + q.a};
}

__device__ __forceinline__ Stat shfl_xor(const Stat& v, int o) {
  Stat r;
  r.m = __shfl_xor_sync(~0u, v.m, o);
  r.s = __shfl_xor_sync(~0u, v.s, o);
  r.a = __shfl_xor_sync(~0u, v.a, o);
  return r;
}

// Order-preserving key of (value, index): larger value first, then the lower
// index; -0 counts as 0.  Every key is above 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
  return (uint64_t(order_of(x)) << 32) | uint32_t(~index);
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = uint32_t(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return ~uint32_t(k); }

template <typename K>
__device__ __forceinline__ K cmp_swap(K k, int mask, bool keep_max) {
  const K o = __shfl_xor_sync(~0u, k, mask);
  return keep_max ? (k > o ? k : o) : (k < o ? k : o);
}

// Lane i of the warp gets the i-th largest of its 32 keys; N sets side by side.
template <int N, typename K>
__device__ __forceinline__ void warp_sort(K (&k)[N], int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int m = size >> 1; m > 0; m >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i)
        k[i] = cmp_swap(k[i], m, ((lane & size) == 0) == ((lane & m) == 0));
}

// The 32 largest of two descending lists of 32 (q: lane i holds the other
// list's entry 31 - i): the larger of each pair is a bitonic sequence.
template <typename K>
__device__ __forceinline__ K warp_merge(K p, K q, int lane) {
  K k = p > q ? p : q;
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) k = cmp_swap(k, m, (lane & m) == 0);
  return k;
}

// The 32 largest of N descending lists, descending.
template <int N, typename K>
__device__ __forceinline__ K warp_merge_all(K (&k)[N], int lane) {
#pragma unroll
  for (int n = 1; n < N; n *= 2)
#pragma unroll
    for (int i = 0; i + n < N; i += 2 * n)
      k[i] = warp_merge(k[i], __shfl_sync(~0u, k[i + n], 31 - lane), lane);
  return k[0];
}

template <int NT>
struct LpShared {
  Stat stat[NT / 32];
  Stat cta[kLpMaxCluster];             // rank 0: the cluster's parts
  uint64_t tops[kLpMaxCluster][32];    // rank 0: the cluster's lists
  uint64_t lists[NT / 32][32];
  uint64_t cand[NT];
  uint64_t sorted[32];
  uint32_t maxima[NT / 4];
  uint32_t bound;
  int n_cand;
};

// The 32 largest of one key per thread, descending, in sh.sorted.
template <int NT>
__device__ __forceinline__ void block_top32(LpShared<NT>& sh, uint64_t key) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t k[1] = {key};
  warp_sort(k, lane);
  sh.lists[warp][lane] = k[0];
  __syncthreads();
#pragma unroll
  for (int w = NT / 64; w > 0; w >>= 1) {
    if (warp < w) {
      k[0] = warp_merge(k[0], sh.lists[warp + w][31 - lane], lane);
      sh.lists[warp][lane] = k[0];
    }
    __syncthreads();
  }
  if (warp == 0) sh.sorted[lane] = k[0];
  __syncthreads();
}

__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(float v) { return v; }

__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b, __nv_bfloat16) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b, __half) {
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b, float) {
  return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
}

// A row as 16-byte vectors: vector i holds elements i*VE - off .. + VE - 1; the
// first and the last may be partial (elements outside the row read as -inf).
template <typename T>
struct Row {
  static constexpr int VE = 16 / int(sizeof(T));
  const T* base;   // 16-byte aligned; element 0 of the row is base[off]
  int off;
  int vocab;
  int full0, full1;  // vectors that lie in the row entirely
  __device__ __forceinline__ uint4 load(int i) const {
    if (i >= full0 && i < full1) return __ldcs(reinterpret_cast<const uint4*>(base) + i);
    uint4 w;
    T* e = reinterpret_cast<T*>(&w);
    const int e0 = i * VE - off;
#pragma unroll
    for (int j = 0; j < VE; ++j)
      e[j] = e0 + j >= 0 && e0 + j < vocab ? base[int64_t(i) * VE + j] : T(-INFINITY);
    return w;
  }
  __device__ static __forceinline__ void unpack(const uint4& w, float (&x)[VE]) {
    const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int j = 0; j < VE; ++j) x[j] = to_f(e[j]);
  }
  // largest element (NaN does not count)
  __device__ static __forceinline__ float largest(uint32_t m) {
    if (sizeof(T) == 4) return __uint_as_float(m);
    const T* e = reinterpret_cast<const T*>(&m);
    return fmaxf(to_f(e[0]), to_f(e[sizeof(T) == 4 ? 0 : 1]));
  }
  // at least about -5e4 (NaN stays): what is smaller has no weight beside a maximum above
  // -4e4, and its product with that weight, 0, stays finite
  __device__ static __forceinline__ uint32_t raised(uint32_t w) {
    uint32_t r;
    if constexpr (sizeof(T) == 4) {
      float f;
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(__uint_as_float(w)), "f"(-5e4f));
      r = __float_as_uint(f);
    } else if constexpr (std::is_same<T, __half>::value) {
      asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0xfa1afa1au));
    } else {
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0xc744c744u));
    }
    return r;
  }
  __device__ static __forceinline__ uint4 raised(const uint4& w) {
    return make_uint4(raised(w.x), raised(w.y), raised(w.z), raised(w.w));
  }
};

// Adds a thread's N vectors to its state.
template <typename T, bool FULL, int N>
__device__ __forceinline__ void add_vectors(Stat& st, const uint4 (&w)[N], float c) {
  constexpr int VE = Row<T>::VE;
  uint32_t top = max_pair(max_pair(w[0].x, w[0].y, T()), max_pair(w[0].z, w[0].w, T()), T());
#pragma unroll
  for (int u = 1; u < N; ++u)
    top = max_pair(top, max_pair(max_pair(w[u].x, w[u].y, T()), max_pair(w[u].z, w[u].w, T()), T()), T());
  const float gm = Row<T>::largest(top);
  if (gm > st.m) rescale(st, gm, c);
  if (fabsf(st.m) < 4e4f && c < 1e3f && c > 0.05f) {
    // Exponents by one fma, x c - fl(m c); what rounding m c took, r, is the same for all
    // of them: 2^-r is multiplied out of the sums, so that a common offset of the
    // logits costs nothing.
    const float mc = st.m * c, r = fmaf(st.m, c, -mc);
    float s[2] = {0.f, 0.f}, a[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < N; ++u) {
      float x[VE];
      Row<T>::unpack(FULL ? Row<T>::raised(w[u]) : w[u], x);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float d = fmaf(x[j], c, -mc), e = ex2(d);
        s[j & 1] += e;
        if (FULL) a[j & 1] = fmaf(e, d, a[j & 1]);
      }
    }
    const float sum = s[0] + s[1], k = ex2(-r);
    st.s = fmaf(sum, k, st.s);
    if (FULL) st.a = fmaf(fmaf(-r, sum, a[0] + a[1]), k, st.a);
  } else {
    const float m0 = st.m == -INFINITY ? 0.f : st.m;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      float x[VE];
      Row<T>::unpack(w[u], x);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float d = scaled(x[j], m0, c), e = ex2(d);
        st.s += e;
        if (FULL) st.a = fmaf(e, fmaxf(d, kFar), st.a);
      }
    }
  }
}

// The vectors of the lanes of this warp that `mine` names, read again, a vector per
// lane: elements whose key reaches `bound` go to sh.cand.
template <typename T, int NT>
__device__ __forceinline__ void collect(LpShared<NT>& sh, const Row<T>& row, int lo, int hi,
                                        bool mine, uint64_t bound) {
  constexpr int VE = Row<T>::VE;
  const int lane = threadIdx.x & 31;
  for (uint32_t left = __ballot_sync(~0u, mine); left != 0; left &= left - 1) {
    const int owner = (threadIdx.x & ~31) + __ffs(left) - 1;
    // too many already: the rest would be in vain (the lanes leave together)
    if (__any_sync(~0u, *const_cast<volatile int*>(&sh.n_cand) > NT)) return;
    for (int i = lo + owner + lane * NT; i < hi; i += 32 * NT) {
      float x[VE];
      row.unpack(row.load(i), x);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const uint64_t k = key_of(x[j], uint32_t(i * VE + j - row.off));
        if (x[j] > -INFINITY && k >= bound) {
          const int at = atomicAdd(&sh.n_cand, 1);
          if (at < NT) sh.cand[at] = k;
        }
      }
    }
    __syncwarp();
  }
}

// The alternatives of a slice when many elements reach the bound (ties; or short rows with
// many alternatives, such as 500 in bf16 with 20): the bound among exact keys, and if even
// those are too many -- the largest logits lie in a few threads' vectors, or there are fewer
// threads with a vector than alternatives -- one alternative per round.
template <typename T, int NT>
__device__ __noinline__ void top_of_ties(LpShared<NT>& sh, const Row<T>& row, int lo, int hi,
                                         float thread_max, int n_top) {
  constexpr int VE = Row<T>::VE;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // The caller's threads chose this path by n_cand: all have read it before it is set to 0, or
  // one that comes late would choose another path and wait at another barrier.
  __syncthreads();
  uint64_t key = 0;  // the first place of this thread's maximum
  if (thread_max > -INFINITY)
    for (int i = lo + tid; i < hi && key == 0; i += NT) {
      float x[VE];
      row.unpack(row.load(i), x);
#pragma unroll
      for (int j = VE - 1; j >= 0; --j)
        if (x[j] == thread_max) key = key_of(x[j], uint32_t(i * VE + j - row.off));
    }
  if (tid == 0) sh.n_cand = 0;
  block_top32(sh, key);
  const uint64_t bound = max(sh.sorted[n_top - 1], uint64_t(1));
  collect(sh, row, lo, hi, key >= bound, bound);
  __syncthreads();
  const int n = sh.n_cand;
  if (n <= NT) {
    block_top32(sh, tid < n ? sh.cand[tid] : 0);
    return;
  }
  uint64_t last = ~uint64_t(0);
  for (int k = 0; k < n_top; ++k) {
    uint64_t best = 0;
    for (int i = lo + tid; i < hi; i += NT) {
      float x[VE];
      row.unpack(row.load(i), x);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const uint64_t kk = key_of(x[j], uint32_t(i * VE + j - row.off));
        if (x[j] > -INFINITY && kk < last && kk > best) best = kk;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(~0u, best, o);
      best = best > other ? best : other;
    }
    if (lane == 0) sh.lists[warp][0] = best;
    __syncthreads();
    for (int w = 0; w < NT / 32; ++w) best = max(best, sh.lists[w][0]);
    last = best;
    if (tid == 0) sh.sorted[k] = best;
    __syncthreads();
    if (best == 0) {
      if (tid > k && tid < 32) sh.sorted[tid] = 0;
      break;
    }
  }
  __syncthreads();
}

// FULL: entropy, log-sum-exp or alternatives are asked for
template <typename T, bool FULL, int NT>
__global__ void __launch_bounds__(NT, NT == 512 ? 3 : 1) logprob_kernel(const LpParams P) {
  constexpr int VE = Row<T>::VE;
  __shared__ LpShared<NT> sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = cluster.num_blocks(), rank = cluster.block_rank();
  cluster.barrier_arrive();  // waited for before the first remote store: every CTA has started
  follow_previous();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x / nc;
  const int64_t b = r / P.n_tokens, t = r - b * P.n_tokens;
  const T* first = static_cast<const T*>(P.logits) + b * P.stride_b + t * P.stride_t;
  Row<T> row;
  row.off = int((reinterpret_cast<uintptr_t>(first) & 15) / sizeof(T));
  row.base = first - row.off;
  row.vocab = int(P.vocab);
  row.full0 = row.off > 0 ? 1 : 0;
  row.full1 = (row.off + row.vocab) / VE;
  const int nv = (row.off + row.vocab + VE - 1) / VE;
  const int lo = int(int64_t(nv) * rank / nc), hi = int(int64_t(nv) * (rank + 1) / nc);
  const float c = P.scale * kLog2e;

  int64_t tok = -1;
  float tok_x = 0.f;
  if (rank == 0 && tid == 0) {
    const int64_t ti = b * P.token_stride_b + t;
    tok = P.tokens64 ? static_cast<const int64_t*>(P.tokens)[ti]
                     : int64_t(static_cast<const int32_t*>(P.tokens)[ti]);
    if (tok >= 0 && tok < P.vocab) tok_x = to_f(first[tok]);
  }

  // one pass: m, s, a of this thread's vectors lo + tid + NT * i
  Stat st{-INFINITY, 0.f, 0.f};
  constexpr int kStep = NT * kLpUnroll;
  const int n_groups = (hi - lo + kStep - 1) / kStep;
  for (int g = 0; g < n_groups; ++g) {
    const int g0 = lo + g * kStep;
    uint4 w[kLpUnroll];
    if (g0 >= row.full0 && g0 + kStep <= min(hi, row.full1)) {
      const uint4* src = reinterpret_cast<const uint4*>(row.base) + g0 + tid;
#pragma unroll
      for (int u = 0; u < kLpUnroll; ++u) w[u] = __ldcs(src + u * NT);
      add_vectors<T, FULL>(st, w, c);
    } else {
      const T none = T(-INFINITY);
      uint4 blank;
#pragma unroll
      for (int j = 0; j < VE; ++j) reinterpret_cast<T*>(&blank)[j] = none;
#pragma unroll
      for (int u = 0; u < kLpUnroll; ++u) {
        const int i = g0 + tid + u * NT;
        w[u] = i < hi ? row.load(i) : blank;
      }
      add_vectors<T, FULL>(st, w, c);
    }
  }
  const float thread_max = st.m;

#pragma unroll
  for (int o = 16; o > 0; o >>= 1) st = join(st, shfl_xor(st, o), c);
  if (lane == 0) sh.stat[warp] = st;
  const bool tops = FULL && P.n_top > 0;
  const uint32_t order = thread_max > -INFINITY ? order_of(thread_max) : 0u;
  if (tops) {
    if (tid == 0) sh.n_cand = 0;
    uint32_t m = max(order, __shfl_xor_sync(~0u, order, 1));
    m = max(m, __shfl_xor_sync(~0u, m, 2));
    if ((lane & 3) == 0) sh.maxima[tid / 4] = m;
  }
  __syncthreads();
  cluster.barrier_wait();
  if (warp == 1) {  // beside warp 0, which looks for the bound
    st = lane < NT / 32 ? sh.stat[lane] : Stat{-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int o = NT / 64; o > 0; o >>= 1) st = join(st, shfl_xor(st, o), c);
    if (lane == 0) cluster.map_shared_rank(&sh, 0)->cta[rank] = st;
  }
  if (tops) {
    if (warp == 0) {
      uint32_t k[NT / 128];
#pragma unroll
      for (int i = 0; i < NT / 128; ++i) k[i] = sh.maxima[32 * i + lane];
      warp_sort(k, lane);
      const uint32_t m = warp_merge_all(k, lane);
      if (lane == P.n_top - 1) sh.bound = max(m, 1u);
    }
    __syncthreads();
    const bool mine = order >= sh.bound;
    // as a rule n_top threads or little more
    if (__syncthreads_count(mine) <= 2 * P.n_top + 32) {
      collect(sh, row, lo, hi, mine, uint64_t(sh.bound) << 32);
      __syncthreads();
      const int n = sh.n_cand;
      if (n <= 32) {
        if (warp == 0) {
          uint64_t k[1] = {lane < n ? sh.cand[lane] : 0};
          warp_sort(k, lane);
          sh.sorted[lane] = k[0];
        }
      } else if (n <= NT) {
        block_top32(sh, tid < n ? sh.cand[tid] : 0);
      } else {
        top_of_ties(sh, row, lo, hi, thread_max, P.n_top);
      }
    } else {
      top_of_ties(sh, row, lo, hi, thread_max, P.n_top);
    }
    if (warp == 0)
      cluster.map_shared_rank(&sh, 0)->tops[rank][lane] = lane < P.n_top ? sh.sorted[lane] : 0;
  }
  cluster.sync();  // the parts of every CTA are in rank 0's shared memory
  if (rank != 0 || warp != 0) return;

  Stat all = sh.cta[0];
  for (int k = 1; k < nc; ++k) all = join(all, sh.cta[k], c);
  const bool bad = isnan(all.s) || all.m == INFINITY;
  const float ln_s = logf(all.s);
  const float top = all.m == -INFINITY ? all.m : P.scale * all.m;
  const int64_t o = b * P.out_stride_b + t;
  if (tid == 0) {
    float lp;
    if (tok == -1) {
      lp = bad ? NAN : 0.f;
    } else if (tok < 0 || tok >= P.vocab) {
      lp = NAN;
      set_device_error(P.status, DEV_BAD_LIST, int32_t(r > INT32_MAX ? INT32_MAX : r));
    } else if (bad) {
      lp = NAN;
    } else if (tok_x == -INFINITY) {
      lp = -INFINITY;
    } else {
      lp = scaled(tok_x, all.m, P.scale) - ln_s;
    }
    P.logprob[o] = P.negate && !isnan(lp) ? 0.f - lp : lp;
    if (P.negate && t == 0) P.logprob[o - 1] = 0.f;
    if (FULL && P.lse) P.lse[o] = bad ? NAN : all.s > 0.f ? top + ln_s : -INFINITY;
    if (FULL && P.entropy)
      P.entropy[o] = bad ? NAN : all.s > 0.f ? ln_s - all.a / all.s * kLn2 : 0.f;
  }
  if (tops) {
    uint64_t k = sh.tops[0][lane];
    if (nc > 1) {
      uint64_t list[kLpMaxCluster];
#pragma unroll
      for (int i = 0; i < kLpMaxCluster; ++i) list[i] = i < nc ? sh.tops[i][lane] : 0;
      k = warp_merge_all(list, lane);
    }
    if (lane < P.n_top) {
      const bool none = k == 0 || bad;
      P.top_ids[o * P.n_top + lane] = none ? -1 : int32_t(key_index(k));
      P.top_lp[o * P.n_top + lane] =
          bad ? NAN : k == 0 ? -INFINITY : scaled(key_value(k), all.m, P.scale) - ln_s;
    }
  }
}

template <typename T, bool FULL, int NT>
sekv_status launch_logprobs(const LpParams& P, int64_t rows, int nc, cudaStream_t stream) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(unsigned(rows * nc));
  lc.blockDim = dim3(NT);
  lc.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = nc;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  // Blocks on their way while the kernel before still runs: 5.6 us for 6.2 with one row of
  // 32000.  Where there is more than one for each SM they would gather on the SMs that are
  // free first (257 rows of 50021: 18.6 us for 16.1).
  lc.numAttrs = rows * nc <= device_sm_count() ? 2 : 1;
  if (cudaLaunchKernelEx(&lc, logprob_kernel<T, FULL, NT>, P) != cudaSuccess) {
    cudaGetLastError();
    return SEKV_ERR_CUDA;
  }
  count_launch(1);
  return SEKV_OK;
}

template <typename T>
sekv_status logprobs_of(const LpParams& P, int64_t rows, bool full, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return SEKV_ERR_CUDA;
  // CTAs per row: doubled while the rows alone leave SMs without a CTA and a CTA's share is
  // more than one vector per thread.  More only multiplies the joins: 257 rows of 50021
  // in f32 with three alternatives take 16 us with one CTA, 23 with two, 29 with four.
  const int64_t vecs = P.vocab / Row<T>::VE + 1;
  int nc = 1;
  while (nc < kLpMaxCluster && rows * nc < sms && vecs > int64_t(nc) * 512) nc *= 2;
  if (rows * nc > INT32_MAX) return SEKV_ERR_UNSUPPORTED;
  // threads by the CTA's share: 2000 rows of 500 take 10 us with 128 threads, 15 with 256 and
  // 26 with 512, 1000 rows of 128000 53 us with 256 and 49 with 512
  if (vecs / nc <= 256)
    return full ? launch_logprobs<T, true, 128>(P, rows, nc, stream)
                : launch_logprobs<T, false, 128>(P, rows, nc, stream);
  if (vecs / nc <= 1024)
    return full ? launch_logprobs<T, true, 256>(P, rows, nc, stream)
                : launch_logprobs<T, false, 256>(P, rows, nc, stream);
  return full ? launch_logprobs<T, true, 512>(P, rows, nc, stream)
              : launch_logprobs<T, false, 512>(P, rows, nc, stream);
}

sekv_status logprobs_impl(const LpParams& P, int32_t dtype, int64_t batch, bool full,
                          cudaStream_t stream) {
  const int64_t rows = batch * P.n_tokens;
  if (dtype == SEKV_F32) return logprobs_of<float>(P, rows, full, stream);
  if (dtype == SEKV_F16) return logprobs_of<__half>(P, rows, full, stream);
  return logprobs_of<__nv_bfloat16>(P, rows, full, stream);
}

sekv_status check_logits(const void* logits, int32_t dtype, int64_t batch, int64_t n_tokens,
                         int64_t vocab, const void* tokens, int32_t tokens_64, void* workspace,
                         size_t workspace_bytes) {
  if (dtype < SEKV_BF16 || dtype > SEKV_F32 || batch < 0 || n_tokens < 0 || vocab < 1 ||
      ((!logits || !tokens) && batch > 0 && n_tokens > 0) || !workspace)
    return SEKV_ERR_INVALID;
  const int elem = dtype == SEKV_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % elem ||
      reinterpret_cast<uintptr_t>(tokens) % (tokens_64 ? 8 : 4) ||
      reinterpret_cast<uintptr_t>(workspace) % 4)
    return SEKV_ERR_INVALID;
  if (workspace_bytes < 64) return SEKV_ERR_CAPACITY;
  if (vocab > (int64_t(1) << 30) || batch > INT32_MAX || n_tokens > INT32_MAX ||
      batch * n_tokens > INT32_MAX)
    return SEKV_ERR_UNSUPPORTED;
  return SEKV_OK;
}

}  // namespace

extern "C" sekv_status sekv_token_logprobs(const void* logits, int32_t dtype, int64_t batch,
                                           int64_t n_tokens, int64_t vocab, int64_t stride_b,
                                           int64_t stride_t, const void* tokens,
                                           int32_t tokens_64, int64_t token_stride_b, float scale,
                                           int32_t n_top, float* logprob, float* lse,
                                           float* entropy, int32_t* top_ids, float* top_logprobs,
                                           void* workspace, size_t workspace_bytes,
                                           cudaStream_t stream) {
  reset_launches();
  const sekv_status st = check_logits(logits, dtype, batch, n_tokens, vocab, tokens, tokens_64,
                                      workspace, workspace_bytes);
  if (st != SEKV_OK) return st;
  if (!(scale > 0.f) || !isfinite(scale * kLog2e) || n_top < 0) return SEKV_ERR_INVALID;
  if (batch > 0 && n_tokens > 0 &&
      (!logprob || (n_top > 0) != (top_ids != nullptr) || (n_top > 0) != (top_logprobs != nullptr)))
    return SEKV_ERR_INVALID;
  if (n_top > SEKV_MAX_TOP) return SEKV_ERR_UNSUPPORTED;
  if (batch == 0 || n_tokens == 0) return SEKV_OK;
  LpParams P{};
  P.logits = logits;
  P.tokens = tokens;
  P.logprob = logprob;
  P.lse = lse;
  P.entropy = entropy;
  P.top_ids = top_ids;
  P.top_lp = top_logprobs;
  P.status = static_cast<int32_t*>(workspace);
  P.stride_b = stride_b;
  P.stride_t = stride_t;
  P.token_stride_b = token_stride_b;
  P.out_stride_b = P.n_tokens = n_tokens;
  P.vocab = vocab;
  P.scale = scale;
  P.tokens64 = tokens_64 != 0;
  P.n_top = n_top;
  return logprobs_impl(P, dtype, batch, lse || entropy || n_top > 0, stream);
}

extern "C" sekv_status sekv_surprisal(const void* logits, int32_t dtype, int64_t batch,
                                      int64_t ctx_len, int64_t vocab, int64_t stride_b,
                                      int64_t stride_t, const void* tokens, int32_t tokens_64,
                                      int64_t token_stride_b, float* H, void* workspace,
                                      size_t workspace_bytes, cudaStream_t stream) {
  reset_launches();
  const sekv_status st = check_logits(logits, dtype, batch, ctx_len, vocab, tokens, tokens_64,
                                      workspace, workspace_bytes);
  if (st != SEKV_OK) return st;
  if (batch == 0 || ctx_len == 0) return SEKV_OK;
  if (!H) return SEKV_ERR_INVALID;
  if (ctx_len == 1)  // nothing is predicted: H is all zeros
    return cudaMemsetAsync(H, 0, size_t(batch) * 4, stream) == cudaSuccess ? SEKV_OK : SEKV_ERR_CUDA;
  LpParams P{};
  P.logits = logits;
  P.tokens = static_cast<const char*>(tokens) + (tokens_64 ? 8 : 4);  // row t: token t + 1
  P.logprob = H + 1;
  P.status = static_cast<int32_t*>(workspace);
  P.stride_b = stride_b;
  P.stride_t = stride_t;
  P.token_stride_b = token_stride_b;
  P.out_stride_b = ctx_len;
  P.n_tokens = ctx_len - 1;
  P.vocab = vocab;
  P.scale = 1.f;
  P.tokens64 = tokens_64 != 0;
  P.negate = 1;
  return logprobs_impl(P, dtype, batch, false, stream);
}
