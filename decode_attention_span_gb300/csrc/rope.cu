// sekv_rope: rotary positions of queries and keys, and the host-side table of
// their frequencies.
//
// Pair i of a token at position p turns by p f_i.  The table holds f_i / (2 pi)
// as a 64-bit fixed-point fraction of a turn, so p * table[i] modulo 2^64 (one
// integer product) is the angle's fraction of a turn, and only the entry's own
// error grows with p: the entries are computed in fp64, which puts an angle off
// by at most p 2^-49 (below fp32's step up to p of 2^25).  The upper 32 bits go to
// sincospi.  An fp32 product p * f_i would lose the angle from positions of
// about 10^5 on.
//
// Bound by memory: every value is read and written once.  One thread owns a
// few neighbouring pairs of one token, takes their sines once and applies them
// to several heads, so the sines' cost is shared and several heads' loads are
// in flight.  Measured: 32768 tokens of 32 + 8 heads in bf16 (671 MB) 112 us, 88% of the
// copy rate; one token 2.0 us.
#include <cuda_fp16.h>
#include <math.h>

#include "decode_host.h"
#include "host_common.h"

using namespace sekv;

namespace {

constexpr int kRopeThreads = 128;
// heads whose loads a thread issues together: 32768 tokens take 112 us with 2, 144 with 4
// (fewer warps fit), 108 with 1 (which was behind, 124 to 116, before the streaming stores)
constexpr int kHeadsInFlight = 2;

struct RopeHeads {
  const void* x;
  void* y;
  int64_t xs[3], ys[3];
  int n, zero_padding;
};

struct RopeParams {
  RopeHeads q, k;
  const uint64_t* freqs;
  const void* pos;
  int64_t pos_stride_b;
  float mscale;
  int pos64, backward;
  int rot;                 // rotated dimensions
  int nrot, nvec;          // work items of a token: rotated ones, all
  int tok_per_block;
  uint32_t n_tokens;       // per sequence
  uint32_t total;          // tokens
  int heads_per_thread;
};

__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f(float v) { return v; }

template <int BYTES> struct Word;
template <> struct Word<16> { typedef uint4 type; };
template <> struct Word<8> { typedef uint2 type; };
template <> struct Word<4> { typedef uint32_t type; };
template <> struct Word<2> { typedef uint16_t type; };

// N elements of T moved with one access.
template <typename T, int N>
union Pack {
  typename Word<N * int(sizeof(T))>::type w;
  T e[N];
};

// One thread: N pairs (two accesses of N elements) of a token in the half
// layout, or N/2 pairs (one access) in the interleaved one, for every head of
// its head range; items past the rotated ones copy N elements that pass
// through.
template <typename T, int N, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams P) {
  follow_previous();
  constexpr int NP = INTER ? (N > 1 ? N / 2 : 1) : N;  // pairs of a thread
  typedef Pack<T, N> V;
  const int per = min(P.nvec, kRopeThreads);  // a token's items, or a block's share of them
  const int ti = threadIdx.x / per;
  const int vec = threadIdx.x - ti * per + blockIdx.z * kRopeThreads;
  const uint32_t tok = blockIdx.x * uint32_t(P.tok_per_block) + ti;
  if (ti >= P.tok_per_block || tok >= P.total || vec >= P.nvec) return;
  const uint32_t b = tok / P.n_tokens, t = tok - b * P.n_tokens;
  const int64_t pi = int64_t(b) * P.pos_stride_b + t;
  const int64_t pos = P.pos64 ? static_cast<const int64_t*>(P.pos)[pi]
                              : int64_t(static_cast<const int32_t*>(P.pos)[pi]);
  const bool pad = pos < 0;
  if (pad && !P.q.zero_padding && !P.k.zero_padding) return;
  const bool rotated = vec < P.nrot;
  const int half = P.rot >> 1;
  float cs[NP], sn[NP];
  int d0, pair0;
  if (rotated) {
    // INTER: elements [vec*N, vec*N + N) hold pairs from vec*NP on; with N == 1
    // (no vector access) a thread takes the two elements of pair `vec`
    pair0 = vec * NP;
    d0 = INTER ? 2 * pair0 : pair0;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint64_t turn = P.freqs[pair0 + i] * uint64_t(pos);
      const int32_t frac = int32_t(uint32_t(turn >> 32));
      sincospif(float(frac) * 4.656612873077393e-10f, &sn[i], &cs[i]);  // 2^-31: half turns
      sn[i] *= P.backward ? -P.mscale : P.mscale;
      cs[i] *= P.mscale;
    }
  } else {
    d0 = P.rot + (vec - P.nrot) * N;
  }
  const int h_all = P.q.n + P.k.n;
  const int h_end = min(h_all, int(blockIdx.y + 1) * P.heads_per_thread);
  for (int h0 = blockIdx.y * P.heads_per_thread; h0 < h_end; h0 += kHeadsInFlight) {
    V a[kHeadsInFlight], c[kHeadsInFlight];
    T* dst[kHeadsInFlight];
#pragma unroll
    for (int i = 0; i < kHeadsInFlight; ++i) {
      const int h = h0 + i;
      dst[i] = nullptr;
      if (h < h_end) {
        const bool isq = h < P.q.n;
        const RopeHeads& H = isq ? P.q : P.k;
        const int hh = isq ? h : h - P.q.n;
        const T* x = static_cast<const T*>(H.x) + b * H.xs[0] + t * H.xs[1] + hh * H.xs[2] + d0;
        T* y = static_cast<T*>(H.y) + b * H.ys[0] + t * H.ys[1] + hh * H.ys[2] + d0;
        if (pad) {
          a[i].w = c[i].w = typename Word<N * int(sizeof(T))>::type();
          dst[i] = H.zero_padding ? y : nullptr;
        } else if (rotated || x != y) {
          dst[i] = y;
          a[i].w = *reinterpret_cast<const decltype(a[i].w)*>(x);
          if (rotated) {
            if (!INTER) c[i].w = *reinterpret_cast<const decltype(a[i].w)*>(x + half);
            if (INTER && N == 1) c[i].w = *reinterpret_cast<const decltype(a[i].w)*>(x + 1);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kHeadsInFlight; ++i) {
      if (!dst[i]) continue;
      if (!rotated) {
        __stcs(reinterpret_cast<decltype(a[i].w)*>(dst[i]), a[i].w);
        continue;
      }
      if (INTER && N > 1) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const float u = to_f(a[i].e[2 * j]), v = to_f(a[i].e[(2 * j + 1) % N]);
          a[i].e[2 * j] = from_f<T>(u * cs[j] - v * sn[j]);
          a[i].e[(2 * j + 1) % N] = from_f<T>(v * cs[j] + u * sn[j]);
        }
        __stcs(reinterpret_cast<decltype(a[i].w)*>(dst[i]), a[i].w);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float u = to_f(a[i].e[j]), v = to_f(c[i].e[j]);
          a[i].e[j] = from_f<T>(u * cs[j % NP] - v * sn[j % NP]);
          c[i].e[j] = from_f<T>(v * cs[j % NP] + u * sn[j % NP]);
        }
        __stcs(reinterpret_cast<decltype(a[i].w)*>(dst[i]), a[i].w);
        __stcs(reinterpret_cast<decltype(a[i].w)*>(dst[i] + (INTER ? 1 : half)), c[i].w);
      }
    }
  }
}

template <typename T, int N>
sekv_status launch_rope(const RopeParams& P, bool inter, dim3 grid, cudaStream_t stream) {
  return launch_following(inter ? rope_kernel<T, N, true> : rope_kernel<T, N, false>, grid,
                          kRopeThreads, 0, stream, P);
}

bool rope_ok(const sekv_rope_config* r, sekv_status* why) {
  *why = SEKV_ERR_INVALID;
  if (!r) return false;
  if (r->rot_dim < 2 || r->rot_dim % 2 != 0) return false;
  if (r->rot_dim > 512) { *why = SEKV_ERR_UNSUPPORTED; return false; }
  if (r->scaling < SEKV_ROPE_NONE || r->scaling > SEKV_ROPE_BANDED) return false;
  if (!(r->base > 1.0) || !isfinite(r->base)) return false;
  if (r->scaling != SEKV_ROPE_NONE && (!(r->factor > 0.0) || !isfinite(r->factor))) return false;
  if (r->scaling == SEKV_ROPE_NTK && r->rot_dim <= 2) return false;
  if (r->scaling >= SEKV_ROPE_PARTS && r->original_context < 1) return false;
  if (r->scaling == SEKV_ROPE_PARTS &&
      !(r->beta_fast > 0.0 && r->beta_slow > 0.0 && isfinite(r->beta_fast) && isfinite(r->beta_slow)))
    return false;
  if (r->scaling == SEKV_ROPE_BANDED &&
      !(r->high_freq_factor > r->low_freq_factor && isfinite(r->low_freq_factor) &&
        isfinite(r->high_freq_factor)))
    return false;
  if (!(r->attention_factor >= 0.0) || !isfinite(r->attention_factor)) return false;
  return true;
}

// Whether every row of the tensor starts on a multiple of `bytes`.
bool rows_aligned(const sekv_heads* h, int elem, int bytes, int64_t batch, int64_t n_tokens) {
  if (!h) return true;
  auto ok = [&](const void* p, const int64_t* s) {
    if (reinterpret_cast<uintptr_t>(p) % bytes != 0) return false;
    if (batch > 1 && s[0] * elem % bytes != 0) return false;
    if (n_tokens > 1 && s[1] * elem % bytes != 0) return false;
    return h->n_heads <= 1 || s[2] * elem % bytes == 0;
  };
  return ok(h->x, h->x_stride) && ok(h->y, h->y_stride);
}

RopeHeads kernel_heads(const sekv_heads* h) {
  RopeHeads r{};
  if (!h) return r;
  r.x = h->x;
  r.y = h->y;
  r.n = h->n_heads;
  r.zero_padding = h->zero_padding != 0;
  for (int i = 0; i < 3; ++i) {
    r.xs[i] = h->x_stride[i];
    r.ys[i] = h->y_stride[i];
  }
  return r;
}

}  // namespace

extern "C" sekv_status sekv_rope_freqs(const sekv_rope_config* r, uint64_t* freqs,
                                       float* mscale) {
  sekv_status why;
  if (!rope_ok(r, &why)) return why;
  if (!freqs || !mscale) return SEKV_ERR_INVALID;
  const double two_pi = 6.283185307179586476925286766559;
  const double d = r->rot_dim, orig = r->original_context;
  const double base = r->scaling == SEKV_ROPE_NTK ? r->base * pow(r->factor, d / (d - 2.0)) : r->base;
  double lo = 0.0, hi = 0.0;
  if (r->scaling == SEKV_ROPE_PARTS) {
    const double per = d / (2.0 * log(base));
    lo = fmax(0.0, floor(per * log(orig / (r->beta_fast * two_pi))));
    hi = fmin(d - 1.0, ceil(per * log(orig / (r->beta_slow * two_pi))));
  }
  for (int i = 0; i < r->rot_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / d);
    if (r->scaling == SEKV_ROPE_LINEAR) {
      f /= r->factor;
    } else if (r->scaling == SEKV_ROPE_PARTS) {
      const double ramp = fmin(1.0, fmax(0.0, (i - lo) / fmax(hi - lo, 0.001)));
      f = (1.0 - ramp) * f + ramp * f / r->factor;
    } else if (r->scaling == SEKV_ROPE_BANDED) {
      const double s = fmin(1.0, fmax(0.0, (orig * f / two_pi - r->low_freq_factor) /
                                               (r->high_freq_factor - r->low_freq_factor)));
      f = (1.0 - s) * f / r->factor + s * f;
    }
    double turn = f / two_pi;
    turn -= floor(turn);  // whole turns do not matter at whole positions
    freqs[i] = uint64_t(ldexp(turn, 63)) * 2u;
  }
  double m = 1.0;
  if (r->scaling == SEKV_ROPE_PARTS && r->factor > 1.0) m = 0.1 * log(r->factor) + 1.0;
  if (r->attention_factor > 0.0) m = r->attention_factor;
  *mscale = float(m);
  return SEKV_OK;
}

extern "C" sekv_status sekv_rope(const sekv_rope_config* r, const uint64_t* freqs, float mscale,
                                 int32_t dtype, int32_t head_dim, int64_t batch,
                                 int64_t n_tokens, const void* positions, int32_t positions_64,
                                 int64_t pos_stride_b, const sekv_heads* q, const sekv_heads* k,
                                 int32_t flags, cudaStream_t stream) {
  reset_launches();
  sekv_status why;
  if (!rope_ok(r, &why)) return why;
  if (dtype < SEKV_BF16 || dtype > SEKV_F32 || head_dim < r->rot_dim || batch < 0 || n_tokens < 0 ||
      !freqs || (!positions && batch > 0 && n_tokens > 0) || (!q && !k) || (flags & ~SEKV_ROPE_BACKWARD) || !isfinite(mscale))
    return SEKV_ERR_INVALID;
  if (head_dim > 1024 || batch > INT32_MAX || n_tokens > INT32_MAX ||
      batch * n_tokens > INT32_MAX)
    return SEKV_ERR_UNSUPPORTED;
  const int elem = dtype == SEKV_F32 ? 4 : 2;
  for (const sekv_heads* h : {q, k}) {
    if (!h) continue;
    if (h->n_heads < 0 || h->n_heads > 65535) return SEKV_ERR_INVALID;
    // what has no elements may have no address, and any strides
    if (batch == 0 || n_tokens == 0 || h->n_heads == 0) continue;
    if (!h->x || !h->y || reinterpret_cast<uintptr_t>(h->x) % elem ||
        reinterpret_cast<uintptr_t>(h->y) % elem)
      return SEKV_ERR_INVALID;
    const int64_t size[3] = {batch, n_tokens, h->n_heads};
    for (int i = 0; i < 3; ++i) {
      if (size[i] <= 1) continue;  // the stride of a single row means nothing
      // rows of the output that lie on one another, or on other rows of the input
      if (h->y_stride[i] == 0 || (h->x == h->y && h->x_stride[i] != h->y_stride[i]))
        return SEKV_ERR_INVALID;
    }
  }
  if (reinterpret_cast<uintptr_t>(freqs) % 8 ||
      reinterpret_cast<uintptr_t>(positions) % (positions_64 ? 8 : 4))
    return SEKV_ERR_INVALID;
  const int heads = (q ? q->n_heads : 0) + (k ? k->n_heads : 0);
  if (heads > 65535) return SEKV_ERR_UNSUPPORTED;
  if (batch == 0 || n_tokens == 0 || heads == 0) return SEKV_OK;
  // widest access that every row and every part of a row allows: 16 bytes,
  // 8 bytes, or one element
  int n = 1;
  for (const int bytes : {16, 8}) {
    const int e = bytes / elem;
    const int part = r->interleaved ? r->rot_dim : r->rot_dim / 2;
    if (part % e == 0 && (head_dim - r->rot_dim) % e == 0 && r->rot_dim % e == 0 &&
        rows_aligned(q, elem, bytes, batch, n_tokens) &&
        rows_aligned(k, elem, bytes, batch, n_tokens)) {
      n = e;
      break;
    }
  }
  RopeParams P{};
  P.q = kernel_heads(q);
  P.k = kernel_heads(k);
  P.freqs = freqs;
  P.pos = positions;
  P.pos_stride_b = pos_stride_b;
  P.mscale = mscale;
  P.pos64 = positions_64 != 0;
  P.backward = (flags & SEKV_ROPE_BACKWARD) != 0;
  P.rot = r->rot_dim;
  const int pairs = r->interleaved ? (n > 1 ? n / 2 : 1) : n;
  P.nrot = r->rot_dim / 2 / pairs;
  P.nvec = P.nrot + (head_dim - r->rot_dim) / n;
  P.tok_per_block = P.nvec < kRopeThreads ? kRopeThreads / P.nvec : 1;
  P.n_tokens = uint32_t(n_tokens);
  P.total = uint32_t(batch * n_tokens);
  const int sms = device_sm_count();
  if (sms <= 0) return SEKV_ERR_CUDA;
  const uint32_t blocks = (P.total + P.tok_per_block - 1) / P.tok_per_block;
  // Heads of one thread: halved until the blocks make some four waves (32768 tokens: 112 us;
  // with one wave of longer threads 116, with eight 117, the sines being taken more often);
  // a step of a few tokens spreads its heads over blocks one by one.
  int hpt = heads;
  while (hpt > kHeadsInFlight && uint64_t(blocks) * ((heads + hpt - 1) / hpt) < uint64_t(sms) * 32)
    hpt = (hpt + 1) / 2;
  if (uint64_t(blocks) < uint64_t(sms)) hpt = 1;
  P.heads_per_thread = hpt;
  // a wide head moved by single elements has more items than a block has threads
  const dim3 grid(blocks, (heads + hpt - 1) / hpt, (P.nvec + kRopeThreads - 1) / kRopeThreads);
  const bool inter = r->interleaved != 0;
  if (dtype == SEKV_F32) {
    if (n == 4) return launch_rope<float, 4>(P, inter, grid, stream);
    if (n == 2) return launch_rope<float, 2>(P, inter, grid, stream);
    return launch_rope<float, 1>(P, inter, grid, stream);
  }
  if (dtype == SEKV_BF16) {
    if (n == 8) return launch_rope<__nv_bfloat16, 8>(P, inter, grid, stream);
    if (n == 4) return launch_rope<__nv_bfloat16, 4>(P, inter, grid, stream);
    return launch_rope<__nv_bfloat16, 1>(P, inter, grid, stream);
  }
  if (n == 8) return launch_rope<__half, 8>(P, inter, grid, stream);
  if (n == 4) return launch_rope<__half, 4>(P, inter, grid, stream);
  return launch_rope<__half, 1>(P, inter, grid, stream);
}
