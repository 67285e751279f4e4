// Rotary positions: every pair (a, b) of a head's first rotary_dim elements is turned by
// the angle p w_i (p the token's position, w_i the pair's frequency) and multiplied by m:
//
//   (a, b) -> m (a cos - b sin, b cos + a sin);
//
// the adjoint (the backward pass: the transpose of that matrix) turns by -p w_i with the
// same m.  Elements from rotary_dim on pass through.  Pairs are (i, i + rotary_dim / 2), or
// (2i, 2i + 1) in the interleaved layout.
//
// HBM-bound: every element is read and written once, 2 * N * (Hq + Hk) * d elements.  A CTA takes a
// few tokens: it forms their cosines and sines once in shared memory, then streams the tokens'
// heads (queries, then keys: one launch for both), a thread two 16-byte vectors of a head -- P pairs
// -- with neighbouring threads on neighbouring vectors and heads.  The angle is formed in float64 in
// units of turns and reduced to [-1/2, 1/2] before the float32 sine and cosine.  The reduced turn rounded to float32 is off
// by up to 2^-26 of a turn, 1e-7 rad at every position; the float64 steps before it add four roundings of the
// whole angle, position w_i 2^-51 (5e-10 rad at 2^20, 5e-4 at 2^40).  A float32 product would be off by 0.06 rad at 2^20.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "common.cuh"
#include "splitkv.h"
#include "splitkv_internal.h"
#include "strided.h"

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;     // heads whose loads are in flight together (32 warps an SM; four heads take 116 registers
                               // at 16 bits and ran at 3.8 TB/s, two at 5.6)
constexpr int kMaxPairs = 512; // pairs of one CTA's tokens in shared memory

struct Side {
  const char* in;
  char* out;
  int64_t in_tok, in_head, out_tok, out_head;   // strides in bytes
  int heads;
};

struct RopeParams {
  Side q, k;
  const void* positions;
  const double* freqs;
  int64_t n_tokens;
  int half;          // rotary_dim / 2
  int units;         // thread columns a token: units that turn, then units that copy
  int turn_units;
  int copy_vecs;     // 16-byte vectors (or elements) of a head that pass through
  int cols;          // units of one CTA (blockIdx.y takes cols * blockIdx.y onwards)
  int rows;          // threads side by side over (token, head)
  int tokens;        // of one CTA
  int heads;         // of one CTA (blockIdx.z)
  float m;
  int pos64, adjoint;
};

template <typename T>
__device__ __forceinline__ float to_f(T x) {
  return static_cast<float>(x);
}
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float x) {
  return __float2half_rn(x);
}

// P values of type T, moved as one aligned access (16 bytes, or one element when P = 1).
template <typename T, int P>
struct alignas(sizeof(T) * P < 16 ? sizeof(T) * P : 16) Vec {
  T v[P];
};

// The arrays pass through once: 16-byte accesses marked for early eviction (64k tokens of 32 + 8 heads, kernel alone: 239 us
// without the marks, 207 with them; calls in a loop 211 to 221 us on several GPUs, 93 to 97 % of the copy rate).
template <typename V>
__device__ __forceinline__ V load_once(const char* q) {
  if constexpr (sizeof(V) == 16) {
    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(q));
    return *reinterpret_cast<const V*>(&x);
  } else {
    return *reinterpret_cast<const V*>(q);
  }
}
template <typename V>
__device__ __forceinline__ void store_once(char* q, const V& v) {
  if constexpr (sizeof(V) == 16)
    __stcs(reinterpret_cast<uint4*>(q), *reinterpret_cast<const uint4*>(&v));
  else
    *reinterpret_cast<V*>(q) = v;
}

// P pairs per thread: 16 / sizeof(T) where rows allow 16-byte accesses, else 1.
template <typename T, int P, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const RopeParams p) {
  using V = Vec<T, P>;
  __shared__ __align__(16) float s_c[kMaxPairs], s_s[kMaxPairs];
  const int64_t tok0 = int64_t(blockIdx.x) * p.tokens;
  const int tokens = int(min(int64_t(p.tokens), p.n_tokens - tok0));
  const int unit0 = blockIdx.y * p.cols;
  const int turn = min(p.cols, p.turn_units - unit0);          // of this CTA's units (none: <= 0)
  const int pairs = max(0, turn) * P;
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int t = i / pairs, j = i - t * pairs;
    const double pos = p.pos64 ? double(static_cast<const int64_t*>(p.positions)[tok0 + t])
                               : double(static_cast<const int32_t*>(p.positions)[tok0 + t]);
    constexpr double kInv2Pi = 0.15915494309189533577;
    const double turns = pos * (p.freqs[unit0 * P + j] * kInv2Pi);
    float sn, cs;
    sincospif(2.0f * float(turns - rint(turns)), &sn, &cs);
    s_c[i] = cs * p.m;
    s_s[i] = (p.adjoint ? -sn : sn) * p.m;
  }
  __syncthreads();
  const int col = threadIdx.x % p.cols, row0 = threadIdx.x / p.cols;
  const int unit = unit0 + col;
  if (row0 >= p.rows || unit >= p.units) return;
  const bool turns = unit < p.turn_units;
  int off0, off1;          // element offsets of the thread's two vectors inside a head
  bool second = true;
  if (turns) {
    const int i0 = unit * P;
    off0 = kInterleaved ? 2 * i0 : i0;
    off1 = kInterleaved ? 2 * i0 + P : p.half + i0;
  } else {
    const int v0 = 2 * (unit - p.turn_units);
    off0 = 2 * p.half + v0 * P;
    off1 = off0 + P;
    second = v0 + 1 < p.copy_vecs;
  }

  const int h_first = blockIdx.z * p.heads, n_heads = min(p.heads, p.q.heads + p.k.heads - h_first);
  const int n = tokens * n_heads;    // (token, head) rows of this CTA
  for (int r0 = row0; r0 < n; r0 += kUnroll * p.rows) {
    V a[kUnroll], b[kUnroll];
    char* dst[kUnroll];
    int tl[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * p.rows;
      if (r < n) {
        tl[u] = r / n_heads;
        const int h = h_first + r - tl[u] * n_heads;
        const bool is_q = h < p.q.heads;
        const Side& sd = is_q ? p.q : p.k;
        const int hh = is_q ? h : h - p.q.heads;
        const char* src = sd.in + (tok0 + tl[u]) * sd.in_tok + hh * sd.in_head;
        dst[u] = sd.out + (tok0 + tl[u]) * sd.out_tok + hh * sd.out_head;
        a[u] = load_once<V>(src + off0 * sizeof(T));
        if (second) b[u] = load_once<V>(src + off1 * sizeof(T));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (r0 + u * p.rows < n) {
        if (turns) {
          const Vec<float, P> c = *reinterpret_cast<const Vec<float, P>*>(s_c + tl[u] * pairs + col * P);
          const Vec<float, P> s = *reinterpret_cast<const Vec<float, P>*>(s_s + tl[u] * pairs + col * P);
          if (kInterleaved && P > 1) {
            // element pairs (2j, 2j + 1) over the two vectors
#pragma unroll
            for (int j = 0; j < P; j += 2) {
              const float x = to_f(a[u].v[j]), y = to_f(a[u].v[j + 1]);
              a[u].v[j] = from_f<T>(x * c.v[j / 2] - y * s.v[j / 2]);
              a[u].v[j + 1] = from_f<T>(y * c.v[j / 2] + x * s.v[j / 2]);
              const float z = to_f(b[u].v[j]), w = to_f(b[u].v[j + 1]);
              b[u].v[j] = from_f<T>(z * c.v[(P + j) / 2] - w * s.v[(P + j) / 2]);
              b[u].v[j + 1] = from_f<T>(w * c.v[(P + j) / 2] + z * s.v[(P + j) / 2]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < P; ++j) {
              const float x = to_f(a[u].v[j]), y = to_f(b[u].v[j]);
              a[u].v[j] = from_f<T>(x * c.v[j] - y * s.v[j]);
              b[u].v[j] = from_f<T>(y * c.v[j] + x * s.v[j]);
            }
          }
        }
        store_once<V>(dst[u] + off0 * sizeof(T), a[u]);
        if (second) store_once<V>(dst[u] + off1 * sizeof(T), b[u]);
      }
    }
  }
}

template <typename T, int P>
cudaError_t launch(const RopeParams& p, bool interleaved, dim3 grid, cudaStream_t s) {
  if (interleaved)
    rope_kernel<T, P, true><<<grid, kThreads, 0, s>>>(p);
  else
    rope_kernel<T, P, false><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

int dtype_bytes(int dt) { return dt == SPLITKV_DTYPE_F32 ? 4 : 2; }

splitkv::Strided side(const splitkv_rope_args& a, const void* ptr, int heads, const int64_t* s) {
  const int64_t es = dtype_bytes(a.dtype);
  return {ptr, a.head_dim * es, 2, {a.num_tokens, heads}, {s[0] * es, s[1] * es}};
}

// One side by itself: pointers, strides within range, and an output whose elements are apart from each other.
bool side_ok(const splitkv_rope_args& a, const void* in, const void* out, int heads, const int64_t* is,
             const int64_t* os) {
  if (heads == 0) return true;
  if (!in || !out) return false;
  const int64_t es = dtype_bytes(a.dtype), d = a.head_dim, n = a.num_tokens;
  const int64_t kMax = int64_t(1) << 44;
  for (int i = 0; i < 2; ++i)
    if (is[i] < 0 || os[i] < 0 || is[i] > kMax || os[i] > kMax) return false;
  if (n > kMax / (1 + is[0] + os[0])) return false;
  if (reinterpret_cast<uintptr_t>(in) % es || reinterpret_cast<uintptr_t>(out) % es) return false;
  const bool token_major = (heads == 1 || os[1] >= d) && (n == 1 || os[0] >= (heads - 1) * os[1] + d);
  const bool head_major = (n == 1 || os[0] >= d) && (heads == 1 || os[1] >= (n - 1) * os[0] + d);
  return token_major || head_major;
}

// An output against one input: exactly that input, where it is its own (in place: a thread reads what it writes), or
// memory apart from it.  Queries and keys share the launch, so each output is held against both inputs.
bool output_ok(const splitkv_rope_args& a, const void* out, int heads, const int64_t* os, const void* in, int in_heads,
               const int64_t* is, bool own) {
  if (heads == 0 || in_heads == 0) return true;
  const bool same = own && in == out && (a.num_tokens == 1 || is[0] == os[0]) && (heads == 1 || is[1] == os[1]);
  return same || splitkv::apart(side(a, out, heads, os), side(a, in, in_heads, is));
}

}  // namespace

extern "C" int splitkv_rope_freqs(int32_t rotary_dim, double base, int scaling, double factor, double original_len,
                                  double turns_low, double turns_high, double* freqs, double* scale) {
  if (rotary_dim < 2 || rotary_dim % 2 || !freqs || !scale || !(base > 0) || !std::isfinite(base) || !(factor > 0) ||
      !std::isfinite(factor))
    return SPLITKV_ERR_INVALID_ARG;
  if (scaling < SPLITKV_ROPE_SCALE_NONE || scaling > SPLITKV_ROPE_SCALE_PARTS) return SPLITKV_ERR_INVALID_ARG;
  if (scaling == SPLITKV_ROPE_SCALE_PARTS && !(original_len > 0 && turns_high > turns_low)) return SPLITKV_ERR_INVALID_ARG;
  if (scaling == SPLITKV_ROPE_SCALE_BASE && rotary_dim > 2) base *= std::pow(factor, double(rotary_dim) / (rotary_dim - 2));
  *scale = 1.0;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double w = std::pow(base, -2.0 * i / rotary_dim);
    if (scaling == SPLITKV_ROPE_SCALE_LINEAR) w /= factor;
    if (scaling == SPLITKV_ROPE_SCALE_PARTS) {
      const double turns = original_len * w / 6.283185307179586476925;
      double keep = (turns - turns_low) / (turns_high - turns_low);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      w = w / factor * (1 - keep) + w * keep;
    }
    freqs[i] = w;
  }
  if (scaling == SPLITKV_ROPE_SCALE_PARTS) *scale = 0.1 * std::log(factor) + 1.0;
  return SPLITKV_OK;
}

extern "C" int splitkv_rope(const splitkv_rope_args* a, void* stream) {
  if (!a) return SPLITKV_ERR_INVALID_ARG;
  if (a->num_tokens < 0 || a->q_heads < 0 || a->k_heads < 0 || a->head_dim < 1 || a->rotary_dim < 2 ||
      a->rotary_dim % 2 || a->rotary_dim > a->head_dim || a->head_dim > 65536 || a->q_heads > 65536 ||
      a->k_heads > 65536)
    return SPLITKV_ERR_INVALID_ARG;
  if (a->dtype != SPLITKV_DTYPE_F32 && a->dtype != SPLITKV_DTYPE_BF16 && a->dtype != SPLITKV_DTYPE_F16)
    return SPLITKV_ERR_INVALID_ARG;
  if (a->flags & ~(SPLITKV_ROPE_INTERLEAVED | SPLITKV_ROPE_ADJOINT | SPLITKV_ROPE_POS64)) return SPLITKV_ERR_INVALID_ARG;
  const int heads = a->q_heads + a->k_heads;
  if (a->num_tokens == 0 || heads == 0) return SPLITKV_OK;
  const bool pos64 = (a->flags & SPLITKV_ROPE_POS64) != 0;
  if (!a->positions || !a->freqs || !splitkv::ptr_aligned(a->positions, pos64 ? 8 : 4) ||
      !splitkv::ptr_aligned(a->freqs, 8))
    return SPLITKV_ERR_INVALID_ARG;
  if (!side_ok(*a, a->q, a->q_out, a->q_heads, a->q_stride, a->q_out_stride) ||
      !side_ok(*a, a->k, a->k_out, a->k_heads, a->k_stride, a->k_out_stride))
    return SPLITKV_ERR_INVALID_ARG;
  if (!output_ok(*a, a->q_out, a->q_heads, a->q_out_stride, a->q, a->q_heads, a->q_stride, true) ||
      !output_ok(*a, a->q_out, a->q_heads, a->q_out_stride, a->k, a->k_heads, a->k_stride, false) ||
      !output_ok(*a, a->k_out, a->k_heads, a->k_out_stride, a->q, a->q_heads, a->q_stride, false) ||
      !output_ok(*a, a->k_out, a->k_heads, a->k_out_stride, a->k, a->k_heads, a->k_stride, true) ||
      !output_ok(*a, a->q_out, a->q_heads, a->q_out_stride, a->k_out, a->k_heads, a->k_out_stride, false))
    return SPLITKV_ERR_INVALID_ARG;

  const int es = dtype_bytes(a->dtype), P = 16 / es;
  // 16-byte accesses need every vector on a 16-byte boundary.  Otherwise a thread moves one element at a time: 40000 tokens of
  // 32 + 8 heads with 100 of 128 elements turned take 434 us in bfloat16 (29 % of the copy rate; 135 us with all 128) and
  // 428 us in float32 (58 %), 24 of 96 334 us (28 %; 48 of 96 105 us, 89 %), both layouts alike.
  bool vec = (a->rotary_dim / 2) % P == 0 && a->head_dim % P == 0;
  const auto fits = [&](const void* in, const void* out, int n, const int64_t* is, const int64_t* os) {
    return n == 0 || (splitkv::ptr_aligned(in, 16) && splitkv::ptr_aligned(out, 16) && is[0] % P == 0 &&
                      is[1] % P == 0 && os[0] % P == 0 && os[1] % P == 0);
  };
  vec = vec && fits(a->q, a->q_out, a->q_heads, a->q_stride, a->q_out_stride) &&
        fits(a->k, a->k_out, a->k_heads, a->k_stride, a->k_out_stride);
  const int pairs = vec ? P : 1;

  RopeParams p;
  p.q = Side{static_cast<const char*>(a->q), static_cast<char*>(a->q_out), a->q_stride[0] * es, a->q_stride[1] * es,
             a->q_out_stride[0] * es, a->q_out_stride[1] * es, a->q_heads};
  p.k = Side{static_cast<const char*>(a->k), static_cast<char*>(a->k_out), a->k_stride[0] * es, a->k_stride[1] * es,
             a->k_out_stride[0] * es, a->k_out_stride[1] * es, a->k_heads};
  p.positions = a->positions;
  p.freqs = a->freqs;
  p.n_tokens = a->num_tokens;
  p.half = a->rotary_dim / 2;
  p.turn_units = p.half / pairs;
  const bool in_place = (a->q_heads == 0 || a->q == a->q_out) && (a->k_heads == 0 || a->k == a->k_out);
  p.copy_vecs = in_place ? 0 : (a->head_dim - a->rotary_dim) / pairs;
  p.units = p.turn_units + (p.copy_vecs + 1) / 2;
  p.m = float(a->scale);
  p.pos64 = pos64;
  p.adjoint = (a->flags & SPLITKV_ROPE_ADJOINT) != 0;

  // A CTA's share: columns of units side by side (all of them, unless a head is very wide), then as many tokens as
  // give every thread two rounds of loads; with few tokens in all, one token and one round of heads, so that a
  // short call spreads over the SMs.
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  p.cols = p.units < 64 ? p.units : 64;
  p.rows = kThreads / p.cols;
  const int64_t gy = (p.units + p.cols - 1) / p.cols;
  const int max_tokens = kMaxPairs / (p.cols * pairs) > 0 ? kMaxPairs / (p.cols * pairs) : 1;
  int tokens = (2 * kUnroll * p.rows + heads - 1) / heads;
  tokens = tokens > max_tokens ? max_tokens : tokens;
  p.tokens = tokens;
  p.heads = heads;
  if ((p.n_tokens + tokens - 1) / tokens * gy < int64_t(4) * sms) {
    p.tokens = 1;
    const int per = p.n_tokens * gy < 2 * sms ? p.rows : kUnroll * p.rows;
    p.heads = per < heads ? per : heads;
  }
  const int64_t blocks = (p.n_tokens + p.tokens - 1) / p.tokens;
  const int64_t gz = (heads + p.heads - 1) / p.heads;
  if (blocks > 0x7fffffff || gy > 65535 || gz > 65535) return SPLITKV_ERR_UNSUPPORTED;
  const dim3 grid{unsigned(blocks), unsigned(gy), unsigned(gz)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool il = (a->flags & SPLITKV_ROPE_INTERLEAVED) != 0;
  cudaError_t e;
  if (a->dtype == SPLITKV_DTYPE_F32)
    e = vec ? launch<float, 4>(p, il, grid, s) : launch<float, 1>(p, il, grid, s);
  else if (a->dtype == SPLITKV_DTYPE_BF16)
    e = vec ? launch<__nv_bfloat16, 8>(p, il, grid, s) : launch<__nv_bfloat16, 1>(p, il, grid, s);
  else
    e = vec ? launch<__half, 8>(p, il, grid, s) : launch<__half, 1>(p, il, grid, s);
  if (e == cudaSuccess) return SPLITKV_OK;
  return SPLITKV_ERR_CUDA;
}
