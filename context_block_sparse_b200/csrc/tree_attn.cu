// Attention of draft trees over a paged cache: every row against its sequence's cached keys and its own
// tree, the work cut over the CTAs (here on mma.sync, for few rows and short contexts; on tcgen05 in
// tree_context_sm100.cu and tree_rows_sm100.cu), and the merge of the rows that were cut.
//
// Per row (node i, query head h) of sequence b, over the keys j of its context [0, len_b) and
// the nodes j of its own tree that mask lets i see, with KV head h / G:
//   s_j = scale q.k_j, m = max s_j, l = sum exp(s_j - m), o = sum exp(s_j - m) v_j / l,
//   lse = m + log l;  a row with no key: o = 0, lse = -inf.
//
// A few rows read a long cache once, so the context kernel is HBM-bound: 4 len_b d bytes a KV
// head.  The G heads of all a sequence's nodes share every key tile (16, 32 or 64 rows of a
// CTA); 64-key tiles flow through a ring of cp.async stages that does not drain at unit
// boundaries, two CTAs to an SM: 128 KB of loads in flight per SM against the ~35 KB that
// 6.5 TB/s at 0.8 us of latency need.  Pages are resolved per key (any power-of-two page size,
// any strides), one tile ahead.  With 16 rows the four warps share the tile by keys, with 64 by
// rows, and softmax statistics stay in registers; scores, maxima, sums and O are float32, P is
// rounded to the keys' type for the second product, as in the training kernels.
#include <cstdint>
#include <cstdlib>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "strided.h"
#include "tree.h"

namespace splitkv {
namespace tree {
namespace {

constexpr int kThreads = 128;
constexpr int kTileKeys = 64;      // keys of a tile
constexpr int kPgRing = 8;         // page-id slots (tiles): at least the stages + 1

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                         __nv_bfloat16) {
  mma_bf16_16816(c, a, b0, b1);
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) { return pack_bf16(lo, hi); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// The A fragments of 16 rows of Q straight from global memory (rows past the tile's are zero):
// thread t holds rows t/4 and t/4 + 8, column pairs 2 (t % 4) of every 8 columns.
template <int D>
__device__ __forceinline__ void load_q(uint32_t (&qf)[D / 16][4], const TreeParams& p, int n0, int n, int head,
                                       int row0) {
  const int lane = threadIdx.x & 31;
  const char* ptr[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = row0 + (lane >> 2) + 8 * k;
    const int node = r / p.G, g = r - node * p.G;
    ptr[k] = node < n ? p.q + int64_t(n0 + node) * p.q_node + int64_t(head * p.G + g) * p.q_head + 4 * (lane & 3)
                      : nullptr;
  }
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const char* base = ptr[e & 1];
      qf[kk][e] = base ? *reinterpret_cast<const uint32_t*>(base + kk * 32 + (e >> 1) * 16) : 0u;
    }
  }
}

// S (16 rows x kKeys keys) = Q K^T, K rows [key0, key0 + kKeys) of a swizzled [64][D] tile.
template <typename T, int D, int kKeys>
__device__ __forceinline__ void scores(float (&s)[kKeys / 8][4], const uint32_t (&qf)[D / 16][4], const T* sk,
                                       int key0) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kKeys / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
  const int row = key0 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
    for (int g = 0; g < kKeys / 16; ++g) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4(b0, b1, b2, b3, sk + swz<D>(row + 16 * g, kk * 2 + ((lane >> 3) & 1)));
      mma16816(s[2 * g], qf[kk], b0, b1, T());
      mma16816(s[2 * g + 1], qf[kk], b2, b3, T());
    }
  }
}

template <typename T>
constexpr int kLift = lift_of(std::is_same_v<T, __half>, false);

// The state of two rows of a thread: reference (the maximum less kLift; log2 units), this thread's share of the sum, and
// the rows' NC columns of O.
template <int NC>
struct Rows {
  float m[2], l[2];
  float o[NC / 8][4];
  __device__ __forceinline__ void clear() {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < NC / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  }
};

// One online-softmax step: s (log2 units, masked scores -inf) against V rows [key0, ...) and
// columns of a swizzled [64][NC] tile.
template <typename T, int NC, int kKeys>
__device__ __forceinline__ void softmax_step(Rows<NC>& st, float (&s)[kKeys / 8][4], const T* sv, int key0) {
  const int lane = threadIdx.x & 31;
  float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < kKeys / 8; ++i) {
    mx[0] = fmaxf(mx[0], fmaxf(s[i][0], s[i][1]));
    mx[1] = fmaxf(mx[1], fmaxf(s[i][2], s[i][3]));
  }
  float ref[2], f[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 1));
    mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 2));
    const float m = fmaxf(st.m[k], mx[k] - float(kLift<T>));
    ref[k] = m == -INFINITY ? 0.f : m;    // no key yet: every exponential below is exp2(-inf) = 0
    f[k] = fast_exp2(st.m[k] - ref[k]);
    st.m[k] = m;
    st.l[k] *= f[k];
  }
#pragma unroll
  for (int i = 0; i < kKeys / 8; ++i) {
    s[i][0] = fast_exp2(s[i][0] - ref[0]);
    s[i][1] = fast_exp2(s[i][1] - ref[0]);
    s[i][2] = fast_exp2(s[i][2] - ref[1]);
    s[i][3] = fast_exp2(s[i][3] - ref[1]);
    st.l[0] += s[i][0] + s[i][1];
    st.l[1] += s[i][2] + s[i][3];
  }
  if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
    for (int i = 0; i < NC / 8; ++i) {
      st.o[i][0] *= f[0];
      st.o[i][1] *= f[0];
      st.o[i][2] *= f[1];
      st.o[i][3] *= f[1];
    }
  }
  const int row = key0 + (lane & 15);
#pragma unroll
  for (int g = 0; g < kKeys / 16; ++g) {
    const uint32_t a[4] = {pack2(s[2 * g][0], s[2 * g][1], T()), pack2(s[2 * g][2], s[2 * g][3], T()),
                           pack2(s[2 * g + 1][0], s[2 * g + 1][1], T()), pack2(s[2 * g + 1][2], s[2 * g + 1][3], T())};
#pragma unroll
    for (int c = 0; c < NC / 16; ++c) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(b0, b1, b2, b3, sv + swz<NC>(row + 16 * g, c * 2 + (lane >> 4)));
      mma16816(st.o[2 * c], a, b0, b1, T());
      mma16816(st.o[2 * c + 1], a, b2, b3, T());
    }
  }
}

// Four elements of a finished row of O.
template <typename T>
__device__ __forceinline__ void store4(const TreeParams& p, size_t at, float4 o, float inv) {
  o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (p.o_f32)
    *reinterpret_cast<float4*>(p.o + at * 4) = o;
  else
    *reinterpret_cast<uint2*>(p.o + at * 2) = make_uint2(pack2(o.x, o.y, T()), pack2(o.z, o.w, T()));
}

// Sixteen rows of a whole unit from the context kernel: each thread's float4s of the sums in s_o, the rows' statistics of
// the kKG warps in s_ml; row0: the first row's number in the unit, whose first node's first head is hr0.  Kept out of the
// kernel's straight code, which a call of one tile a CTA runs once, on a cold instruction cache (one token over 1k keys: 9.5 us,
// 11.3 in line).
template <typename T, int D, int kKG>
__device__ __noinline__ void finish_rows(const TreeParams& p, const float* s_o, const float2 (*s_ml)[16], size_t hr0,
                                         int row0, int rows) {
#pragma unroll 1
  for (int i = 0; i < D / 32; ++i) {
    const int e = (i * kThreads + threadIdx.x) * 4, r = e / D, c = e % D, row = row0 + r;
    if (row >= rows) break;
    float m = -INFINITY, l = 0.f;
    for (int x = 0; x < kKG; ++x) m = fmaxf(m, s_ml[x][r].x);
    for (int x = 0; x < kKG; ++x) l += s_ml[x][r].y * fast_exp2(s_ml[x][r].x - (m == -INFINITY ? 0.f : m));
    const int node = row / p.G;
    const size_t hr = hr0 + size_t(node) * p.Hq + (row - node * p.G);
    store4<T>(p, hr * D + c, *reinterpret_cast<const float4*>(s_o + r * D + (c ^ ((r & 3) << 3))), row_inv(l));
    if (c == 0) p.lse[hr] = row_lse(m, l, kLift<T>);
  }
}

// ---------------------------------------------------------------------------- context kernel
// A CTA's place on the line: the unit and key tile of the tile it points at.
struct Cursor {
  SeqWork w;
  int b, head, rt, tile;     // head: pair of heads where they are walked in pairs
  bool bad;
  __device__ __forceinline__ void enter(const TreeParams& p, int seq, long long rel) {
    b = seq;
    w = seq_work(p, b, bad);
    const long long unit = rel / w.nt;
    tile = int(rel - unit * w.nt);
    head = int(unit / w.rts);
    rt = int(unit - (long long)(head) * w.rts);
  }
  // the next tile of the line; the caller knows that there is one
  __device__ __forceinline__ void step(const TreeParams& p) {
    if (++tile < w.nt) return;
    tile = 0;
    if (++rt < w.rts) return;
    rt = 0;
    if (++head < p.Hkv / p.hg) return;
    head = 0;
    do {
      ++b;
      if (b >= p.B) return;
      w = seq_work(p, b, bad);
    } while (w.places == 0);
  }
};

template <int D, int RG>
struct Cfg {
  static constexpr int kKG = 4 / RG;                    // warps that share a row group's keys
  static constexpr int kKeysW = kTileKeys / kKG;        // keys of a tile that one warp takes
  static constexpr int kStages = D == 128 ? 3 : 5;
  static constexpr int kStageElems = 2 * kTileKeys * D; // K then V
  static constexpr int kSmem = kStages * kStageElems * 2 + 16 * D * 4 /* O exchange */;
};

template <typename T, int D, int RG>
__global__ void __launch_bounds__(kThreads, 2) tree_context_mma_kernel(const __grid_constant__ TreeParams p) {
  using C = Cfg<D, RG>;
  extern __shared__ __align__(1024) uint8_t smem[];
  T* stages = reinterpret_cast<T*>(smem);
  float* s_o = reinterpret_cast<float*>(smem + C::kStages * C::kStageElems * 2);   // [16][D]
  __shared__ long long s_scan[kThreads / 32];
  __shared__ long long s_rel;
  __shared__ long long s_line[2];           // places of the line, the stretch's end
  __shared__ int s_seq, s_ctas;
  __shared__ int s_pg[kPgRing][kTileKeys];
  __shared__ int s_part[kPgRing][2];        // a tile's first and second 32 keys: not all of them are there
  __shared__ float2 s_ml[4][16];
  __shared__ unsigned long long s_flag;     // nodes of a tree tile whose V is not all finite

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rg = warp / C::kKG, kg = warp % C::kKG;

  // this CTA's stretch of the line, and the sequence it begins in
  if (tid == 0) p.split[blockIdx.x].w = -1;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  long long mine = 0, before;
  bool bad = false;
  for (int b = b0; b < b1; ++b) mine += seq_work(p, b, bad).places;
  if (bad && blockIdx.x == 0) atomicCAS(p.status, 0, SPLITKV_ERR_INVALID_ARG);
  const long long W = block_prefix<kThreads>(mine, before, s_scan);
  const int ctas = int(min((long long)(p.ctas), W)), mine_c = blockIdx.x / p.hg, sub = blockIdx.x % p.hg;
  if (mine_c >= ctas) return;
  const long long x0 = stretch(W, mine_c, ctas);
  const int n_tiles = int(stretch(W, mine_c + 1, ctas) - x0);
  if (tid == 0) {
    s_line[0] = W;
    s_line[1] = x0 + n_tiles;
    s_ctas = ctas;
  }
  if (x0 >= before && x0 < before + mine) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const long long t = seq_work(p, b, bad).places;
      if (x0 < at + t) {
        s_seq = b;
        s_rel = x0 - at;
        break;
      }
      at += t;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the merge finds its rows
  __syncthreads();
  Cursor load, use;   // the tile whose pages come next; the tile computed now
  load.bad = use.bad = false;
  use.enter(p, s_seq, s_rel);
  load = use;
  Cursor fill = use;  // the tile whose keys and values are requested next

  // page ids of the `load` cursor's tile, or rows of the tree (-1: no such key), by 64 threads
  auto resolve = [&](int t) {
    if (tid < kTileKeys) {
      int key = load.tile * kTileKeys + tid;
      int page = -1;
      if (load.tile >= load.w.ctx) {           // a tile of the tree: the node's row
        key -= load.w.ctx * kTileKeys;
        if (key < load.w.n) page = load.w.n0 + key;
      } else if (key < load.w.len) {
        page = p.table[load.b * p.table_row + (key >> p.page_shift)];
        if (page < 0 || page >= p.num_pages) {
          page = -1;
          atomicCAS(p.status, 0, SPLITKV_ERR_INVALID_ARG);
        }
      }
      s_pg[t % kPgRing][tid] = page;
      const bool part = __any_sync(0xffffffffu, page < 0);
      if (lane == 0) s_part[t % kPgRing][warp] = part;
    }
  };
  // with `load` at the stretch's last tile: does its unit begin here and end in a later stretch?  Then the merge finds it
  // in `split`
  auto note_split = [&]() {
    const int rest = load.w.nt - load.tile - 1;
    if (tid == kThreads - 1 && load.tile < n_tiles && rest > 0)
      p.split[blockIdx.x] = make_int4(load.w.n0, load.w.n, (load.head * p.hg + sub) | load.rt << 16,
                                      cta_before(s_line[0], s_line[1] + rest, s_ctas));
  };
  constexpr int kChunks = D / 8;                    // 16-byte chunks of a key row
  constexpr int kRowsPer = kThreads / kChunks;      // rows of one pass of the CTA
  auto request = [&](int t) {
    T* sk = stages + (t % C::kStages) * C::kStageElems;
    T* sv = sk + kTileKeys * D;
    const int ch = tid % kChunks;
    const bool tree = fill.tile >= fill.w.ctx;
    const int head = fill.head * p.hg + sub;
    const char* kbase = (tree ? p.kb + head * p.kb_head : p.kc + head * p.kc_head) + ch * 16;
    const char* vbase = (tree ? p.vb + head * p.vb_head : p.vc + head * p.vc_head) + ch * 16;
    const int64_t kpage = tree ? p.kb_node : p.kc_page, kslot = tree ? 0 : p.kc_slot;
    const int64_t vpage = tree ? p.vb_node : p.vc_page, vslot = tree ? 0 : p.vc_slot;
    const int slot_mask = (1 << p.page_shift) - 1;
#pragma unroll
    for (int i = 0; i < kTileKeys / kRowsPer; ++i) {
      const int r = tid / kChunks + i * kRowsPer;
      const int page = s_pg[t % kPgRing][r];
      const int slot = (fill.tile * kTileKeys + r) & slot_mask;
      const bool there = page >= 0;
      const int64_t pg = there ? page : 0, sl = there ? slot : 0;
      cp_async16(sk + swz<D>(r, ch), kbase + pg * kpage + sl * kslot, there);
      cp_async16(sv + swz<D>(r, ch), vbase + pg * vpage + sl * vslot, there);
    }
  };

  for (int t = 0; t < C::kStages && t < n_tiles; ++t) {
    resolve(t);
    if (t + 1 < n_tiles) load.step(p);
  }
  __syncthreads();
  for (int t = 0; t < C::kStages - 1; ++t) {
    if (t < n_tiles) {
      request(t);
      if (t + 1 < n_tiles) fill.step(p);
    }
    cp_async_commit();
  }
  if (n_tiles <= C::kStages) note_split();

  uint32_t qf[D / 16][4];
  Rows<D> st;
  bool fresh = true, from_start = false;   // at the first tile of this CTA's part of a unit; that part is its first
  for (int t = 0; t < n_tiles; ++t) {
    cp_async_wait<C::kStages - 2>();
    __syncthreads();   // tile t has landed; every warp is done with tile t - 1's stage
    if (t + C::kStages - 1 < n_tiles) {
      request(t + C::kStages - 1);
      if (t + C::kStages < n_tiles) fill.step(p);
    }
    cp_async_commit();
    if (t + C::kStages < n_tiles) {
      resolve(t + C::kStages);
      if (t + C::kStages + 1 < n_tiles)
        load.step(p);
      else
        note_split();
    }
    if (fresh) {
      load_q<D>(qf, p, use.w.n0, use.w.n, use.head * p.hg + sub, use.rt * p.Mt + rg * 16);
      st.clear();
      fresh = false;
      from_start = use.tile == 0;
    }
    T* sk = stages + (t % C::kStages) * C::kStageElems;
    float s[C::kKeysW / 8][4];
    scores<T, D, C::kKeysW>(s, qf, sk, kg * C::kKeysW);
    const int tree0 = use.tile >= use.w.ctx ? (use.tile - use.w.ctx) * kTileKeys : -1;   // a tree tile's first node
    if (tree0 >= 0) {
      // A node's V may hold infinities or NaN that only the rows which see it may meet, but the product multiplies
      // every V by P = 0 elsewhere: take such values out here and add them back where they are seen.
      if (tid == 0) s_flag = 0;
      __syncthreads();
      const int here = min(kTileKeys, use.w.n - tree0);
#pragma unroll 2
      for (int i = tid; i < here * kChunks; i += kThreads) {
        uint4* at = reinterpret_cast<uint4*>(sk + kTileKeys * D + swz<D>(i / kChunks, i % kChunks));
        uint4 x = *at;
        if (take_out<T>(x)) {
          *at = x;
          atomicOr(&s_flag, 1ull << (i / kChunks));
        }
      }
      __syncthreads();
    }
    // row r of this thread's two: what it sees of the tree
    auto sees = [&](int k, int j) -> bool {
      const int node = (use.rt * p.Mt + rg * 16 + (lane >> 2) + 8 * k) / p.G;
      return j < use.w.n && (p.mask == nullptr || (node < use.w.n && p.mask[int64_t(use.w.n0 + node) * p.mask_row + j]));
    };
    const bool part = s_part[t % kPgRing][0] || s_part[t % kPgRing][1];
#pragma unroll
    for (int i = 0; i < C::kKeysW / 8; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] *= p.scale_log2;
      if (part) {
        const int col = kg * C::kKeysW + 8 * i + 2 * (lane & 3);
        if (s_pg[t % kPgRing][col] < 0) s[i][0] = s[i][2] = -INFINITY;
        if (s_pg[t % kPgRing][col + 1] < 0) s[i][1] = s[i][3] = -INFINITY;
      }
      if (tree0 >= 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!sees(e >> 1, tree0 + kg * C::kKeysW + 8 * i + 2 * (lane & 3) + (e & 1))) s[i][e] = -INFINITY;
      }
    }
    softmax_step<T, D, C::kKeysW>(st, s, sk + kTileKeys * D, kg * C::kKeysW);
    if (tree0 >= 0) {
      unsigned long long flag = s_flag >> (kg * C::kKeysW);
      if (C::kKeysW < 64) flag &= (1ull << (C::kKeysW & 63)) - 1;
      while (flag) {
        const int j = tree0 + kg * C::kKeysW + __ffsll(flag) - 1;
        flag &= flag - 1;
        const bool see[2] = {sees(0, j), sees(1, j)};
        const T* v = reinterpret_cast<const T*>(p.vb + int64_t(use.w.n0 + j) * p.vb_node +
                                                (use.head * p.hg + sub) * p.vb_head);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = float(v[8 * i + 2 * (lane & 3) + (e & 1)]);
            if (!isfinite(x) && see[e >> 1]) st.o[i][e] += x;
          }
      }
    }

    const bool last = t + 1 == n_tiles || use.tile + 1 == use.w.nt;
    if (last) {
      // the unit's part of this CTA is complete: add the key groups; write the record, or, of a whole unit, the rows
      const int rest = use.w.nt - use.tile - 1, head = use.head * p.hg + sub, row0 = use.rt * p.Mt;
      const int rec = from_start ? (rest > 0 ? 2 * int(blockIdx.x) + 1 : -1) : 2 * int(blockIdx.x);
      const int rows = min(p.Mt, use.w.n * p.G - row0);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        st.l[k] += __shfl_xor_sync(0xffffffffu, st.l[k], 1);
        st.l[k] += __shfl_xor_sync(0xffffffffu, st.l[k], 2);
        if ((lane & 3) == 0) s_ml[warp][(lane >> 2) + 8 * k] = make_float2(st.m[k], st.l[k]);
      }
      __syncthreads();
      float f[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = (lane >> 2) + 8 * k;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int x = 0; x < C::kKG; ++x) m = fmaxf(m, s_ml[rg * C::kKG + x][r].x);
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int x = 0; x < C::kKG; ++x) l += s_ml[rg * C::kKG + x][r].y * fast_exp2(s_ml[rg * C::kKG + x][r].x - ref);
        f[k] = fast_exp2(st.m[k] - ref);
        if (rec >= 0 && kg == 0 && (lane & 3) == 0 && rg * 16 + r < rows)
          p.rec_ml[size_t(rec) * p.Mt + rg * 16 + r] = make_float2(m, l);
      }
      float4 acc[D / 32];   // this thread's float4s of the [16][D] block
#pragma unroll 1
      for (int w = 0; w < 4; ++w) {
        if (warp == w) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              *reinterpret_cast<float2*>(s_o + ((lane >> 2) + 8 * k) * D +
                                         ((8 * i + 2 * (lane & 3)) ^ (((lane >> 2) & 3) << 3))) =
                  make_float2(st.o[i][2 * k] * f[k], st.o[i][2 * k + 1] * f[k]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const int e = (i * kThreads + tid) * 4, r = e / D, c = e % D;
          const float4 x = *reinterpret_cast<const float4*>(s_o + r * D + (c ^ ((r & 3) << 3)));
          if (w % C::kKG == 0)
            acc[i] = x;
          else
            acc[i] = make_float4(acc[i].x + x.x, acc[i].y + x.y, acc[i].z + x.z, acc[i].w + x.w);
          if (w % C::kKG == C::kKG - 1) {
            const int row = (w / C::kKG) * 16 + r;
            float* dst = rec >= 0 ? p.rec_o + (size_t(rec) * p.Mt + row) * D + c : s_o + r * D + (c ^ ((r & 3) << 3));
            if (rec < 0 || row < rows) *reinterpret_cast<float4*>(dst) = acc[i];
          }
        }
        if (rec < 0 && w % C::kKG == C::kKG - 1) {
          const int g = w / C::kKG;
          finish_rows<T, D, C::kKG>(p, s_o, s_ml + g * C::kKG, size_t(use.w.n0) * p.Hq + head * p.G, row0 + g * 16,
                                    row0 + rows);
        }
        __syncthreads();
      }
      fresh = true;
    }
    if (t + 1 < n_tiles) use.step(p);
  }
  cp_async_wait<0>();
}

// ------------------------------------------------------------------------------------ merge
// A block per split unit and some of its rows (4 at d = 128, 8 at d = 64), a thread per four elements of a row: the
// row's records in CTA order, each weighted by exp2(m_x - max m) (a record without keys has m = -inf, l = 0).  A
// stream over the records, a few microseconds; launched early, it waits while they are still being written.  (Two
// sequences of 9 nodes over 10k keys, 74 records a row: 30 us a call with two rows a thread one after the other, 26 with one.
// 16 ragged trees of 16 nodes take 62 us either way, 67 with blocks of 256 threads, 71 of 64.)
constexpr int kMergeThreads = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const TreeParams p) {
  constexpr int kRows = kMergeThreads / (D / 4);
  const int first = blockIdx.x, c = threadIdx.x % (D / 4) * 4;       // the CTA in whose stretch the unit begins
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 u = p.split[first];
  if (u.w < 0) return;
  const int head = u.z & 0xffff, row0 = (u.z >> 16) * p.Mt, n_rec = u.w - first / p.hg + 1;
  const int r = blockIdx.y * kRows + threadIdx.x / (D / 4);
  if (r >= min(p.Mt, u.y * p.G - row0)) return;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = 8;
#pragma unroll 1
  for (int k0 = 0; k0 < n_rec; k0 += kBatch) {
    float2 ml[kBatch];
    float4 y[kBatch];
    float nm = m;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
      if (k0 + k < n_rec) {
        const size_t at = size_t(k0 + k == 0 ? 2 * first + 1 : 2 * (first + (k0 + k) * p.hg)) * p.Mt + r;
        ml[k] = p.rec_ml[at];
        y[k] = *reinterpret_cast<const float4*>(p.rec_o + at * D + c);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) nm = fmaxf(nm, ml[k].x);
    const float ref = nm == -INFINITY ? 0.f : nm;
    const float f0 = fast_exp2(m - ref);
    l *= f0;
    o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (k0 + k < n_rec) {
        const float f = fast_exp2(ml[k].x - ref);
        l += ml[k].y * f;
        o = make_float4(o.x + y[k].x * f, o.y + y[k].y * f, o.z + y[k].z * f, o.w + y[k].w * f);
      }
    }
    m = nm;
  }
  const size_t hr = size_t(u.x + (row0 + r) / p.G) * p.Hq + head * p.G + (row0 + r) % p.G;
  store4<T>(p, hr * D + c, o, row_inv(l));
  if (c == 0) p.lse[hr] = row_lse(m, l, p.lift);
}

template <typename T, int D, int RG>
cudaError_t context(const TreeParams& p, cudaStream_t s) {
  constexpr int kSmem = Cfg<D, RG>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(tree_context_mma_kernel<T, D, RG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmem);
  if (e != cudaSuccess) return e;
  tree_context_mma_kernel<T, D, RG><<<p.ctas * p.hg, kThreads, kSmem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t context_rows(const TreeParams& p, cudaStream_t s) {
  return p.Mt == 16 ? context<T, D, 1>(p, s) : p.Mt == 32 ? context<T, D, 2>(p, s) : context<T, D, 4>(p, s);
}

template <typename T, int D>
cudaError_t merge(const TreeParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.ctas * p.hg, p.Mt / (kMergeThreads / (D / 4)));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<T, D>, p);
}

}  // namespace

cudaError_t launch_tree_context_mma(const TreeParams& p, int dtype, cudaStream_t s) {
  if (dtype == SPLITKV_DTYPE_BF16)
    return p.d == 128 ? context_rows<__nv_bfloat16, 128>(p, s) : context_rows<__nv_bfloat16, 64>(p, s);
  return p.d == 128 ? context_rows<__half, 128>(p, s) : context_rows<__half, 64>(p, s);
}

cudaError_t launch_tree_merge(const TreeParams& p, int dtype, cudaStream_t s) {
  if (dtype == SPLITKV_DTYPE_BF16) return p.d == 128 ? merge<__nv_bfloat16, 128>(p, s) : merge<__nv_bfloat16, 64>(p, s);
  return p.d == 128 ? merge<__half, 128>(p, s) : merge<__half, 64>(p, s);
}

}  // namespace tree
}  // namespace splitkv

// -------------------------------------------------------------------------------- C entries
namespace {

using splitkv::tree::TreeParams;

struct TreeSizes {
  int Mt, hg, ctas, tile_shift;
  size_t ml_off, split_off, status_off, total;
};

int sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaGetLastError();
  return sms;
}

// Whether tensor maps can describe the cache and the nodes' keys and values: pages of 8 tokens or more (a swizzle atom), and a
// stride for every dimension longer than one.
bool maps_ok(const splitkv_tree_args* a) {
  const auto side = [&](const int64_t* s) {
    return (a->num_pages == 1 || s[0] > 0) && s[1] > 0 && (a->num_kv_heads == 1 || s[2] > 0);
  };
  const auto rows = [&](const int64_t* s) {
    return (a->num_nodes == 1 || s[0] > 0) && (a->num_kv_heads == 1 || s[1] > 0);
  };
  return a->page_size >= 8 && a->num_pages > 0 && a->max_pages > 0 && side(a->k_stride) && side(a->v_stride) &&
         rows(a->kb_stride) && rows(a->vb_stride) && splitkv::tensor_maps_available();
}

// SPLITKV_TREE_KERNEL=mma or =tcgen05 in the environment asks for one of the context kernels.
char asked_kernel() {
  const char* e = std::getenv("SPLITKV_TREE_KERNEL");
  return e ? e[0] : 0;
}

int check_sizes(const splitkv_tree_args* a, TreeSizes* z) {
  if (!a || a->num_seqs < 0 || a->num_nodes < 0 || a->max_nodes < 1 || a->num_kv_heads < 1 || a->num_q_heads < 1 ||
      a->num_q_heads % a->num_kv_heads || a->num_pages < 0 || a->max_pages < 0)
    return SPLITKV_ERR_INVALID_ARG;
  if (a->page_size < 1 || a->page_size > 65536 || (a->page_size & (a->page_size - 1))) return SPLITKV_ERR_INVALID_ARG;
  if (a->dtype != SPLITKV_DTYPE_BF16 && a->dtype != SPLITKV_DTYPE_F16) return SPLITKV_ERR_INVALID_ARG;
  if (a->o_dtype != a->dtype && a->o_dtype != SPLITKV_DTYPE_F32) return SPLITKV_ERR_INVALID_ARG;
  if (a->head_dim != 64 && a->head_dim != 128) return SPLITKV_ERR_UNSUPPORTED;
  if (a->max_nodes > splitkv::tree::kMaxNodes || a->num_q_heads > 1024 || a->num_seqs > 65536)
    return SPLITKV_ERR_UNSUPPORTED;
  if (int64_t(a->max_pages) * a->page_size > 0x7fffffff - 128) return SPLITKV_ERR_UNSUPPORTED;
  const int rows = a->num_q_heads / a->num_kv_heads * a->max_nodes;
  // Up to 16 rows both kernels are fit: mma.sync starts sooner and its units are cheap, tcgen05 streams faster.  The
  // lengths are on the device, so the choice goes by the longest context the tables can name: 64 sequences of one node
  // and 8 heads of d = 128 took (mma.sync / tcgen05) 70 / 74 us over 1k keys, 205 / 175 us over 4k; at d = 64
  // 33 / 34 us over 512 and 148 / 95 us over 4k; one sequence over 1k 12.4 / 14.5 us.
  const bool far = int64_t(a->max_pages) * a->page_size >= 2048;
  const char ask = asked_kernel();
  const bool tc = maps_ok(a) && ask != 'm' && (rows > 16 || far || ask == 't');
  if (tc)
    z->Mt = rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
  else
    z->Mt = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  z->tile_shift = tc ? 7 : 6;
  const size_t units = size_t(a->num_seqs) * a->num_kv_heads * ((rows + z->Mt - 1) / z->Mt);
  // One tcgen05 CTA to an SM (two at d = 64 and few rows), two of mma.sync, and no more than the longest line has tiles.
  z->hg = a->head_dim == 64 && a->num_kv_heads % 2 == 0 ? 2 : 1;
  const size_t round = (size_t(1) << z->tile_shift) - 1;
  const size_t tiles = units / z->hg * (((size_t(a->max_pages) * a->page_size + round) >> z->tile_shift) +
                                           ((size_t(a->max_nodes) + round) >> z->tile_shift));
  const size_t ctas = size_t(tc && !(a->head_dim == 64 && z->Mt <= 64) ? 1 : 2) * sm_count() / z->hg;
  z->ctas = int(tiles < ctas ? (tiles > 0 ? tiles : 1) : ctas);
  const size_t ctas_all = size_t(z->ctas) * z->hg;
  z->ml_off = splitkv::align_up(2 * ctas_all * z->Mt * a->head_dim * sizeof(float), 256);
  z->split_off = z->ml_off + splitkv::align_up(2 * ctas_all * z->Mt * sizeof(float2), 256);
  z->status_off = z->split_off + splitkv::align_up(ctas_all * sizeof(int4), 256);
  z->total = z->status_off + 256;
  return SPLITKV_OK;
}

// A row-strided 16-bit array read in 16-byte pieces.
bool rows_ok(const void* ptr, int64_t s0, int64_t s1, int64_t s2 = 0) {
  const int64_t kMax = int64_t(1) << 38;   // elements; a tensor map's strides stay below 2^40 bytes
  return ptr && splitkv::ptr_aligned(ptr, 16) && s0 >= 0 && s1 >= 0 && s2 >= 0 && s0 < kMax && s1 < kMax &&
         s2 < kMax && s0 % 8 == 0 && s1 % 8 == 0 && s2 % 8 == 0;
}

// o, lse and the workspace share no memory with each other and with what the call reads, but o may be q itself (a
// unit's rows are read before they are written, and by that unit alone).
bool outputs_apart(const splitkv_tree_args* a, const void* ws, size_t ws_bytes) {
  using splitkv::Strided;
  const int64_t nq = a->num_nodes, hq = a->num_q_heads, hkv = a->num_kv_heads, row = 2 * a->head_dim;
  const int64_t es = a->o_dtype == SPLITKV_DTYPE_F32 ? 4 : 2;
  const auto nodes = [&](const void* ptr, const int64_t* s, int64_t heads) {
    return Strided{ptr, row, 2, {nq, heads}, {s[0] * 2, s[1] * 2}};
  };
  const auto cache = [&](const void* ptr, const int64_t* s) {
    return Strided{ptr, row, 3, {a->num_pages, a->page_size, hkv}, {s[0] * 2, s[1] * 2, s[2] * 2}};
  };
  const Strided out[3] = {{a->o, nq * hq * a->head_dim * es, 0, {}, {}}, {a->lse, nq * hq * 4, 0, {}, {}},
                          {ws, int64_t(ws_bytes), 0, {}, {}}};
  const Strided in[5] = {nodes(a->q, a->q_stride, hq), nodes(a->kb, a->kb_stride, hkv), nodes(a->vb, a->vb_stride, hkv),
                         cache(a->k_cache, a->k_stride), cache(a->v_cache, a->v_stride)};
  const int n_in = a->max_pages > 0 && a->num_pages > 0 ? 5 : 3;
  const bool in_place = a->o == a->q && es == 2 && (hq == 1 || a->q_stride[1] == a->head_dim) &&
                        (nq == 1 || a->q_stride[0] == hq * a->head_dim);
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      if (!splitkv::apart(out[i], out[j])) return false;
    for (int j = i == 0 && in_place ? 1 : 0; j < n_in; ++j)
      if (!splitkv::apart(out[i], in[j])) return false;
  }
  return true;
}

}  // namespace

extern "C" int splitkv_tree_workspace_size(const splitkv_tree_args* args, size_t* bytes) {
  if (!bytes) return SPLITKV_ERR_INVALID_ARG;
  TreeSizes z;
  const int st = check_sizes(args, &z);
  if (st == SPLITKV_OK) *bytes = z.total;
  return st;
}

extern "C" int splitkv_tree_attn(const splitkv_tree_args* a, void* ws, size_t ws_bytes, void* stream) {
  TreeSizes z;
  const int st = check_sizes(a, &z);
  if (st != SPLITKV_OK) return st;
  if (a->num_seqs == 0 || a->num_nodes == 0) return SPLITKV_OK;
  if (!rows_ok(a->q, a->q_stride[0], a->q_stride[1]) || !rows_ok(a->kb, a->kb_stride[0], a->kb_stride[1]) ||
      !rows_ok(a->vb, a->vb_stride[0], a->vb_stride[1]) || !splitkv::all_aligned16(a->o, ws) || !a->lse ||
      !a->node_ptr || !a->context_lens || !splitkv::all_aligned4(a->lse, a->node_ptr, a->context_lens, a->status))
    return SPLITKV_ERR_INVALID_ARG;
  if (a->mask && a->mask_stride < 0) return SPLITKV_ERR_INVALID_ARG;
  // (the page table is read even where the cache has no page: every entry is then a bad one)
  if (a->max_pages > 0 && (!a->page_table || !splitkv::ptr_aligned(a->page_table, 4) || a->table_stride < 0))
    return SPLITKV_ERR_INVALID_ARG;
  if (a->max_pages > 0 && a->num_pages > 0 &&
      (!rows_ok(a->k_cache, a->k_stride[0], a->k_stride[1], a->k_stride[2]) ||
       !rows_ok(a->v_cache, a->v_stride[0], a->v_stride[1], a->v_stride[2])))
    return SPLITKV_ERR_INVALID_ARG;
  if (ws_bytes < z.total) return SPLITKV_ERR_WORKSPACE_TOO_SMALL;
  if (!outputs_apart(a, ws, z.total)) return SPLITKV_ERR_INVALID_ARG;
  TreeParams p;
  p.q = static_cast<const char*>(a->q);
  p.kb = static_cast<const char*>(a->kb);
  p.vb = static_cast<const char*>(a->vb);
  p.kc = static_cast<const char*>(a->k_cache);
  p.vc = static_cast<const char*>(a->v_cache);
  p.o = static_cast<char*>(a->o);
  p.lse = a->lse;
  p.mask = static_cast<const uint8_t*>(a->mask);
  p.node_ptr = a->node_ptr;
  p.lens = a->context_lens;
  p.table = a->page_table;
  p.status = a->status ? a->status : reinterpret_cast<int*>(static_cast<char*>(ws) + z.status_off);
  p.q_node = a->q_stride[0] * 2;
  p.q_head = a->q_stride[1] * 2;
  p.kb_node = a->kb_stride[0] * 2;
  p.kb_head = a->kb_stride[1] * 2;
  p.vb_node = a->vb_stride[0] * 2;
  p.vb_head = a->vb_stride[1] * 2;
  p.kc_page = a->k_stride[0] * 2;
  p.kc_slot = a->k_stride[1] * 2;
  p.kc_head = a->k_stride[2] * 2;
  p.vc_page = a->v_stride[0] * 2;
  p.vc_slot = a->v_stride[1] * 2;
  p.vc_head = a->v_stride[2] * 2;
  p.mask_row = a->mask_stride;
  p.table_row = a->table_stride;
  p.B = a->num_seqs;
  p.Nq = a->num_nodes;
  p.T = a->max_nodes;
  p.Hq = a->num_q_heads;
  p.Hkv = a->num_kv_heads;
  p.G = a->num_q_heads / a->num_kv_heads;
  p.d = a->head_dim;
  p.Mt = z.Mt;
  p.tile_shift = z.tile_shift;
  // A unit on tcgen05 costs about as much as three tiles more than its tiles (first references, queries, record): 16 ragged
  // trees over 1k-8k took 75 us with none, 68 with three.  The mma.sync kernel's units are cheap.
  p.lead = z.tile_shift == 7 ? 3 : 0;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a->page_size) ++p.page_shift;
  p.num_pages = a->num_pages;
  p.max_pages = a->max_pages;
  p.hg = z.hg;
  p.ctas = z.ctas;
  p.o_f32 = a->o_dtype == SPLITKV_DTYPE_F32;
  p.lift = splitkv::tree::lift_of(a->dtype == SPLITKV_DTYPE_F16, z.tile_shift == 7);
  // (a scale of 0 as a tiny one: scores stay 0 for any finite product, and a masked score can still be -inf)
  p.scale_log2 = a->scale == 0.f ? 1e-30f : a->scale * splitkv::kLog2e;
  p.rec_o = static_cast<float*>(ws);
  p.rec_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + z.ml_off);
  p.split = reinterpret_cast<int4*>(static_cast<char*>(ws) + z.split_off);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = z.tile_shift == 7 ? splitkv::tree::launch_tree_context_sm100(p, a->dtype, s)
                                    : splitkv::tree::launch_tree_context_mma(p, a->dtype, s);
  if (e == cudaSuccess) e = splitkv::tree::launch_tree_merge(p, a->dtype, s);
  if (e == cudaSuccess) return SPLITKV_OK;
  cudaGetLastError();
  return SPLITKV_ERR_CUDA;
}
