// Shared by the tree-attention kernels: the device view of a call, and how the context work
// is cut over the CTAs of a launch.  Not part of the public ABI.
//
// A unit is one (sequence, KV head, row tile): up to Mt rows (node-major, the G query heads
// of a node next to each other) against the sequence's whole context and then its own tree, in
// key tiles of 64 or 128 keys (a tile holds one kind).  All units' tiles lie on one line, in
// (sequence, KV head, row tile, key tile) order, each unit behind `lead` empty places that stand
// for what a unit costs besides its tiles, and
// CTA c of C takes the stretch [c W / C, (c + 1) W / C) of its W places: every CTA has the same
// work to within a tile, whatever the lengths, and the lengths stay on the device (a
// captured graph replays with new ones).  A unit that lies in one stretch is finished there.  Of the
// others, at most one that begins earlier and one that ends later in a stretch, a CTA writes its part as
// a record (unnormalised O, row maximum, row sum), number 2 c for the former and 2 c + 1 for the latter;
// the CTA where a unit begins notes it in `split`, and the merge joins the records of at most C units, in
// a fixed order and without atomics.  (With a record for every unit and a merge of all of them, 256
// sequences of 4 nodes over 256 keys took 148 us, 26 of them in the merge.)
//
// A key of d = 64 is a 128-byte row beside its neighbouring heads', and HBM brings more than that at a
// time (64 sequences of 8 heads over 4k read 804 MB for 537 MB of keys and values).  So at d = 64 two
// neighbouring heads are walked by two CTAs in step (`hg` = 2): the line is cut over pairs of heads, and
// CTA 2 c + e takes head e of each pair in stretch c.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "splitkv.h"
#include "splitkv_internal.h"

namespace splitkv {

// Paged cache [pages][slots][heads][d] of 16-bit elements with any strides (bytes, multiples of 16),
// box {64, 1, box_slots, 1}, 128-byte swizzle, zero fill out of bounds.
bool make_page_map_4d(void* map, const void* base, bool f16, uint64_t d, uint64_t heads, uint64_t slots, uint64_t pages,
                      int64_t head_bytes, int64_t slot_bytes, int64_t page_bytes, uint32_t box_slots);   // (tensor_maps.cpp)

namespace tree {

constexpr int kMaxNodes = 256;     // nodes of a sequence
// P = exp2(s - reference) is rounded to the keys' type for the product with V.  float16 has 2^-14 .. 2^15 with all bits and
// ends at 2^-24, so there the reference lies this many powers of two below the row's maximum, and P runs up to 2^15: with P up
// to 1, a long context 18 (nats) below one dominating key of small V was rounded away.  A weight is then held to half a step
// of itself, or to 2^-(25 + lift) of the row's largest where that is more.  On mma.sync the reference is the running
// maximum itself; on tcgen05 it may stay behind it by `headroom` (rescaling O costs a tile's time), which takes its
// share of the range: 8 for bfloat16, whose range is float32's, 3 for float16 (18 nats are 26 powers of two: 12 - 26 = -14).
constexpr int lift_of(bool f16, bool tcgen05) { return f16 ? (tcgen05 ? 12 : 15) : 0; }
constexpr int headroom_of(bool f16) { return f16 ? 3 : 8; }
// On tcgen05: row tiles that are rows as M (tree_rows_sm100.cu); the others are rows as N (tree_context_sm100.cu).  N / M
// measured: 256 rows, d = 128, 4 x 64 nodes over 68k to 79k 427 / 335 us (now 327); 128 rows (32 nodes of G = 4, 8 KV heads): d = 64,
// 128 sequences over 4k 404 / 302, 32 over 1k 52 / 49, one over 2k 20.7 / 20.6; d = 128, 128 over 4k 467 / 434, but 32 over
// 1k 62 / 72, one over 64k 70 / 79; 64 rows, d = 64, 64 over 4k 124 / 154.
constexpr bool rows_as_m(int Mt, int d) { return Mt == 256 || (Mt == 128 && d == 64); }

struct TreeParams {
  const char *q, *kb, *vb, *kc, *vc;
  char* o;
  float* lse;
  const uint8_t* mask;             // NULL: a node sees every node of its sequence
  const int *node_ptr, *lens, *table;
  int* status;                     // two words: code, site of a timed-out wait
  // strides in bytes
  int64_t q_node, q_head, kb_node, kb_head, vb_node, vb_head;
  int64_t kc_page, kc_slot, kc_head, vc_page, vc_slot, vc_head;
  int64_t mask_row, table_row;     // elements
  int B, Nq, T, Hq, Hkv, G, d;
  int Mt;                          // rows of a row tile
  int lead;                        // empty places before a unit's tiles
  int tile_shift;                  // log2 of the keys of a tile: 6 (mma.sync) or 7 (tcgen05)
  int page_shift, num_pages, max_pages;
  int hg;                          // neighbouring heads that as many CTAs walk in step: 1 or 2
  int ctas;                        // C: stretches; the context kernel has C hg CTAs
  int o_f32;
  int lift;                        // powers of two from a row's reference up to its maximum (lift_of)
  float scale_log2;
  float* rec_o;                    // [2 hg C][Mt][d]
  float2* rec_ml;                  // [2 hg C][Mt]: reference (log2 units), sum
  int4* split;                     // [hg C]: the unit that begins in this CTA's stretch and ends in a later one:
                                   // first node, nodes, head + (row tile << 16), the last stretch (-1: none)
};

#ifdef __CUDACC__

// Nodes, first row and context length of sequence b as the kernels take them: what lies
// outside the call's arrays counts as nothing (the context kernel records the error).
__device__ __forceinline__ int seq_nodes(const TreeParams& p, int b, int& n0, bool& bad) {
  n0 = p.node_ptr[b];
  const int n1 = p.node_ptr[b + 1];
  if (n0 < 0 || n1 < n0 || n1 > p.Nq || n1 - n0 > p.T) {
    bad = true;
    return 0;
  }
  return n1 - n0;
}
__device__ __forceinline__ int seq_len(const TreeParams& p, int b, bool& bad) {
  const int len = p.lens[b];
  const int64_t cap = int64_t(p.max_pages) << p.page_shift;
  if (len < 0 || len > cap) {
    bad = true;
    return len < 0 ? 0 : int(cap);
  }
  return len;
}

struct SeqWork {
  int n0, n, len, rts;       // first node, nodes, context length, row tiles
  int ctx, nt;               // context tiles of a unit, and all of them
  long long places;          // Hkv / hg * rts * (lead + nt)
};

__device__ __forceinline__ SeqWork seq_work(const TreeParams& p, int b, bool& bad) {
  SeqWork w;
  w.n = seq_nodes(p, b, w.n0, bad);
  w.len = seq_len(p, b, bad);
  w.rts = (w.n * p.G + p.Mt - 1) / p.Mt;
  const int round = (1 << p.tile_shift) - 1;
  w.ctx = (w.len + round) >> p.tile_shift;
  w.nt = w.ctx + ((w.n + round) >> p.tile_shift);
  w.places = (long long)(p.Hkv / p.hg) * w.rts * (p.lead + w.nt);
  return w;
}

// Block-wide: exclusive prefix of the threads' sums (each thread takes consecutive
// sequences), through `scratch` [kThreads / 32 + 1].  Returns the total.
template <int kThreads>
__device__ __forceinline__ long long block_prefix(long long mine, long long& before, long long* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  long long add = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) add += scratch[w];
    all += scratch[w];
  }
  before = add + inc - mine;
  return all;
}

// First place of CTA c's stretch (c in [0, C]); C never exceeds the line's length W.
__device__ __forceinline__ long long stretch(long long W, int c, int C) { return W * c / C; }

// The CTA whose stretch holds place x - 1: the last c with c W < x C.
__device__ __forceinline__ int cta_before(long long W, long long x, int C) {
  long long c = (long long)(float(x) * float(C) / float(W));   // (off by one at most)
  while (c * W >= x * C) --c;
  while ((c + 1) * W < x * C) ++c;
  return int(c);
}

// A finished row: what O's sums are multiplied by, and its lse (m: the row's reference, `lift` below its maximum; adding
// that back and taking it out of l costs nothing and keeps the logarithm small).
__device__ __forceinline__ float row_inv(float l) { return l == 0.f ? 0.f : 1.f / l; }   // no key: o = 0 (a NaN stays NaN)
__device__ __forceinline__ float row_lse(float m, float l, int lift) {
  const float down = __int_as_float((127 - lift) << 23);   // 2^-lift
  return l == 0.f ? -INFINITY : ((m + float(lift)) + log2f(l * down)) * 0.693147180559945309f;
}

// Infinities and NaN among the 16-bit values of x are replaced by 0; returns whether there were any.
template <typename T>
__device__ __forceinline__ bool take_out(uint4& x);
__device__ __forceinline__ bool take_out_bits(uint4& x, uint32_t exponent) {
  uint32_t* w = &x.x;
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= __vcmpeq2(w[i] & exponent, exponent);
  if (any == 0) return false;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] &= ~__vcmpeq2(w[i] & exponent, exponent);
  return true;
}
template <>
__device__ __forceinline__ bool take_out<__nv_bfloat16>(uint4& x) {
  return take_out_bits(x, 0x7f807f80u);
}
template <>
__device__ __forceinline__ bool take_out<__half>(uint4& x) {
  return take_out_bits(x, 0x7c007c00u);
}

#endif  // __CUDACC__

// ---- launchers
cudaError_t launch_tree_context_mma(const TreeParams& p, int dtype, cudaStream_t s);
cudaError_t launch_tree_context_sm100(const TreeParams& p, int dtype, cudaStream_t s);
cudaError_t launch_tree_merge(const TreeParams& p, int dtype, cudaStream_t s);

}  // namespace tree
}  // namespace splitkv
