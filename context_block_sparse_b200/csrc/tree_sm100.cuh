// Shared by the two tcgen05 kernels of tree attention: the line's segments, the loading warp and the
// barriers it works with.
#pragma once

#include "sm100.cuh"
#include "tree.h"

namespace splitkv {
namespace tree {

using namespace sm100;

constexpr int kKeys = 128;                    // keys of a tile (M of the first product)
constexpr uint32_t kHalf = kKeys * 128;       // bytes of 128 rows x 64 columns
constexpr uint32_t kBarBytes = 960;           // barrier block
constexpr int kMetaRing = 16;                 // page-error masks in flight (K tiles)

#ifdef __CUDACC__

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// kind::f16, float32 accumulator; A and B of one 16-bit type.
__host__ __device__ constexpr uint32_t idesc(bool f16, int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | (uint32_t(a_mn) << 15) |
         (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

template <typename T>
constexpr bool kIsF16 = false;
template <>
constexpr bool kIsF16<__half> = true;
// log2: how far a row's reference lies below its first maximum, and by how much more a later one may exceed it
template <typename T>
constexpr float kLift = float(lift_of(kIsF16<T>, true));
template <typename T>
constexpr float kHeadroom = float(headroom_of(kIsF16<T>));
template <typename T>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  if constexpr (kIsF16<T>) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  } else {
    return pack_bf16(lo, hi);
  }
}

// One lane of a converged warp.  The warp that issues the products runs them as a whole and lets this lane act: its
// operands then stay in uniform registers.  With one lane in a branch of its own each product takes some ten instructions
// more, and beside eight busy softmax warps a pair of row tiles' products took 4350 clocks instead of 2260 (2050 alone).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// Barriers over one softmax group (128 threads); vote returns whether any thread's predicate holds.
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(g + 1) : "memory"); }
__device__ __forceinline__ bool group_any(int g, bool pred) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(out)
      : "r"(g + 1), "r"(pred ? 1u : 0u)
      : "memory");
  return out != 0;
}
// The same over both groups of tree_rows_sm100.cu.
__device__ __forceinline__ void both_sync() { asm volatile("bar.sync 3, 256;" ::: "memory"); }
__device__ __forceinline__ bool both_any(bool pred) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 3, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(out)
      : "r"(pred ? 1u : 0u)
      : "memory");
  return out != 0;
}
// The parameters of both kernels: tensor maps of the cache's and the nodes' keys and values.
#define SPLITKV_TREE_MAPS                                                                                  \
  const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,                      \
      const __grid_constant__ CUtensorMap tm_kb, const __grid_constant__ CUtensorMap tm_vb

// A unit's tiles in this CTA's stretch, as the loading warp hands it to the others.
struct Segment {
  int n0, n, rows, len;    // first node, nodes; rows of the row tile (past NR: a full one); context length
  int tile0, tiles, ctx;   // key tiles (tiles == 0: the end); tiles from number ctx on are the tree's
  int rt, head;
  int rec;                 // this part's record; -1: the unit is all here
};
constexpr int kSegRing = 4;

struct CommonBars {
  uint64_t full[8], empty[8];       // the ring of tiles
  uint64_t q_full;
  uint64_t seg_full[kSegRing], seg_empty[kSegRing];   // one arrival of the loading warp; of every reader
  Segment seg[kSegRing];
  long long scan[20];
  long long rel, line, stop;          // first place within sequence seq, places of the line, the stretch's end
  int seq, ctas;
  uint32_t tmem_base;
  int abort_flag;
  int bad[kMetaRing];
  uint32_t flag[2][kMaxNodes / 32];   // by segment parity: nodes whose V is not all finite
};

// The segments of a CTA's stretch of the line, in order.
struct Walk {
  long long left;   // places not yet handed out
  int rest;         // places of the unit handed out last in later stretches
  int b, unit, at;  // the next place: `at` of unit `unit` of sequence b
  SeqWork w;
  bool bad;
  __device__ void begin(const TreeParams& p, const CommonBars* c, long long n) {
    left = n;
    b = n > 0 ? c->seq : 0;
    bad = false;
    if (n <= 0) return;
    w = seq_work(p, b, bad);
    unit = int(c->rel / (p.lead + w.nt));
    at = int(c->rel % (p.lead + w.nt));
  }
  __device__ bool next(const TreeParams& p, Segment& s) {
    while (left > 0) {
      while (unit >= p.Hkv / p.hg * w.rts || w.places == 0) {
        if (++b >= p.B) return false;
        w = seq_work(p, b, bad);
        unit = at = 0;
      }
      const int take = int(min((long long)(p.lead + w.nt - at), left));
      const int pair = unit / w.rts;
      s.head = pair * p.hg + blockIdx.x % p.hg;
      s.rt = unit % w.rts;
      s.tile0 = max(0, at - p.lead);
      s.tiles = max(0, at + take - p.lead) - s.tile0;
      rest = p.lead + w.nt - at - take;
      s.rec = s.tile0 > 0 ? 2 * int(blockIdx.x) : rest > 0 ? 2 * int(blockIdx.x) + 1 : -1;
      left -= take;
      ++unit;
      at = 0;
      if (s.tiles == 0) continue;      // (only the places before a unit's tiles)
      s.n0 = w.n0;
      s.n = w.n;
      s.ctx = w.ctx;
      s.rows = w.n * p.G - s.rt * p.Mt;
      s.len = w.len;
      return true;
    }
    return false;
  }
};

// The mask row of a node is wanted soon: its lines are asked for into L2.
__device__ __forceinline__ void want_mask(const TreeParams& p, int node, int n) {
  if (p.mask == nullptr) return;
  const uint8_t* m = p.mask + int64_t(node) * p.mask_row;
  for (int i = 0; i < n; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(m + i));
  asm volatile("prefetch.global.L2 [%0];" ::"l"(m + n - 1));
}

// Block-wide: this CTA's stretch of the line, and the sequence it begins in (bars->seq, rel, line, stop, ctas: valid
// after the next block barrier).  Returns its places.
template <int kThreads>
__device__ __forceinline__ long long find_stretch(const TreeParams& p, CommonBars* bars) {
  const int tid = threadIdx.x;
  if (tid == 0) p.split[blockIdx.x].w = -1;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  long long mine = 0, before;
  bool bad = false;
  for (int b = b0; b < b1; ++b) mine += seq_work(p, b, bad).places;
  if (bad && blockIdx.x == 0) atomicCAS(p.status, 0, SPLITKV_ERR_INVALID_ARG);
  const long long W = block_prefix<kThreads>(mine, before, bars->scan);
  const int ctas = int(min((long long)(p.ctas), W)), c = blockIdx.x / p.hg;
  if (c >= ctas) return 0;
  const long long x0 = stretch(W, c, ctas), x1 = stretch(W, c + 1, ctas);
  if (tid == 0) {
    bars->line = W;
    bars->stop = x1;
    bars->ctas = ctas;
  }
  if (x0 >= before && x0 < before + mine) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const long long t = seq_work(p, b, bad).places;
      if (x0 < at + t) {
        bars->seq = b;
        bars->rel = x0 - at;
        break;
      }
      at += t;
    }
  }
  return x1 - x0;
}

// The loading warp: hands out the segments, and brings their tiles into the ring in the order in which the products
// take them -- K0, K1, V0, K2, V1, ... (kAhead) or K0, V0, K1, V1, ....
template <int D, int kStages, bool kAhead>
__device__ __forceinline__ void load_tiles(CommonBars* bars, uint8_t* smem, const CUtensorMap& tm_k,
                                           const CUtensorMap& tm_v, const CUtensorMap& tm_kb, const CUtensorMap& tm_vb,
                                           const TreeParams& p, long long n_places, const WaitCtx& wctx) {
  constexpr int kFile = 9 * 10000;
  constexpr uint32_t kTile = uint32_t(D / 64) * kHalf;
  const int lane = threadIdx.x & 31;
  const int page = 1 << p.page_shift, box = min(page, kKeys);      // keys of a page, of a TMA box
  uint32_t c = 0, kc = 0, seg = 0;
  bool ok = true;
  Walk walk;
  walk.begin(p, bars, n_places);
  const int boxes = kKeys / box;
  // lane l's page of a tile
  auto page_of = [&](const Segment& s, int j) -> int {
    const int key = (s.tile0 + j) * kKeys + lane * box;
    if (s.tile0 + j >= s.ctx) return lane == 0 ? -3 : -2;   // a tile of the tree: one box
    if (lane >= boxes || key >= s.len) return -2;           // no box
    const int pg = p.table[walk.b * p.table_row + (key >> p.page_shift)];
    return pg < 0 || pg >= p.num_pages ? -1 : pg;           // -1: a page that does not exist
  };
  auto load = [&](const CUtensorMap* map, const CUtensorMap* tree, const Segment& s, int j, int pg) -> bool {
    const int slot = int(c % kStages);
    if (!warp_wait(&bars->empty[slot], ((c / kStages) & 1) ^ 1, wctx, kFile + __LINE__)) return false;
    const bool nodes = s.tile0 + j >= s.ctx;
    const int n = __popc(__ballot_sync(0xffffffffu, pg != -2));
    if (lane == 0) mbar_expect_tx(&bars->full[slot], nodes ? kTile : uint32_t(n) * box * 128 * (D / 64));
    __syncwarp();
    if (pg == -3) {
      // 128 rows of the nodes' array: rows of other sequences are masked, rows behind the array read as zeros
      for (int h = 0; h < D / 64; ++h)
        tma_load_4d(smem + slot * kTile + h * kHalf, tree, &bars->full[slot], h * 64, s.head,
                    s.n0 + (s.tile0 + j - s.ctx) * kKeys, 0);
    } else if (pg != -2) {
      // a page outside the cache reads as zeros: a page coordinate past the last one
      const int pc = pg < 0 ? p.num_pages : pg;
      const int at = ((s.tile0 + j) * kKeys + lane * box) & (page - 1);
      for (int h = 0; h < D / 64; ++h)
        tma_load_4d(smem + slot * kTile + h * kHalf + lane * box * 128, map, &bars->full[slot], h * 64, s.head, at,
                    pc);
    }
    ++c;
    return true;
  };
  auto note = [&](int pg) {     // pages of a K tile that do not exist, for the softmax
    const bool wrong = pg == -1;
    const uint32_t m = __ballot_sync(0xffffffffu, wrong);
    if (lane == 0) {
      bars->bad[kc % kMetaRing] = int(m);
      if (m) atomicCAS(p.status, 0, SPLITKV_ERR_INVALID_ARG);
    }
    ++kc;
  };
  for (;;) {
    Segment sg;
    const bool more = walk.next(p, sg);
    const int ring = int(seg % kSegRing);
    if (!warp_wait(&bars->seg_empty[ring], ((seg / kSegRing) & 1) ^ 1, wctx, kFile + __LINE__)) { ok = false; break; }
    if (!more) sg.tiles = 0;
    if (lane == 0) bars->seg[ring] = sg;
    warp_arrive(&bars->seg_full[ring]);
    ++seg;
    if (!more) break;
    if (lane == 0 && sg.tile0 == 0 && walk.rest > 0) {      // the merge finds the unit here
      p.split[blockIdx.x] = make_int4(sg.n0, sg.n, sg.head | sg.rt << 16,
                                      cta_before(bars->line, bars->stop + walk.rest, bars->ctas));
    }
    int now = page_of(sg, 0), nxt = sg.tiles > 1 ? page_of(sg, 1) : -2;
    note(now);
    if (!load(&tm_k, &tm_kb, sg, 0, now)) { ok = false; break; }
    for (int j = 0; j < sg.tiles; ++j) {
      const int ahead = j + 2 < sg.tiles ? page_of(sg, j + 2) : -2;
      if (!kAhead && !load(&tm_v, &tm_vb, sg, j, now)) { ok = false; break; }
      if (j + 1 < sg.tiles) {
        note(nxt);
        if (!load(&tm_k, &tm_kb, sg, j + 1, nxt)) { ok = false; break; }
      }
      if (kAhead && !load(&tm_v, &tm_vb, sg, j, now)) { ok = false; break; }
      now = nxt;
      nxt = ahead;
    }
    if (!ok) break;
  }
  if (!ok) bars->abort_flag = 1;
  // copies in flight land before the CTA may exit
  if (lane == 0)
    for (uint32_t i = c >= uint32_t(kStages) ? c - kStages : 0; i < c; ++i)
      mbar_drain(&bars->full[i % kStages], (i / kStages) & 1, wctx, kFile + __LINE__);
  __syncwarp();
}

#endif  // __CUDACC__

cudaError_t launch_tree_rows_sm100(const TreeParams& p, int dtype, const CUtensorMap* m, cudaStream_t s);

}  // namespace tree
}  // namespace splitkv
