// Draft-tree attention on tcgen05 with rows as N, for row tiles of 32 and 64 rows, and 128 at d = 128: every row of a unit
// (sequence, KV head, row tile) against the sequence's cached keys and the tree's.
//
// A row tile's keys stream past it once, so the kernel wants HBM speed: a 128-key tile of K and V
// (64 KB at d = 128) reaches an SM every ~2700 clocks.  A tcgen05.mma needs M = 128 (or 64) rows in
// its A operand, and most draft trees have 4 to 128 rows a KV head; so both products are transposed, with
// keys and the head dimension as M and the rows as N:
//   S^T [128 keys x N rows] = K Q^T,     O^T [d x N rows] += V^T P^T,
// 16 instructions a tile at d = 128, of 40 / 48 / 64 clocks at N = 32 / 64 / 128 (measured).
//
// In S^T a TMEM lane is a key, so a softmax thread holds one key's scores of 32 rows.
// Its row maxima would need 128 lanes' agreement at every tile; instead a row keeps a reference, the
// maximum of its first tile (less kLift), and P = exp2(s - reference) may grow by 2^kHeadroom before the
// reference moves (O^T and the sums are then rescaled): a tile costs one barrier vote instead of a
// reduction.  Row sums stay in registers, one lane's share of 32 rows, and are reduced when the unit
// ends.  A thread's 32 probabilities are half a 128-byte row of P^T in the swizzled layout that the
// second product reads as its MN-major B operand.
//
// The first warps are softmax groups of four, 32 rows each, which also load Q and write the
// records or, of whole units, the finished rows.  Behind them one warp loads pages by TMA (one box a page and 64 columns) into a ring of
// tiles in the order in which the products take them: K0, K1, V0, K2, V1, ...; the last issues the
// products, S(j + 1) before PV(j), so that scores are formed while the softmax of the tile before
// runs.
// Keys behind the context's end or on a bad page are masked as lanes; their V rows are zeroed in
// shared memory before the product (P = 0 does not hide a NaN).
//
// Measured (8 KV heads): d = 128, 32 sequences over 8k keys, 32 rows 172 us and 64 rows 186 (165 at the copy rate), 128
// rows 223 (255 in a loop, where the GPU runs at its power limit); 16 ragged trees of 64 rows over 1k-8k 62 (47); d = 64,
// 64 sequences over 4k, 32 rows 99 (83).  A long unit runs at HBM's rate up to 64 rows; what is lost is a tile's chain of
// product, softmax and product at 128 rows, and at every unit's ends its first references, its row sums and stores,
// 3000 to 5000 clocks.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tree_sm100.cuh"

namespace splitkv {
namespace tree {
namespace {

constexpr int kFile = 8 * 10000;              // site number of this file's waits

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

template <int D, int NR>
struct Dims {
  // Rows (TMEM columns) of a softmax group.  With one or two groups a thread keeps its scores in registers from the
  // check to the exponentials; with four it has 96 registers, and scores are read twice, 16 at a time.
  static constexpr int kCols = 32;
  static constexpr int kGroups = NR / kCols;
  static constexpr int kThreads = 128 * kGroups + 64;
  // Two CTAs to an SM at d = 64 and few rows (a tile is half as long there as one CTA's chain of products, softmax and
  // barriers), else one with P^T double-buffered where it fits.
  static constexpr int kPerSm = D == 64 && NR <= 64 ? 2 : 1;
  static constexpr int kPBufs = kPerSm == 1 ? 2 : 1;
  static constexpr uint32_t kTile = uint32_t(D / 64) * kHalf;
  static constexpr uint32_t kQ = uint32_t(D / 64) * NR * 128;
  static constexpr uint32_t kP = uint32_t((NR + 63) / 64) * kHalf;
  // barriers, shifts, factors, and the warps' maxima and row sums
  static constexpr uint32_t kMeta = kBarBytes + NR * 8 + NR * 16;
  static constexpr int kFit = int(((kPerSm == 2 ? 115712 : 232448) - kMeta - kQ - kPBufs * kP) / kTile);
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static_assert(kStages >= 3, "ring");
  // the ring comes first: at d = 64 the second half of the V^T operand's M is whatever follows the tile
  static constexpr uint32_t kOffQ = kStages * kTile;
  static constexpr uint32_t kOffP = kOffQ + kQ;
  static constexpr uint32_t kOffMeta = kOffP + kPBufs * kP;
  static constexpr uint32_t kSmem = kOffMeta + kMeta;
  static constexpr uint32_t kTmem = NR * 2;
};

struct Bars : CommonBars {
  uint64_t s_full, s_free, p_ready[2], p_free[2], mma_done;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block");

template <typename T, int D, int NR>
__global__ void __launch_bounds__(Dims<D, NR>::kThreads, Dims<D, NR>::kPerSm)
    tree_context_sm100_kernel(SPLITKV_TREE_MAPS, const TreeParams p) {
  using Dm = Dims<D, NR>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bars = reinterpret_cast<Bars*>(smem + Dm::kOffMeta);
  // a row's shift: minus its reference (log2 units); -0.0: it has none yet (a reference of 0 is stored as +0.0)
  float* s_nref = reinterpret_cast<float*>(smem + Dm::kOffMeta + kBarBytes);
  float* s_f = s_nref + NR;   // factor of a moved reference
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const WaitCtx wctx{&bars->abort_flag, p.status, kWaitLimitNs};
  constexpr int kSoftWarps = 4 * Dm::kGroups;

  if (tid == 0) {
    for (int s = 0; s < Dm::kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->q_full, kSoftWarps);
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->s_free, kSoftWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->p_ready[i], kSoftWarps);   // by tile parity: a group may be a tile ahead of another
      mbar_init(&bars->p_free[i], 1);
    }
    mbar_init(&bars->mma_done, 1);
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(&bars->seg_full[i], 1);
      mbar_init(&bars->seg_empty[i], kSoftWarps + 1);
    }
    bars->abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == kSoftWarps + 1) {
    tmem_alloc(&bars->tmem_base, Dm::kTmem);
    tmem_relinquish();
  }
  if (warp == kSoftWarps && lane == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    prefetch_tmap(&tm_kb);
    prefetch_tmap(&tm_vb);
  }
  const long long n_places = find_stretch<Dm::kThreads>(p, bars);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = bars->tmem_base;
  const int box = min(1 << p.page_shift, kKeys);      // keys of a page in a tile

  if (warp == kSoftWarps) {
    // ------------------------------------------------------------ TMA producer
    load_tiles<D, Dm::kStages, true>(bars, smem, tm_k, tm_v, tm_kb, tm_vb, p, n_places, wctx);
  } else if (warp == kSoftWarps + 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool one = elect_one();
    constexpr uint32_t kIdS = idesc(kIsF16<T>, kKeys, NR, 0, 0), kIdO = idesc(kIsF16<T>, 128, NR, 1, 1);
    // Operand descriptors of the first tile; a tile's or a step's offset is added to the address field (16-byte
    // units, no carry out of it).  Building them at each instruction instead made this thread's integer code the
    // limit: ~200 clocks an instruction, where N = 32 / 64 / 128 take 40 / 48 / 64.
    const uint64_t dK = smem_desc_sw128(smem_u32(smem), 16, 1024), dV = smem_desc_sw128(smem_u32(smem), kHalf, 1024);
    const uint64_t dQ = smem_desc_sw128(smem_u32(smem + Dm::kOffQ), 16, 1024);
    const uint64_t dP = smem_desc_sw128(smem_u32(smem + Dm::kOffP), kHalf, 1024);
    uint32_t c = 0, t = 0, seg = 0;     // ring slots, tiles, segments so far
    bool ok = true;
    // scores of the next tile: S^T = K Q^T once its K has landed and the scores before are read
    auto issue_s = [&](uint32_t tile) -> bool {
      const int slot = int(c % Dm::kStages);
      if (tile > 0 && !warp_wait(&bars->s_free, (tile - 1) & 1, wctx, kFile + __LINE__)) return false;
      if (!warp_wait(&bars->full[slot], (c / Dm::kStages) & 1, wctx, kFile + __LINE__)) return false;
      tc_fence_after();
      const uint64_t a = dK + (uint32_t(slot) * Dm::kTile >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        if (one)
          mma_ss(tmem, a + (((kk >> 2) * kHalf + (kk & 3) * 32) >> 4),
                 dQ + (((kk >> 2) * (NR * 128) + (kk & 3) * 32) >> 4), kIdS, kk > 0 ? 1u : 0u);
      if (one) {
        mma_commit(&bars->empty[slot]);
        mma_commit(&bars->s_full);
      }
      ++c;
      return true;
    };
    while (ok) {
      const int at = int(seg % kSegRing);
      if (!warp_wait(&bars->seg_full[at], (seg / kSegRing) & 1, wctx, kFile + __LINE__)) { ok = false; break; }
      const int tiles = __shfl_sync(0xffffffffu, bars->seg[at].tiles, 0);
      if (tiles == 0) break;
      warp_arrive(&bars->seg_empty[at]);
      if (!warp_wait(&bars->q_full, seg & 1, wctx, kFile + __LINE__)) { ok = false; break; }
      ++seg;
      if (!issue_s(t)) { ok = false; break; }
      for (int j = 0; j < tiles; ++j, ++t) {
        if (j + 1 < tiles && !issue_s(t + 1)) { ok = false; break; }
        const int slot = int(c % Dm::kStages);
        if (!warp_wait(&bars->p_ready[t & 1], (t >> 1) & 1, wctx, kFile + __LINE__)) { ok = false; break; }
        if (!warp_wait(&bars->full[slot], (c / Dm::kStages) & 1, wctx, kFile + __LINE__)) { ok = false; break; }
        tc_fence_after();
        const uint64_t a = dV + (uint32_t(slot) * Dm::kTile >> 4);
        const uint64_t b = dP + (Dm::kPBufs == 2 ? (t & 1) * (Dm::kP >> 4) : 0u);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          if (one)
            mma_ss(tmem + NR, a + (kk * 2048 >> 4), b + (kk * 2048 >> 4), kIdO, kk > 0 ? 1u : (j > 0 ? 1u : 0u));
        if (one) {
          mma_commit(&bars->empty[slot]);
          mma_commit(&bars->p_free[t & 1]);
        }
        ++c;
      }
    }
    if (!ok) bars->abort_flag = 1;
    if (one) {
      mma_commit(&bars->mma_done);   // every product ends before tensor memory is released
      mbar_drain(&bars->mma_done, 0, wctx, kFile + __LINE__);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax groups
    const int g = warp >> 2, wq = warp & 3;
    const int key_lane = wq * 32 + lane;               // key of a tile = TMEM lane; head element in O^T
    const int col0 = g * Dm::kCols;                    // this group's rows
    constexpr bool kKeep = NR <= 64 && (NR == 32 || Dm::kPerSm == 1);   // scores stay in registers between the check and the exponentials
    constexpr int kW = kKeep ? Dm::kCols : 16;         // rows of one pass of exponentials
    const uint32_t tS = tmem + (uint32_t(wq * 32) << 16) + col0, tO = tS + NR;
    // this thread's key row of P^T: 128 bytes of 64 rows, 16-byte chunks swizzled
    uint8_t* my_p = smem + Dm::kOffP + (col0 >> 6) * kHalf + key_lane * 128;
    const int pch0 = (col0 & 63) >> 3;
    float* nref = s_nref + col0;
    float* fac = s_f + col0;
    float* s_x = s_f + NR + g * (4 * Dm::kCols);   // the warps' maxima, then their row sums
    const float scale = p.scale_log2;
    uint32_t t = 0, ring0 = 0;      // tiles and ring slots of the segments before
    bool ok = true;

    // Rows col0.. of a row tile's queries into the K-major operand layout, rows past the tile's end zero: requested
    // (after the last scores that read the buffer) and, a tile later, handed to the products.
    auto request_q = [&](const Segment& s) {
      constexpr int kCh = D / 8;
      const int n_rows = s.rows, n0 = s.n0, first = s.rt * NR, h0 = s.head * p.G;
#pragma unroll 1
      for (int i = tid & 127; i < Dm::kCols * kCh; i += 128) {
        const int r = col0 + i / kCh, ch = i % kCh;
        const int row = r < n_rows ? first + r : first, node = row / p.G, h = h0 + row - node * p.G;
        cp_async16(smem + Dm::kOffQ + (ch >> 3) * (NR * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4),
                   p.q + int64_t(n0 + node) * p.q_node + int64_t(h) * p.q_head + ch * 16, r < n_rows);
      }
      cp_async_commit();
    };
    auto deliver_q = [&]() {
      cp_async_wait<0>();
      fence_async_smem();
      warp_arrive(&bars->q_full);
    };
    // A tile with keys that are not there or that not every row sees: their scores in tensor memory become what the
    // scale turns into -inf, so that nothing after this knows of masks.
    const float hidden = scale > 0.f ? -INFINITY : INFINITY;
    auto hide = [&](const Segment& s, bool tree, int key0, int limit, uint32_t wrong) {
      uint32_t bits = key_lane < limit && !((wrong >> (key_lane / box)) & 1u) ? 0xffffffffu : 0u;   // bit c: row col0 + c
      if (tree && bits != 0 && p.mask != nullptr) {
        bits = 0;
        const int first = s.rt * NR + col0, last = min(first + Dm::kCols, s.rt * NR + s.rows);
        const uint8_t* m = p.mask + int64_t(s.n0) * p.mask_row + key0 + key_lane;
#pragma unroll 1
        for (int i0 = first / p.G; i0 * p.G < last; i0 += 8) {
          uint8_t y[8];      // (eight nodes' bytes asked for at once)
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = (i0 + k) * p.G < last ? m[(i0 + k) * p.mask_row] : uint8_t(0);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int i = i0 + k, lo = max(i * p.G - first, 0), n = min((i + 1) * p.G - first, 32) - lo;
            const uint32_t some = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1;
            if (y[k]) bits |= some << (lo & 31);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < Dm::kCols; e += 16) {
        uint32_t v[16];
        tmem_ld16(tS + e, v);
        tmem_wait_ld();
        reg_fence<16>(v);
        const uint32_t see = bits >> e;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = see >> i & 1u ? v[i] : __float_as_uint(hidden);
        tmem_st16(tS + e, v);
      }
      tmem_wait_st();
    };
    // After a wait gave up (ok is false, the kernel winds down) a warp goes on without waiting to the end of its segment,
    // where the group leaves together: its barriers always meet.  What is written until then lies inside its records.
    auto open = [&](uint32_t i) -> bool {
      ok = ok && warp_wait(&bars->seg_full[i % kSegRing], (i / kSegRing) & 1, wctx, kFile + __LINE__);
      if (group_any(g, !ok)) return false;
      return bars->seg[i % kSegRing].tiles > 0;
    };
    // Tile i's second product is done.  (By tile parity: with one barrier for all tiles, this wait could meet it two
    // phases back and take that for done.  The product of tile i - 2 is known to be: tile i's P^T waited for it.)
    auto done = [&](uint32_t i) -> bool {
      return warp_wait(&bars->p_free[i & 1], (i >> 1) & 1, wctx, kFile + __LINE__);
    };
    uint32_t seg = 0;
    bool more = open(0);
    if (more) {
      request_q(bars->seg[0]);
      deliver_q();
    }
    while (more) {
      const Segment& s = bars->seg[seg % kSegRing];
      const int rows = min(NR, s.rows), len = s.len, tiles = s.tiles;
      const bool live = rows > col0;   // this group has rows
      float l[Dm::kCols];              // a thread's own share of its rows' sums
#pragma unroll
      for (int i = 0; i < Dm::kCols; ++i) l[i] = 0.f;
      if ((tid & 127) < Dm::kCols) nref[tid & 127] = -0.0f;
      bool need = live;           // a row has no reference yet
      group_sync(g);
      const int tile0 = s.tile0, ctx = s.ctx, nodes = s.n;
      if ((tid & 127) < Dm::kCols && col0 + (tid & 127) < rows && tile0 + tiles > ctx)
        want_mask(p, s.n0 + (s.rt * NR + col0 + (tid & 127)) / p.G, nodes);
      for (int j = 0; j < tiles; ++j, ++t) {
        const bool tree = tile0 + j >= ctx;
        const int key0 = (tile0 + j - (tree ? ctx : 0)) * kKeys, limit = (tree ? nodes : len) - key0;   // keys there are
        ok = ok && warp_wait(&bars->s_full, t & 1, wctx, kFile + __LINE__);
        tc_fence_after();
        if (j + 1 == tiles) {
          // the unit's last scores are formed: the next unit's queries may come
          more = open(seg + 1);
          if (more) request_q(bars->seg[(seg + 1) % kSegRing]);
        }
        const uint32_t wrong = uint32_t(bars->bad[t % kMetaRing]);
        const bool part = wrong != 0 || limit < kKeys || tree;
        if (part && live) hide(s, tree, key0, limit, wrong);
        // scores in log2 units, shifted by the rows' references; is one of them past the headroom?
        float x[kW];
        float mx = -INFINITY;
        if (live && !need) {
#pragma unroll
          for (int e = 0; e < Dm::kCols; e += 16) {
            uint32_t v[16];
            tmem_ld16(tS + e, v);
            tmem_wait_ld();
            reg_fence<16>(v);
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 r = *reinterpret_cast<const float4*>(nref + e + i);
              float y0, y1, y2, y3;
              ffma2(y0, y1, __uint_as_float(v[i]), __uint_as_float(v[i + 1]), scale, scale, r.x, r.y);
              ffma2(y2, y3, __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]), scale, scale, r.z, r.w);
              mx = fmax3(mx, y0, y1);
              mx = fmax3(mx, y2, y3);
              if constexpr (kKeep) {
                x[e + i] = y0;
                x[e + i + 1] = y1;
                x[e + i + 2] = y2;
                x[e + i + 3] = y3;
              }
            }
          }
        }
        bool over = need;
        if (!need && live) over = group_any(g, mx > kLift<T> + kHeadroom<T>);
        if (over) {
          need = false;
          // new references of the group's rows: lane i of every warp gets column i's maximum
          float m = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; e += 16) {
            uint32_t v[16];
            tmem_ld16(tS + e, v);
            tmem_wait_ld();
            reg_fence<16>(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float y = warp_max(__uint_as_float(v[i]) * scale);
              m = lane == e + i ? y : m;
            }
          }
          const uint32_t was = __float_as_uint(nref[lane]);
          const float old = was == 0x80000000u ? -INFINITY : -__uint_as_float(was);
          s_x[wq * Dm::kCols + lane] = m;
          group_sync(g);
#pragma unroll
          for (int w = 0; w < 4; ++w) m = fmaxf(m, s_x[w * Dm::kCols + lane]);
          // (the four warps hold the same values, so their votes agree)
          m -= kLift<T>;
          const float to = old == -INFINITY ? m : (m > old + kHeadroom<T> ? m : old);
          const float f = old == -INFINITY ? 1.f : fast_exp2(old - to);
          if (wq == 0) {
            nref[lane] = to == -INFINITY ? -0.0f : 0.f - to;
            fac[lane] = f;
          }
          const bool moved = __any_sync(0xffffffffu, f != 1.f);
          need = __any_sync(0xffffffffu, to == -INFINITY) != 0;
          group_sync(g);
          if (moved) {
#pragma unroll
            for (int i = 0; i < Dm::kCols; ++i) l[i] *= fac[i];
            if (j > 0) {
              ok = ok && done(t - 1);
              tc_fence_after();
#pragma unroll 1
              for (int e = 0; e < 32; e += 16) {
                uint32_t o[16];
                tmem_ld16(tO + e, o);
                tmem_wait_ld();
                reg_fence<16>(o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fac[e + i]);
                tmem_st16(tO + e, o);
              }
              tmem_wait_st();
            }
          }
          if constexpr (kKeep) {
#pragma unroll
            for (int e = 0; e < Dm::kCols; e += 16) {
              uint32_t v[16];
              tmem_ld16(tS + e, v);
              tmem_wait_ld();
              reg_fence<16>(v);
#pragma unroll
              for (int i = 0; i < 16; ++i) x[e + i] = fmaf(__uint_as_float(v[i]), scale, nref[e + i]);
            }
          }
        }
        if (kKeep || !live) {
          tc_fence_before();
          warp_arrive(&bars->s_free);
        }
        // this P^T buffer may be rewritten once the product that read it is done
        constexpr uint32_t kB = Dm::kPBufs;
        if (t >= kB)
          ok = ok && done(t - kB);
        uint8_t* pp = my_p + (kB == 2 ? (t & 1) * Dm::kP : 0);
        if (live) {
#pragma unroll
          for (int w = 0; w < Dm::kCols / kW; ++w) {
            if constexpr (!kKeep) {
              uint32_t v[16];
              tmem_ld16(tS + w * kW, v);
              tmem_wait_ld();
              reg_fence<16>(v);
              if ((w + 1) * kW == Dm::kCols) {
                tc_fence_before();
                warp_arrive(&bars->s_free);
              }
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 r = *reinterpret_cast<const float4*>(nref + w * kW + i);
                ffma2(x[i], x[i + 1], __uint_as_float(v[i]), __uint_as_float(v[i + 1]), scale, scale, r.x, r.y);
                ffma2(x[i + 2], x[i + 3], __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]), scale, scale, r.z, r.w);
              }
            }
#pragma unroll
            for (int i = 0; i < kW; ++i) x[i] = fast_exp2(x[i]);
#pragma unroll
            for (int i = 0; i < kW; i += 2)
              fadd2(l[w * kW + i], l[w * kW + i + 1], l[w * kW + i], l[w * kW + i + 1], x[i], x[i + 1]);
#pragma unroll
            for (int i = 0; i < kW / 8; ++i)
              *reinterpret_cast<uint4*>(pp + (((pch0 + w * (kW / 8) + i) ^ (key_lane & 7)) << 4)) =
                  make_uint4(pack<T>(x[8 * i], x[8 * i + 1]), pack<T>(x[8 * i + 2], x[8 * i + 3]),
                             pack<T>(x[8 * i + 4], x[8 * i + 5]), pack<T>(x[8 * i + 6], x[8 * i + 7]));
          }
        }
        if (g == 0 && part) {
          // V rows of keys that are not there become zeros: P = 0 does not hide a NaN.  Nor does it in a tree's V, which
          // may hold infinities or NaN that only the rows that see them may meet: they are taken out here, and added
          // back in the epilogue to the rows that see them.
          const uint32_t i = ring0 + (j + 1 < tiles ? 2 * j + 2 : 2 * j + 1);
          ok = ok && warp_wait(&bars->full[i % Dm::kStages], (i / Dm::kStages) & 1, wctx, kFile + __LINE__);
          uint32_t* flag = bars->flag[seg & 1];
          if (tree) {
            if (tile0 + j == max(ctx, tile0) && tid < kMaxNodes / 32) flag[tid] = 0;
            group_sync(0);
          }
          uint8_t* v = smem + (i % Dm::kStages) * Dm::kTile;
          if (ok && key_lane >= limit) {
#pragma unroll
            for (int e = 0; e < D / 8; ++e)
              *reinterpret_cast<uint4*>(v + (e >> 3) * kHalf + key_lane * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          if (ok && tree) {
            const int n16 = min(limit, kKeys) * (D / 8);     // 16-byte pieces of the nodes' rows
#pragma unroll 2
            for (int e = tid; e < n16; e += 128) {
              const int key = e / (D / 8), ch = e % (D / 8);
              uint4* at = reinterpret_cast<uint4*>(v + (ch >> 3) * kHalf + key * 128 + (ch & 7) * 16);
              uint4 x = *at;
              if (take_out<T>(x)) {
                *at = x;
                atomicOr(&flag[(key0 + key) >> 5], 1u << (key & 31));
              }
            }
          }
        }
        fence_async_smem();
        tc_fence_before();
        warp_arrive(&bars->p_ready[t & 1]);
      }
      ring0 += 2 * tiles;
      if (more) deliver_q();   // the next unit's first scores overlap this epilogue
      const int rec = s.rec;
      // where this thread's first row goes: the unit's rows are node-major, the G heads of a node next to each other
      const int row0 = s.rt * NR + col0, node0 = row0 / p.G, g0 = row0 - node0 * p.G;
      const size_t hr0 = size_t(s.n0 + node0) * p.Hq + s.head * p.G + g0;
      // row sums: over the warp's lanes (each step leaves half the rows to a lane, at the end one), then over the four warps
      if (live) {
        int r = 0;       // this lane's row after the steps
#pragma unroll
        for (int st = 16; st > 0; st >>= 1) {
          const bool up = (lane & st) != 0;
#pragma unroll
          for (int i = 0; i < st; ++i) {
            const float send = up ? l[i] : l[i + st];
            const float keep = up ? l[i + st] : l[i];
            l[i] = keep + __shfl_xor_sync(0xffffffffu, send, st);
          }
          r += up ? st : 0;
        }
        s_x[wq * Dm::kCols + r] = l[0];
        group_sync(g);
        const int row = tid & 127;
        if (row < Dm::kCols) {
          const float nr = nref[row], m = __float_as_uint(nr) == 0x80000000u ? -INFINITY : -nr;
          const float sum = s_x[row] + s_x[Dm::kCols + row] + s_x[2 * Dm::kCols + row] + s_x[3 * Dm::kCols + row];
          // what the row's O is multiplied by, and where it goes (elements from the first row's)
          const uint32_t at = rec >= 0 ? row : row + (g0 + row) / p.G * (p.Hq - p.G);
          fac[row] = rec >= 0 ? 1.f : row_inv(sum);
          reinterpret_cast<uint32_t*>(s_x)[row] = at * D;
          if (col0 + row < rows) {
            if (rec >= 0)
              p.rec_ml[size_t(rec) * NR + col0 + row] = make_float2(m, sum);
            else
              p.lse[hr0 + at] = row_lse(m, sum, int(kLift<T>));
          }
        }
        group_sync(g);
      }
      ok = ok && done(t - 1);
      tc_fence_after();
      uint32_t odd_v = 0;      // a node whose V is not all finite
      if (tile0 + tiles > ctx)
        for (int i = 0; i < kMaxNodes / 32; ++i) odd_v |= bars->flag[seg & 1][i];
      if (live) {
        uint32_t o[32];
        tmem_ld32(tO, o);
        tmem_wait_ld();
        reg_fence<32>(o);
        if (D == 128 || wq < D / 32) {
          if (odd_v) {
#pragma unroll 1
            for (int j = max(0, tile0 - ctx) * kKeys; j < min(nodes, (tile0 + tiles - ctx) * kKeys); ++j) {
              if (!((bars->flag[seg & 1][j >> 5] >> (j & 31)) & 1u)) continue;
              const float y = float(*reinterpret_cast<const T*>(p.vb + int64_t(s.n0 + j) * p.vb_node +
                                                                s.head * p.vb_head + key_lane * 2));
              if (isfinite(y)) continue;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int node = (s.rt * NR + col0 + i) / p.G;
                if (node < nodes && (p.mask == nullptr || p.mask[int64_t(s.n0 + node) * p.mask_row + j]))
                  o[i] = __float_as_uint(__uint_as_float(o[i]) + y);
              }
            }
          }
          // eight rows at a time, none behind the last: this is one warp's serial code at the end of every unit
          const uint32_t* off = reinterpret_cast<const uint32_t*>(s_x);
          float* f32 = rec >= 0 ? p.rec_o + (size_t(rec) * NR + col0) * D : reinterpret_cast<float*>(p.o) + hr0 * D;
          T* low = reinterpret_cast<T*>(p.o) + hr0 * D;
          const bool wide = rec >= 0 || p.o_f32;
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            if (col0 + e < rows) {
#pragma unroll
              for (int i = e; i < e + 8; ++i) {
                const float y = __uint_as_float(o[i]) * fac[i];
                if (col0 + i < rows) {
                  if (wide)
                    f32[off[i] + key_lane] = y;
                  else
                    low[off[i] + key_lane] = T(y);
                }
              }
            }
          }
        }
      }
      tc_fence_before();
      warp_arrive(&bars->seg_empty[seg % kSegRing]);
      ++seg;
    }
    if (!ok) bars->abort_flag = 1;
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kSoftWarps + 1) tmem_dealloc(tmem, Dm::kTmem);
}

template <typename T, int D, int NR>
cudaError_t launch(const TreeParams& p, const CUtensorMap* m, cudaStream_t s) {
  using Dm = Dims<D, NR>;
  cudaError_t e = cudaFuncSetAttribute(tree_context_sm100_kernel<T, D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       int(Dm::kSmem));
  if (e != cudaSuccess) return e;
  tree_context_sm100_kernel<T, D, NR><<<p.ctas * p.hg, Dm::kThreads, Dm::kSmem, s>>>(m[0], m[1], m[2], m[3], p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t rows(const TreeParams& p, const CUtensorMap* m, cudaStream_t s) {
  switch (p.Mt) {
    case 32: return launch<T, D, 32>(p, m, s);
    case 64: return launch<T, D, 64>(p, m, s);
    default: return launch<T, 128, 128>(p, m, s);      // (at d = 64 these are rows as M)
  }
}

}  // namespace

cudaError_t launch_tree_context_sm100(const TreeParams& p, int dtype, cudaStream_t s) {
  const bool f16 = dtype == SPLITKV_DTYPE_F16;
  const int page = 1 << p.page_shift;
  const uint32_t box = page < kKeys ? page : kKeys;
  CUtensorMap m[4];
  if (!make_page_map_4d(&m[0], p.kc, f16, p.d, p.Hkv, page, p.num_pages, p.kc_head, p.kc_slot, p.kc_page, box) ||
      !make_page_map_4d(&m[1], p.vc, f16, p.d, p.Hkv, page, p.num_pages, p.vc_head, p.vc_slot, p.vc_page, box) ||
      !make_page_map_4d(&m[2], p.kb, f16, p.d, p.Hkv, p.Nq, 1, p.kb_head, p.kb_node, 0, kKeys) ||
      !make_page_map_4d(&m[3], p.vb, f16, p.d, p.Hkv, p.Nq, 1, p.vb_head, p.vb_node, 0, kKeys))
    return cudaErrorInvalidValue;
  if (rows_as_m(p.Mt, p.d)) return launch_tree_rows_sm100(p, dtype, m, s);
  if (f16) return p.d == 128 ? rows<__half, 128>(p, m, s) : rows<__half, 64>(p, m, s);
  return p.d == 128 ? rows<__nv_bfloat16, 128>(p, m, s) : rows<__nv_bfloat16, 64>(p, m, s);
}

}  // namespace tree
}  // namespace splitkv
