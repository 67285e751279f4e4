// Draft-tree attention on tcgen05 with rows as M.  Row tiles of 256 rows: two tiles of 128 rows (A, B) share every
// 128-key tile of K and V,
//   S_x [128 rows x 128 keys] = Q_x K^T,     O_x [128 rows x d] += P_x V.
// Row tiles of 128 rows (kSplit): A and B are the even and the odd key tiles of the same rows, each with a running
// maximum, sum and O of its own, which are joined when the segment ends.
//
// At 256 rows the transposed products (tree_context_sm100.cu) are held up by shared memory and by
// agreeing on row statistics across lanes; here a TMEM lane is a row, so a softmax thread owns a row:
// its maximum, its sum, its reference, no barrier and no exchange, and P goes back over S in tensor
// memory as the second product's A operand instead of through shared memory.  A group's chain a tile (scores, softmax,
// product) is hidden behind the other group's, which is why a row tile of 128 rows is worked on by two as well: with one
// group 32 x 32 nodes over 8k took 291 us at d = 128, 215 so.  rows_as_m() says where this form is taken.
//
// A pair of row tiles costs the tensor core 2048 clocks a key tile at d = 128 (32 instructions of 64 clocks), the
// exponentials 2048 clocks of the MUFU units (128 x 256 at 16 a clock), HBM 2735 at 1965 MHz: while one group of four
// warps forms its tile's probabilities, the other tile's products run.  Long calls are bound by power: 4 x 64 nodes over
// 101k to 124k keys take 495 to 525 us, 55 to 58 % of the measured bf16 and HBM rates each, at 1 kW and 1590 MHz.  Scores in halves
// of 64 keys, whose products overlap the other half's softmax, saved 20 % of the clocks and took 525 us beside 505: the
// clock fell by more (N = 64 products read more of shared memory for the same work).
//
// As in the training kernels P = exp2(s - reference), where the reference is the row's first maximum (less kLift) and
// moves only when a later one exceeds it by kHeadroom (the row's O and sum are then rescaled).  Scores of
// keys that a row does not see are overwritten in tensor memory before anything else reads them; V rows
// that are not there are zeroed in shared memory, and what is not finite in a tree's V is taken out of it
// and added back, in the epilogue, to the rows that see it.
#include <cstdint>

#include "tree_sm100.cuh"

namespace splitkv {
namespace tree {
namespace {

constexpr int kFile = 7 * 10000;              // site number of this file's waits

template <int D, bool kSplit>
struct Dims {
  static constexpr int kThreads = 256 + 64;
  static constexpr int kTiles = kSplit ? 1 : 2;         // row tiles
  static constexpr uint32_t kTile = uint32_t(D / 64) * kHalf;       // 128 rows x D
  static constexpr uint32_t kMeta = kBarBytes + (kSplit ? 2048 : 0);
  static constexpr int kFit = int((232448 - kMeta - kTiles * kTile) / kTile);
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr uint32_t kOffQ = kStages * kTile;
  static constexpr uint32_t kOffMeta = kOffQ + kTiles * kTile;
  static constexpr uint32_t kSmem = kOffMeta + kMeta;
  // tensor memory: S_x in 128 columns each, then O_x in D columns each
  static constexpr uint32_t kTmem = 512;
};

struct Bars : CommonBars {
  uint64_t s_full[2], p_ready[2], o_full[2], mma_done;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block");

template <typename T, int D, bool kSplit>
__global__ void __launch_bounds__(Dims<D, kSplit>::kThreads, 1)
    tree_rows_sm100_kernel(SPLITKV_TREE_MAPS, const TreeParams p) {
  using Dm = Dims<D, kSplit>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bars = reinterpret_cast<Bars*>(smem + Dm::kOffMeta);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const WaitCtx wctx{&bars->abort_flag, p.status, kWaitLimitNs};
  constexpr int kSoftWarps = 8;

  if (tid == 0) {
    for (int s = 0; s < Dm::kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->q_full, kSplit ? 4 : 8);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->p_ready[x], 4);
      mbar_init(&bars->o_full[x], 1);
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
  constexpr uint32_t kO = 256;                         // first column of O_0

  if (warp == kSoftWarps) {
    // ------------------------------------------------------------ TMA producer
    load_tiles<D, Dm::kStages, kSplit>(bars, smem, tm_k, tm_v, tm_kb, tm_vb, p, n_places, wctx);
  } else if (warp == kSoftWarps + 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool one = elect_one();
    constexpr uint32_t kIdS = idesc(kIsF16<T>, 128, kKeys, 0, 0), kIdO = idesc(kIsF16<T>, 128, D, 0, 1);
    const uint64_t dK = smem_desc_sw128(smem_u32(smem), 16, 1024), dV = smem_desc_sw128(smem_u32(smem), kHalf, 1024);
    const uint64_t dQ = smem_desc_sw128(smem_u32(smem + Dm::kOffQ), 16, 1024);
    uint32_t c = 0, seg = 0;                 // ring slots, segments so far
    uint32_t np[2] = {0, 0};                 // tiles of each row tile so far
    bool ok = true;
    auto full = [&](uint32_t i) -> bool {
      return warp_wait(&bars->full[i % Dm::kStages], (i / Dm::kStages) & 1, wctx, kFile + __LINE__);
    };
    // S_x = Q_x K^T from slot i
    auto scores = [&](int x, uint32_t i) {
      const uint64_t a = dQ + (kSplit ? 0u : x * Dm::kTile >> 4), b = dK + ((i % Dm::kStages) * Dm::kTile >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t at = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
        if (one) mma_ss(tmem + x * 128, a + at, b + at, kIdS, kk > 0 ? 1u : 0u);
      }
      if (one) mma_commit(&bars->s_full[x]);
    };
    while (ok) {
      const int at = int(seg % kSegRing);
      if (!warp_wait(&bars->seg_full[at], (seg / kSegRing) & 1, wctx, kFile + __LINE__)) { ok = false; break; }
      const int tiles = __shfl_sync(0xffffffffu, bars->seg[at].tiles, 0);
      const int nx = __shfl_sync(0xffffffffu, bars->seg[at].rows, 0) > 128 ? 2 : 1;   // (row tiles; not with kSplit)
      if (tiles == 0) break;
      warp_arrive(&bars->seg_empty[at]);
      if (!warp_wait(&bars->q_full, seg & 1, wctx, kFile + __LINE__)) { ok = false; break; }
      ++seg;
      if (!full(c)) { ok = false; break; }
      tc_fence_after();
      if constexpr (kSplit) {
        // slots: K(0), K(1), V(0), K(2), V(1), ...
        for (int j = 0; j < min(tiles, 2); ++j) {
          if (j > 0 && !full(c)) { ok = false; break; }
          tc_fence_after();
          scores(j, c);
          if (one) mma_commit(&bars->empty[c % Dm::kStages]);
          ++c;
        }
        for (int j = 0; j < tiles && ok; ++j) {
          const int x = j & 1;
          if (!warp_wait(&bars->p_ready[x], np[x] & 1, wctx, kFile + __LINE__) || !full(c)) { ok = false; break; }
          ++np[x];
          tc_fence_after();
          const uint64_t b = dV + ((c % Dm::kStages) * Dm::kTile >> 4);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            if (one)
              mma_ts(tmem + kO + x * D, tmem + x * 128 + kk * 8, b + (kk * 2048 >> 4), kIdO,
                     kk > 0 ? 1u : (j > 1 ? 1u : 0u));
          if (one) mma_commit(&bars->empty[c % Dm::kStages]);
          ++c;
          if (j + 2 < tiles) {
            if (!full(c)) { ok = false; break; }
            tc_fence_after();
            scores(x, c);
            if (one) mma_commit(&bars->empty[c % Dm::kStages]);
            ++c;
          } else {
            if (one) mma_commit(&bars->o_full[x]);
          }
        }
      } else {
        for (int x = 0; x < nx; ++x) scores(x, c);
        if (one) mma_commit(&bars->empty[c % Dm::kStages]);
        // slots: K(j) at c + 2 j, V(j) at c + 2 j + 1
        for (int j = 0; j < tiles && ok; ++j) {
          const uint32_t v = c + 2 * j + 1, k = v + 1;
          const bool more = j + 1 < tiles;
          for (int x = 0; x < nx; ++x) {
            if (!warp_wait(&bars->p_ready[x], np[x] & 1, wctx, kFile + __LINE__)) { ok = false; break; }
            ++np[x];
            if (x == 0 && !full(v)) { ok = false; break; }
            tc_fence_after();
            const uint64_t b = dV + ((v % Dm::kStages) * Dm::kTile >> 4);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              if (one)
                mma_ts(tmem + kO + x * D, tmem + x * 128 + kk * 8, b + (kk * 2048 >> 4), kIdO,
                       kk > 0 ? 1u : (j > 0 ? 1u : 0u));
            if (one && x == nx - 1) mma_commit(&bars->empty[v % Dm::kStages]);
            if (more) {
              if (x == 0) {
                if (!full(k)) { ok = false; break; }
                tc_fence_after();
              }
              scores(x, k);
              if (one && x == nx - 1) mma_commit(&bars->empty[k % Dm::kStages]);
            } else {
              if (one) mma_commit(&bars->o_full[x]);
            }
          }
        }
        c += 2 * tiles;
      }
    }
    if (!ok) bars->abort_flag = 1;
    if (one) {
      mma_commit(&bars->mma_done);   // every product ends before tensor memory is released
      mbar_drain(&bars->mma_done, 0, wctx, kFile + __LINE__);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax: one group of four warps a row tile
    const int x = warp >> 2, wq = warp & 3;
    const int r = (kSplit ? 0 : x * 128) + wq * 32 + lane;           // row of the row tile(s); its TMEM lane, modulo 128
    const uint32_t tS = tmem + (uint32_t(wq * 32) << 16) + x * 128;
    const uint32_t tO = tmem + (uint32_t(wq * 32) << 16) + kO + x * D;
    const int box = min(1 << p.page_shift, kKeys);                   // keys of a page in a tile
    const float scale = p.scale_log2, hidden = scale > 0.f ? -INFINITY : INFINITY;
    uint8_t* sq = smem + Dm::kOffQ + (kSplit ? 0 : x * Dm::kTile);
    float2* s_ml = reinterpret_cast<float2*>(smem + Dm::kOffMeta + kBarBytes);   // (kSplit) the groups' references and sums
    uint32_t seg = 0, ring0 = 0;         // segments and ring slots so far
    uint32_t ns = 0, no = 0, na = 0;     // tiles and segments of this row tile, and segments of tile A, so far
    bool ok = true;

    // After a wait gave up (ok is false, the kernel winds down) a warp goes on without waiting to the end of its segment,
    // where the group leaves together: its barriers always meet.  What is written until then lies inside its records.
    auto open = [&](uint32_t i) -> bool {
      ok = ok && warp_wait(&bars->seg_full[i % kSegRing], (i / kSegRing) & 1, wctx, kFile + __LINE__);
      if (!kSplit && group_any(x, !ok)) return false;   // (kSplit: both groups leave together, at the segment's end)
      return (!kSplit || ok) && bars->seg[i % kSegRing].tiles > 0;
    };
    auto request_q = [&](const Segment& s) {
      constexpr int kCh = D / 8;
      const int x0 = kSplit ? 0 : x * 128, n_rows = min(s.rows, p.Mt) - x0, first = s.rt * p.Mt + x0, n0 = s.n0;
      const int h0 = s.head * p.G;
#pragma unroll 2
      for (int i = tid & 127; i < 128 * kCh; i += 128) {
        const int q = i / kCh, ch = i % kCh;
        const int row = q < n_rows ? first + q : s.rt * p.Mt, node = row / p.G, h = h0 + row - node * p.G;
        cp_async16(sq + (ch >> 3) * kHalf + q * 128 + (((ch & 7) ^ (q & 7)) << 4),
                   p.q + int64_t(n0 + node) * p.q_node + int64_t(h) * p.q_head + ch * 16, q < n_rows);
      }
      cp_async_commit();
    };
    auto deliver_q = [&]() {
      cp_async_wait<0>();
      fence_async_smem();
      warp_arrive(&bars->q_full);
    };
    // Keys that are not there or that not every row sees: their scores in tensor memory become what the scale turns
    // into -inf.  A row's 128 bits: the keys it sees.
    auto hide = [&](const Segment& s, bool tree, int key0, int limit, uint32_t wrong) {
      uint32_t bits[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = limit - 32 * q;
        bits[q] = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1;
      }
      if (wrong) {
        for (int b = 0; b < kKeys / box; ++b)
          if ((wrong >> b) & 1u)
            for (int i = b * box; i < (b + 1) * box; ++i) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (i >> 5 == q) bits[q] &= ~(1u << (i & 31));
            }
      }
      if (tree && p.mask != nullptr) {
        // the warp's nodes one after the other, their mask bytes side by side over the lanes
        const int row0 = s.rt * p.Mt + r - lane, mine = (row0 + lane) / p.G;
        const int last = min((row0 + 31) / p.G, s.n - 1);
        uint32_t see[4] = {0, 0, 0, 0};
#pragma unroll 1
        for (int node0 = row0 / p.G; node0 <= last; node0 += 8) {
          // (eight nodes' bytes asked for at once: the loop waits for memory, not for its instructions)
          const uint8_t* m = p.mask + int64_t(s.n0 + node0) * p.mask_row + key0 + lane;
          uint8_t y[8][4];
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              y[k][q] = node0 + k <= last && 32 * q + lane < limit ? m[k * p.mask_row + 32 * q] : uint8_t(0);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t w = __ballot_sync(0xffffffffu, y[k][q] != 0);
              if (node0 + k == mine) see[q] = w;
            }
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) bits[q] &= see[q];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t v[32];
        tmem_ld32(tS + q * 32, v);
        tmem_wait_ld();
        reg_fence<32>(v);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = bits[q] >> i & 1u ? v[i] : __float_as_uint(hidden);
        tmem_st16p(tS + q * 32, v);
        tmem_st16p(tS + q * 32 + 16, v + 16);
      }
      tmem_wait_st();
    };

    bool more = open(0);
    if (kSplit && both_any(!ok)) more = false;
    if (more && (!kSplit || x == 0)) {
      request_q(bars->seg[0]);
      deliver_q();
    }
    while (more) {
      const Segment& s = bars->seg[seg % kSegRing];
      const int tiles = s.tiles, tile0 = s.tile0, ctx = s.ctx, nodes = s.n, len = s.len;
      const int rows = min(s.rows, p.Mt);
      const bool rows_here = kSplit || rows > x * 128, mine = kSplit && ((tiles - 1) & 1) == x;
      const bool warp_live = rows > r - lane;       // (a warp without rows only keeps step)
      float ref = -INFINITY, l = 0.f;       // the row's reference (log2 units) and sum
      if (r < rows && tile0 + tiles > ctx) want_mask(p, s.n0 + (s.rt * p.Mt + r) / p.G, nodes);
      if (!rows_here) {
        // (a row tile without rows keeps step with tile A: its queries' arrival must not fall into the segment before)
        more = open(seg + 1);
        ok = ok && warp_wait(&bars->o_full[0], na & 1, wctx, kFile + __LINE__);
        if (more) {
          request_q(bars->seg[(seg + 1) % kSegRing]);
          deliver_q();
        }
      } else {
        for (int j = kSplit ? x : 0; j < tiles; j += kSplit ? 2 : 1, ++ns) {
          const bool tree = tile0 + j >= ctx;
          const int key0 = (tile0 + j - (tree ? ctx : 0)) * kKeys, limit = (tree ? nodes : len) - key0;   // keys there are
          ok = ok && warp_wait(&bars->s_full[x], ns & 1, wctx, kFile + __LINE__);
          tc_fence_after();
          if (j + 1 == tiles) {
            // this tile's last scores are formed: the next unit's queries may come
            more = open(seg + 1);
            if (more) request_q(bars->seg[(seg + 1) % kSegRing]);
          }
          const uint32_t wrong = uint32_t(bars->bad[(ring0 / 2 + j) % kMetaRing]);
          const bool part = wrong != 0 || limit < kKeys || tree;
          if (warp_live) {
            if (part) hide(s, tree, key0, limit, wrong);
            // the row's maximum in log2 units (a scale below zero turns the smallest score into it)
            uint32_t v[128];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32p(tS + q * 32, v + q * 32);
            tmem_wait_ld();
            reg_fence<128>(v);
            float m0 = hidden, m1 = hidden, m2 = hidden, m3 = hidden;
            if (scale > 0.f) {
#pragma unroll
              for (int i = 0; i < 128; i += 8) {
                m0 = fmax3(m0, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                m1 = fmax3(m1, __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                m2 = fmax3(m2, __uint_as_float(v[i + 4]), __uint_as_float(v[i + 5]));
                m3 = fmax3(m3, __uint_as_float(v[i + 6]), __uint_as_float(v[i + 7]));
              }
            } else {
#pragma unroll
              for (int i = 0; i < 128; ++i) m0 = fminf(m0, __uint_as_float(v[i]));
            }
            const float m = (scale > 0.f ? fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * scale : m0 * scale) - kLift<T>;
            float f = 1.f;
            if (ref == -INFINITY) {
              ref = m;                             // (its O and sum are still zero)
            } else if (m > ref + kHeadroom<T>) {
              f = fast_exp2(ref - m);
              ref = m;
            }
            if (__any_sync(0xffffffffu, f != 1.f)) {
              l *= f;
              if (j > (kSplit ? 1 : 0)) {
                // the row's O: its last product is done, the scores' barrier came behind it
#pragma unroll 1
                for (int e = 0; e < D; e += 16) {
                  uint32_t o[16];
                  tmem_ld16(tO + e, o);
                  tmem_wait_ld();
                  reg_fence<16>(o);
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tmem_st16(tO + e, o);
                }
                tmem_wait_st();
              }
            }
            // P over the scores: keys 2 i, 2 i + 1 in column i, 32 scores at a time (never ahead of what is still to be read)
            const float nref = ref == -INFINITY ? 0.f : -ref;
            float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t pk[16];
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                float a, b, c, d;
                ffma2(a, b, __uint_as_float(v[q * 32 + i]), __uint_as_float(v[q * 32 + i + 1]), scale, scale, nref, nref);
                ffma2(c, d, __uint_as_float(v[q * 32 + i + 2]), __uint_as_float(v[q * 32 + i + 3]), scale, scale, nref,
                      nref);
                a = fast_exp2(a);
                b = fast_exp2(b);
                c = fast_exp2(c);
                d = fast_exp2(d);
                fadd2(s0, s1, s0, s1, a, b);
                fadd2(s2, s3, s2, s3, c, d);
                pk[i / 2] = pack<T>(a, b);
                pk[i / 2 + 1] = pack<T>(c, d);
              }
              tmem_st16(tS + q * 16, pk);
            }
            l += (s0 + s1) + (s2 + s3);
          }
          if ((kSplit || x == 0) && part) {
            const uint32_t i = ring0 + 2 * j + (kSplit && j + 1 < tiles ? 2 : 1);
            ok = ok && warp_wait(&bars->full[i % Dm::kStages], (i / Dm::kStages) & 1, wctx, kFile + __LINE__);
            uint32_t* flag = bars->flag[seg & 1];
            if (tree) {
              if ((tid & 127) < 4) flag[key0 / 32 + (tid & 127)] = 0;
              group_sync(x);
            }
            uint8_t* v = smem + (i % Dm::kStages) * Dm::kTile;
            if (ok && (tid & 127) >= limit) {
#pragma unroll
              for (int e = 0; e < D / 8; ++e)
                *reinterpret_cast<uint4*>(v + (e >> 3) * kHalf + (tid & 127) * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            if (ok && tree) {
              const int n16 = min(limit, kKeys) * (D / 8);     // 16-byte pieces of the nodes' rows
#pragma unroll 2
              for (int e = tid & 127; e < n16; e += 128) {
                const int key = e / (D / 8), ch = e % (D / 8);
                uint4* at = reinterpret_cast<uint4*>(v + (ch >> 3) * kHalf + key * 128 + (ch & 7) * 16);
                uint4 y = *at;
                if (take_out<T>(y)) {
                  *at = y;
                  atomicOr(&flag[(key0 + key) >> 5], 1u << (key & 31));
                }
              }
            }
            fence_async_smem();
          }
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(&bars->p_ready[x]);
        }
        if (kSplit && !mine) more = open(seg + 1);
        if (more && (!kSplit || mine)) deliver_q();   // the next unit's first scores overlap this epilogue
        if (!kSplit || x < tiles) {
          ok = ok && warp_wait(&bars->o_full[x], no & 1, wctx, kFile + __LINE__);
          ++no;
        }
        // kSplit: a row's reference, sum and O are the two groups', joined here; each group takes half of the columns
        float f0 = 1.f, f1 = 0.f;
        if constexpr (kSplit) {
          s_ml[x * 128 + r] = make_float2(ref, l);
          tc_fence_before();
          both_sync();
          const float2 a = s_ml[r], b = s_ml[128 + r];
          ref = fmaxf(a.x, b.x);
          const float base = ref == -INFINITY ? 0.f : ref;
          f0 = fast_exp2(a.x - base);
          f1 = fast_exp2(b.x - base);
          l = a.y * f0 + b.y * f1;
        }
        tc_fence_after();
        const int rec = s.rec, row0 = s.rt * p.Mt + r;
        uint32_t odd_v = 0;      // a node whose V is not all finite
        if (tile0 + tiles > ctx)
          for (int i = max(0, tile0 - ctx) * 4; i < (tile0 + tiles - ctx) * 4; ++i) odd_v |= bars->flag[seg & 1][i];
        const bool live = r < rows;
        const size_t at = size_t(max(rec, 0)) * p.Mt + r;                  // the row's place in the records
        const size_t hr = size_t(s.n0 + row0 / p.G) * p.Hq + s.head * p.G + row0 % p.G;   // and in O
        const float inv = row_inv(l);
#pragma unroll 1
        for (int e = kSplit ? x * (D / 2) : 0; e < (kSplit ? (x + 1) * (D / 2) : D); e += 32) {
          uint32_t o[32];
          tmem_ld32(tmem + (uint32_t(wq * 32) << 16) + kO + (kSplit ? 0 : x * D) + e, o);
          tmem_wait_ld();
          reg_fence<32>(o);
          if constexpr (kSplit) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f0);
            if (tiles > 1) {
              uint32_t y[32];
              tmem_ld32(tmem + (uint32_t(wq * 32) << 16) + kO + D + e, y);
              tmem_wait_ld();
              reg_fence<32>(y);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(fmaf(__uint_as_float(y[i]), f1, __uint_as_float(o[i])));
            }
          }
          if (odd_v && live) {
            const int node = row0 / p.G;
#pragma unroll 1
            for (int j = max(0, tile0 - ctx) * kKeys; j < min(nodes, (tile0 + tiles - ctx) * kKeys); ++j) {
              if (!((bars->flag[seg & 1][j >> 5] >> (j & 31)) & 1u)) continue;
              if (p.mask != nullptr && !p.mask[int64_t(s.n0 + node) * p.mask_row + j]) continue;
              const T* v = reinterpret_cast<const T*>(p.vb + int64_t(s.n0 + j) * p.vb_node + s.head * p.vb_head) + e;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float y = float(v[i]);
                if (!isfinite(y)) o[i] = __float_as_uint(__uint_as_float(o[i]) + y);
              }
            }
          }
          if (rec < 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
          }
          if (live && (rec >= 0 || p.o_f32)) {
            float* dst = rec >= 0 ? p.rec_o + at * D + e : reinterpret_cast<float*>(p.o) + hr * D + e;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4*>(dst + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          } else if (live) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack<T>(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<uint4*>(p.o + (hr * D + e + 2 * i) * 2) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
          }
          __syncwarp();
        }
        tc_fence_before();
        if (live && (!kSplit || x == 0)) {
          if (rec >= 0)
            p.rec_ml[at] = make_float2(ref, l);
          else
            p.lse[hr] = row_lse(ref, l, int(kLift<T>));
        }
      }
      ++na;
      ring0 += 2 * tiles;
      warp_arrive(&bars->seg_empty[seg % kSegRing]);
      ++seg;
      // (the other group has read this one's O)
      if (kSplit && both_any(!ok)) break;
    }
    if (!ok) bars->abort_flag = 1;
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kSoftWarps + 1) tmem_dealloc(tmem, Dm::kTmem);
}

template <typename T, int D, bool kSplit>
cudaError_t launch(const TreeParams& p, const CUtensorMap* m, cudaStream_t s) {
  using Dm = Dims<D, kSplit>;
  cudaError_t e = cudaFuncSetAttribute(tree_rows_sm100_kernel<T, D, kSplit>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, int(Dm::kSmem));
  if (e != cudaSuccess) return e;
  tree_rows_sm100_kernel<T, D, kSplit><<<p.ctas * p.hg, Dm::kThreads, Dm::kSmem, s>>>(m[0], m[1], m[2], m[3], p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t rows(const TreeParams& p, const CUtensorMap* m, cudaStream_t s) {
  return p.Mt > 128 ? launch<T, D, false>(p, m, s) : launch<T, 64, true>(p, m, s);
}

}  // namespace

cudaError_t launch_tree_rows_sm100(const TreeParams& p, int dtype, const CUtensorMap* m, cudaStream_t s) {
  if (dtype == SPLITKV_DTYPE_F16) return p.d == 128 ? rows<__half, 128>(p, m, s) : rows<__half, 64>(p, m, s);
  return p.d == 128 ? rows<__nv_bfloat16, 128>(p, m, s) : rows<__nv_bfloat16, 64>(p, m, s);
}

}  // namespace tree
}  // namespace splitkv
