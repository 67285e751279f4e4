// Verification of drafted tokens against the target's distributions, from given uniform
// random numbers (speculative sampling over a tree; a chain is a tree of one child a node).
//
// The walk starts at node 0 of the sequence (the token that is already certain).  At node
// `cur`, with p = target[cur] and q = draft[cur], its children x_1, x_2, ... (in node order)
// were drawn from q independently.  Child k is accepted when
//     u_k S_k q(x_k) < R_k(x_k),
// where R_1 = p, S_1 = 1, and a rejection leaves the residual
//     R_{k+1} = max(R_k - S_k q, 0),   S_{k+1} = sum R_{k+1}.
// Since q >= 0 the clamps nest: R_k = max(p - c_k q, 0) with c_1 = 0, c_{k+1} = c_k + S_k, so a
// node's residual is its two rows and one scalar, and nothing of vocabulary size is stored.
// Without draft distributions a child stands for certainty (q is 1 at x_k): accepted when
// u_k S_k < p(x_k), a rejection takes x_k out of p and S_{k+1} = S_k - p(x_k).
// The walk ends at a node none of whose children is accepted; the next token is the first i
// with R_1 + ... + R_i > u' sum R (R = p where the residual has no mass), so the accepted
// tokens and it are distributed as the target's own samples.
//
// The outputs are whole numbers decided at borders, so a warp's sums are pairs of float32 (an exact
// two-sum and its carried error, some 48 bits), what joins them and every comparison is float64, all in a
// fixed order.  (A conversion and a float64 addition an entry bound the first kernel: 64 chains over 131072
// entries took 67 us, now 24.)
//
// HBM-bound for large batches: the two rows of the node where the walk ends, 2 V elements a
// sequence; otherwise latency.  One cluster of CTAs takes a sequence: each prefetches all
// children's p(x), q(x) at once (one round of gathers instead of one a level), walks in
// shared memory, and sums its slice of the vocabulary; slice sums are exchanged through
// distributed shared memory and read in rank order, so every CTA takes the same decisions.
// Each warp keeps the sums of its chunks of 512 entries: the search for the next token
// re-reads one chunk (from L2).
//
// Measured (whole calls): one chain of 16 nodes over 32000 entries 8 to 10 us; 64 chains over 131072 25 us, 10 of
// them HBM's (39 us with certainty drafts); 24 trees of 40 nodes over
// 50001 (rows that do not begin on 16 bytes) 30 to 36 us.  The rest is the
// walk's serial steps: the gathers, one pass over the rows a rejection or an end, cluster barriers.
#include <cooperative_groups.h>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "splitkv.h"
#include "splitkv_internal.h"
#include "strided.h"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 512;             // vocabulary entries of one warp step
constexpr int kPerLane = kChunk / 32;
constexpr int kMaxNodes = 1024;
constexpr int kMaxVocab = 1 << 21;
constexpr int kMaxChunks = kMaxVocab / kChunk / 8 + 1;   // chunks of one CTA's slice (a cluster of eight)
constexpr int kMaxCluster = 8;

struct VerifyParams {
  const void *target, *draft;
  int64_t target_row, draft_row;   // row strides in elements
  const void* tokens;
  const int *parents, *node_ptr;
  const float *u_accept, *u_sample;
  int *path, *count;
  void* next;
  int* status;
  int64_t path_row;
  int Nq, V, max_nodes, max_path, tok64;
};

__device__ __forceinline__ float val(float x) { return x; }
__device__ __forceinline__ float val(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float val(__half x) { return __half2float(x); }

// A probability as it counts: entries that are negative, infinite or NaN have no mass (one unsigned comparison of
// the bits of 2^-149 .. the largest finite number).
template <typename T>
__device__ __forceinline__ float mass(T x) {
  const float f = val(x);
  return __float_as_uint(f) - 1u < 0x7f7fffffu ? f : 0.f;
}

// Unevaluated sums hi + lo of two floats, ~48 bits: the vocabulary-long sums need more than float32, and float64
// conversions run at a sixteenth of the float32 rate here (the same pass in float64 took 19,000 clocks, not 5,000).
// Knuth's two-sum: a + b = s + e exactly.
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}
struct Sum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float h, float l) {
    float e;
    two_sum(hi, h, hi, e);
    lo = __fadd_rn(lo, __fadd_rn(e, l));
  }
  __device__ __forceinline__ double value() const { return double(hi) + double(lo); }
};

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

// The residual at the walk's current node: the row itself, max(p - c q, 0), or the row without the rejected tokens.
enum Mode { kRow, kMinus1, kMinus, kWithout };   // (kMinus1: c = 1, after a node's first rejection)
template <typename T>
struct Residual {
  const T* p;
  const T* q;
  double c;
  float ch, cl;        // c as hi + lo
  const int* removed;
  int n_removed;
  Mode mode;
  __device__ __forceinline__ void reset() {
    c = 0.0;
    ch = cl = 0.f;
    n_removed = 0;
    mode = kRow;
  }
  __device__ __forceinline__ void set_c(double x) {
    c = x;
    ch = float(x);
    cl = float(x - double(ch));
    mode = x == 1.0 ? kMinus1 : kMinus;
  }
  // R of entry i with p = pv, q = qv, as hi + lo
  template <Mode kM>
  __device__ __forceinline__ void at(T pv, T qv, int i, float& h, float& l) const {
    h = mass(pv);
    l = 0.f;
    if constexpr (kM == kMinus || kM == kMinus1) {
      // where p > x the difference's rounding error is (p - d) - x exactly (Dekker); elsewhere nothing is left
      const float b = mass(qv), x = kM == kMinus1 ? b : __fmul_rn(ch, b), d = __fsub_rn(h, x);
      l = __fsub_rn(__fsub_rn(h, d), x);
      bool some = d > 0.f;
      if constexpr (kM == kMinus) {
        l = __fsub_rn(l, __fmaf_rn(cl, b, __fmaf_rn(ch, b, -x)));   // c q = x + this
        some = d >= 0.f && __fadd_rn(d, l) > 0.f;
      }
      h = some ? d : 0.f;
      l = some ? l : 0.f;
    }
    if constexpr (kM == kWithout) {
      for (int k = 0; k < n_removed; ++k)
        if (removed[k] == i) h = 0.f;
    }
  }
  __device__ __forceinline__ double value(T pv, T qv, int i) const {
    float h, l;
    if (mode == kMinus || mode == kMinus1)
      at<kMinus>(pv, qv, i, h, l);
    else
      at<kWithout>(pv, qv, i, h, l);
    return double(h) + double(l);
  }
};

// This lane's share of the chunk of entries [base, base + kChunk), in N-element vectors that sit on 16-byte
// boundaries (base may be negative, and the chunk may end behind the row: those entries are not there).
template <typename T, int N, Mode kM>
__device__ __forceinline__ double chunk_sum(const Residual<T>& R, int base, int V, int lane) {
  Sum s[2];   // two chains of additions
  constexpr int kSteps = kPerLane / N;
  if (base >= 0 && base + kChunk <= V) {
    constexpr int kBatch = N == 1 ? 8 : kSteps;   // vectors of a row in flight
#pragma unroll 1
    for (int j0 = 0; j0 < kSteps; j0 += kBatch) {
      Pack<T, N> a[kBatch], b[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = base + ((j0 + j) * 32 + lane) * N;
        a[j] = *reinterpret_cast<const Pack<T, N>*>(R.p + i);
        if constexpr (kM == kMinus || kM == kMinus1) b[j] = *reinterpret_cast<const Pack<T, N>*>(R.q + i);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          float h, l;
          R.template at<kM>(a[j].v[e], b[j].v[e], base + ((j0 + j) * 32 + lane) * N + e, h, l);
          s[(j * N + e) & 1].add(h, l);
        }
      }
    }
  } else {
#pragma unroll 1
    for (int j0 = 0; j0 < kPerLane; j0 += 8) {   // the row's first and last chunk
      T a[8], b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = base + (j0 + j) * 32 + lane;
        const bool there = i >= 0 && i < V;
        a[j] = there ? R.p[i] : T(0.f);
        if constexpr (kM == kMinus || kM == kMinus1) b[j] = there ? R.q[i] : T(0.f);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float h, l;
        R.template at<kM>(a[j], b[j], base + (j0 + j) * 32 + lane, h, l);
        s[j & 1].add(h, l);
      }
    }
  }
  return s[0].value() + s[1].value();
}

// (The steps outside the vocabulary loop run once a launch, on cold instruction caches: rolled loops and shared
// functions, since fetching a line of straight code costs more than running it several times.)
__device__ __noinline__ double warp_sum(double s) {
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__device__ __noinline__ double warp_scan(double x) {   // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 3) tree_verify_kernel(const VerifyParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = int(cluster.block_rank()), ranks = int(cluster.num_blocks());
  const int b = int(blockIdx.x) / ranks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  __shared__ int s_parent[kMaxNodes], s_tok[kMaxNodes], s_removed[kMaxNodes], s_path[kMaxNodes];
  __shared__ float s_p[kMaxNodes], s_q[kMaxNodes], s_u[kMaxNodes];
  __shared__ double s_chunk[kMaxChunks];
  __shared__ double s_total[2];   // this CTA's slice sum, by pass parity
  __shared__ int s_found, s_last;
  __shared__ double s_warp[kWarps];
  __shared__ uint8_t s_first[kMaxNodes];   // accepted as its parent's first child

  const int n0 = p.node_ptr[b], n1 = p.node_ptr[b + 1];
  int n = n1 - n0;
  if (n0 < 0 || n1 < n0 || n1 > p.Nq || n > p.max_nodes) {
    if (tid == 0 && p.status) atomicCAS(p.status, 0, SPLITKV_ERR_INVALID_ARG);
    n = 0;
  }
  const T* target = static_cast<const T*>(p.target);
  const T* draft = static_cast<const T*>(p.draft);
  const int V = p.V;

  for (int i = tid; i < n; i += kThreads) {
    int64_t tok = p.tok64 ? static_cast<const int64_t*>(p.tokens)[n0 + i] : static_cast<const int*>(p.tokens)[n0 + i];
    int par = p.parents[n0 + i];
    if (i > 0 && (par < 0 || par >= i || tok < 0 || tok >= V)) {
      // a node that no walk reaches
      if (p.status) atomicCAS(p.status, 0, SPLITKV_ERR_INVALID_ARG);
      par = -1;
    }
    float pv = 0.f, qv = 1.f;
    if (i > 0 && par >= 0) {
      pv = mass(target[int64_t(n0 + par) * p.target_row + tok]);
      if (draft != nullptr) qv = mass(draft[int64_t(n0 + par) * p.draft_row + tok]);
    }
    s_parent[i] = par;
    s_tok[i] = int(tok);
    s_p[i] = pv;
    s_q[i] = qv;
    const float u = p.u_accept[n0 + i];
    s_u[i] = u;
    s_first[i] = double(u) * double(qv) < double(pv);
  }
  if (tid == 0) {
    s_found = 0x7fffffff;
    s_last = -1;
  }
  __syncthreads();

  Residual<T> R;
  R.removed = s_removed;
  R.reset();
  int cur = 0;
  // Chunks are cut at 16-byte boundaries: the current row begins `shift` entries behind one (the same in both rows).
  int shift = 0, c0 = 0, nc = 0;            // this CTA's chunks
  auto place = [&]() {
    R.p = target + int64_t(n0 + cur) * p.target_row;
    R.q = draft ? draft + int64_t(n0 + cur) * p.draft_row : nullptr;
    shift = N == 1 ? 0 : int(reinterpret_cast<uintptr_t>(R.p) / sizeof(T) % N);
    const int all = (V + shift + kChunk - 1) / kChunk, per = (all + ranks - 1) / ranks;
    c0 = rank * per;
    nc = max(0, min(per, all - c0));
  };
  int pass = 0;
  double before = 0.0;   // mass of the slices before this CTA's

  // Sum of R over the vocabulary; leaves the chunk sums and `before` behind.  Every CTA of the
  // cluster calls it the same number of times.
  auto total = [&]() -> double {
    __syncthreads();   // the last pass's readers of s_chunk are done
    place();
    for (int k = warp; k < nc; k += kWarps) {
      const int base = (c0 + k) * kChunk - shift;
      const double s = warp_sum(R.mode == kRow      ? chunk_sum<T, N, kRow>(R, base, V, lane)
                                : R.mode == kMinus1 ? chunk_sum<T, N, kMinus1>(R, base, V, lane)
                                : R.mode == kMinus  ? chunk_sum<T, N, kMinus>(R, base, V, lane)
                                                    : chunk_sum<T, N, kWithout>(R, base, V, lane));
      if (lane == 0) s_chunk[k] = s;
    }
    __syncthreads();
    if (warp == 0) {
      double s = 0.0;
      for (int k = lane; k < nc; k += 32) s += s_chunk[k];
      s = warp_sum(s);
      if (lane == 0) s_total[pass & 1] = s;
    }
    cluster.sync();
    // lane r reads rank r's sum; added in rank order
    const double part = lane < ranks ? *cluster.map_shared_rank(&s_total[pass & 1], lane) : 0.0;
    double all = 0.0;
#pragma unroll 1
    for (int r = 0; r < ranks; ++r) {
      if (r == rank) before = all;
      all += __shfl_sync(0xffffffffu, part, r);
    }
    ++pass;
    return all;
  };

  int len = n > 0 ? 1 : 0;
  double S = 1.0;
  bool first = true;     // no child of cur has been rejected
  bool summed = false;   // the chunk sums are those of the current R
  const bool writer = rank == 0 && tid == 0;
  int at = 0;            // the last node tried
  bool ended = n == 0;
  for (;;) {
    bool rejected = false;
    while (!ended && !rejected) {
      // the next child of cur (every warp by itself, 32 nodes at a time)
      int child = -1;
      if (len < p.max_path) {
        for (int j0 = (at + 1) & ~31; j0 < n && child < 0; j0 += 32) {
          const int j = j0 + lane;
          const unsigned m = __ballot_sync(0xffffffffu, j > at && j < n && s_parent[j] == cur);
          if (m) child = j0 + __ffs(m) - 1;
        }
      }
      if (child < 0) {
        ended = true;
        break;
      }
      at = child;
      bool taken = s_first[at];
      double r = s_p[at];
      if (!first) {
        const double qv = s_q[at];
        if (draft != nullptr) {
          r = fmax(r - R.c * qv, 0.0);
        } else {
          for (int k = 0; k < R.n_removed; ++k)
            if (s_removed[k] == s_tok[at]) r = 0.0;
        }
        taken = double(s_u[at]) * S * qv < r;
      }
      first = taken;
      summed = false;
      if (taken) {
        if (tid == 0) s_path[len] = at;
        ++len;
        cur = at;
        R.reset();
        S = 1.0;
      } else if (draft != nullptr) {
        R.set_c(R.c + S);
        rejected = true;   // S of what is left
      } else {
        __syncthreads();   // every thread has read the removed list
        if (tid == 0) s_removed[R.n_removed] = s_tok[at];
        __syncthreads();
        ++R.n_removed;
        R.mode = kWithout;
        S = fmax(S - r, 0.0);
      }
    }
    if (n == 0 || (summed && (S > 0.0 || R.mode == kRow))) break;
    if (summed) R.reset();   // nothing left at the end: the target's own row
    S = total();
    summed = true;
  }

  // No CTA leaves while another may read its sums.  (Global writes wait until after the last barrier's arrival: its
  // release would wait for them, 2 us in the middle of the walk.)
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  // the next token
  if (n > 0) {
    const double all = S;
    // the first entry whose running sum exceeds the goal; below the total, so one exists
    double goal = double(p.u_sample[b]) * all;
    goal = fmin(fmax(goal, 0.0), all * (1.0 - 1.2e-16));
    const double mine = s_total[(pass - 1) & 1];
    // the CTA in whose slice the goal lies: the slices' sums partition [0, all)
    const bool here = all > 0.0 && mine > 0.0 && before <= goal && goal < before + mine;
    if (here) {
      // the first chunk whose running sum exceeds the goal (every warp by itself), then the first of its entries, two
      // a thread; where rounding leaves none, the last one with mass
      double run = before, run_k = 0.0;
      int k = -1;
#pragma unroll 1
      for (int k0 = 0; k0 < nc; k0 += 32) {
        const double x = k0 + lane < nc ? s_chunk[k0 + lane] : 0.0;
        const double inc = warp_scan(x);
        const unsigned over = __ballot_sync(0xffffffffu, x > 0.0 && run + inc > goal);
        const unsigned some = __ballot_sync(0xffffffffu, x > 0.0);
        if (some) {
          const int f = over ? __ffs(over) - 1 : 31 - __clz(some);
          k = k0 + f;
          run_k = run + __shfl_sync(0xffffffffu, inc, f) - __shfl_sync(0xffffffffu, x, f);
        }
        if (over) break;
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
      constexpr int kEach = kChunk / kThreads;
      const int i0 = (c0 + k) * kChunk - shift + tid * kEach;
      T x[kEach], y[kEach];
      double r[kEach], sum = 0.0;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const bool there = i0 + e >= 0 && i0 + e < V;
        x[e] = there ? R.p[i0 + e] : T(0.f);
        y[e] = there && R.q != nullptr ? R.q[i0 + e] : T(0.f);
      }
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        r[e] = R.value(x[e], y[e], i0 + e);
        sum += r[e];
      }
      const double inc = warp_scan(sum);
      if (lane == 31) s_warp[warp] = inc;
      __syncthreads();
      for (int w = 0; w < warp; ++w) run_k += s_warp[w];
      run_k += inc - sum;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        run_k += r[e];
        if (r[e] > 0.0) {
          if (run_k > goal) atomicMin(&s_found, i0 + e);
          atomicMax(&s_last, i0 + e);
        }
      }
      __syncthreads();
      if (tid == 0) {
        const int token = s_found < V ? s_found : s_last;
        if (p.tok64)
          static_cast<int64_t*>(p.next)[b] = token;
        else
          static_cast<int*>(p.next)[b] = token;
      }
    }
    if (writer && !(all > 0.0)) {
      if (p.tok64)
        static_cast<int64_t*>(p.next)[b] = -1;
      else
        static_cast<int*>(p.next)[b] = -1;
    }
  } else if (writer) {
    if (p.tok64)
      static_cast<int64_t*>(p.next)[b] = -1;
    else
      static_cast<int*>(p.next)[b] = -1;
  }
  if (rank == 0) {
    int* path = p.path + b * p.path_row;
    if (tid == 0) p.count[b] = len;
    for (int i = tid; i < p.max_path; i += kThreads) path[i] = i >= len ? -1 : i == 0 ? 0 : s_path[i];
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, int N>
cudaError_t launch(const VerifyParams& p, int B, int ranks, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(B * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(ranks);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_verify_kernel<T, N>, p);
}

template <typename T>
cudaError_t dispatch(const VerifyParams& p, int B, int ranks, cudaStream_t s) {
  constexpr int N = 16 / int(sizeof(T));
  // 16-byte loads: a node's two rows have to lie alike about the 16-byte boundaries
  const auto at = [](const void* x) { return int64_t(reinterpret_cast<uintptr_t>(x) / sizeof(T) % N); };
  const bool vec = !p.draft || (at(p.target) == at(p.draft) && p.target_row % N == p.draft_row % N);
  return vec ? launch<T, N>(p, B, ranks, s) : launch<T, 1>(p, B, ranks, s);
}

}  // namespace

extern "C" int splitkv_tree_verify(const splitkv_verify_args* a, void* stream) {
  if (!a) return SPLITKV_ERR_INVALID_ARG;
  if (a->num_seqs < 0 || a->num_nodes < 0 || a->vocab < 1 || a->max_nodes < 1 || a->max_path < 1)
    return SPLITKV_ERR_INVALID_ARG;
  if (a->dtype != SPLITKV_DTYPE_F32 && a->dtype != SPLITKV_DTYPE_BF16 && a->dtype != SPLITKV_DTYPE_F16)
    return SPLITKV_ERR_INVALID_ARG;
  if (a->max_nodes > kMaxNodes || a->vocab > kMaxVocab || a->num_seqs > (1 << 24))
    return SPLITKV_ERR_UNSUPPORTED;
  if (a->num_seqs == 0) return SPLITKV_OK;
  const int es = a->dtype == SPLITKV_DTYPE_F32 ? 4 : 2;
  if (!a->node_ptr || !a->path || !a->count || !a->next || !a->u_sample) return SPLITKV_ERR_INVALID_ARG;
  if (a->num_nodes > 0 && (!a->target || !a->tokens || !a->parents || !a->u_accept)) return SPLITKV_ERR_INVALID_ARG;
  if (!splitkv::ptr_aligned(a->target, es) || !splitkv::ptr_aligned(a->draft, es) || a->target_stride < 0 ||
      a->draft_stride < 0 || a->target_stride > (int64_t(1) << 40) || a->draft_stride > (int64_t(1) << 40) ||
      (a->num_seqs > 1 && a->path_stride < a->max_path) || a->path_stride > (int64_t(1) << 40))
    return SPLITKV_ERR_INVALID_ARG;
  const int ts = a->token_int64 ? 8 : 4;
  if (!splitkv::all_aligned4(a->parents, a->node_ptr, a->u_accept, a->u_sample, a->path, a->count, a->status) ||
      !splitkv::ptr_aligned(a->tokens, ts) || !splitkv::ptr_aligned(a->next, ts))
    return SPLITKV_ERR_INVALID_ARG;
  VerifyParams p;
  p.target = a->target;
  p.draft = a->draft;
  p.target_row = a->target_stride;
  p.draft_row = a->draft_stride;
  p.tokens = a->tokens;
  p.parents = a->parents;
  p.node_ptr = a->node_ptr;
  p.u_accept = a->u_accept;
  p.u_sample = a->u_sample;
  p.path = a->path;
  p.count = a->count;
  p.next = a->next;
  p.status = a->status;
  p.path_row = a->path_stride;
  p.Nq = a->num_nodes;
  p.V = a->vocab;
  p.max_nodes = a->max_nodes;
  p.max_path = a->max_path;
  p.tok64 = a->token_int64 ? 1 : 0;
  // CTAs of a sequence: no more than run at once (three to an SM), and no CTA with less than four chunks.
  const int chunks = (a->vocab + kChunk - 1) / kChunk;
  int ranks = 1;
  while (ranks < kMaxCluster && (chunks >= ranks * kMaxChunks ||
                                 (int64_t(a->num_seqs) * ranks * 2 <= 444 && chunks >= ranks * kWarps)))
    ranks *= 2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = a->dtype == SPLITKV_DTYPE_F32    ? dispatch<float>(p, a->num_seqs, ranks, s)
                  : a->dtype == SPLITKV_DTYPE_BF16 ? dispatch<__nv_bfloat16>(p, a->num_seqs, ranks, s)
                                                   : dispatch<__half>(p, a->num_seqs, ranks, s);
  if (e == cudaSuccess) return SPLITKV_OK;
  cudaGetLastError();
  return SPLITKV_ERR_CUDA;
}
