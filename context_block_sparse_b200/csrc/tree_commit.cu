// Commit of a draft tree's accepted nodes: row i of sequence b's path becomes cache position
// context_lens[b] + i, for keys and values and for every layer in one launch,
//
//   cache[l, page_table[b, t / page], t % page] = new[l, node_ptr[b] + path[b, i]],
//   t = context_lens[b] + i, i < count[b];
//
// without a path, every node of the sequence in order (a block of new tokens).
//
// A copy: 4 * L * sum(count) * Hkv * d elements' bytes over HBM, or a launch's latency when
// that is small.  A CTA takes some path rows of one (layer, sequence): its threads resolve
// the rows' source and destination first (the sequence's numbers and its path at once, then the page
// table: two dependent loads, paid once per CTA), then stream 16-byte vectors with eight loads in flight
// per thread.  24 layers of 48 sequences (42 MB where all eight rows stay) take 14.3 us a call, a single layer of one
// sequence 4.6.
#include <cstdint>

#include "common.cuh"
#include "splitkv.h"
#include "splitkv_internal.h"
#include "strided.h"

namespace {

constexpr int kThreads = 128;
constexpr int kMaxRows = 32;   // path rows of one CTA
constexpr int kUnroll = 4;     // vectors of keys and of values in flight a thread

struct CommitParams {
  const char *kb, *vb;
  char *kc, *vc;
  int64_t kb_s[3], vb_s[3], kc_s[4], vc_s[4];   // bytes: layer, node, head / layer, page, slot, head
  const int *node_ptr, *path, *count, *table, *lens;
  int64_t path_row, table_row;
  int* status;
  int B, Nq, rows_per_cta, max_rows, page_shift, num_pages, max_pages, Hkv, vecs;   // vecs: 16-byte vectors of a head
};

__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const CommitParams p) {
  __shared__ int64_t src_node[kMaxRows], dst_page[kMaxRows];
  __shared__ int dst_slot[kMaxRows];
  const int b = blockIdx.y, layer = blockIdx.z;
  const int first = int(blockIdx.x) * p.rows_per_cta;
  // everything but the page is asked for at once, whatever of it turns out to be wanted
  const int i = first + int(threadIdx.x);
  const int n0 = p.node_ptr[b], n1 = p.node_ptr[b + 1], len = p.lens[b];
  int count = p.path ? p.count[b] : 0, node = i;
  if (p.path && int(threadIdx.x) < p.rows_per_cta && i < p.max_rows) node = p.path[b * p.path_row + i];
  const int64_t t = int64_t(len) + i, pi = t >> p.page_shift;
  int page = -1;
  if (len >= 0 && int(threadIdx.x) < p.rows_per_cta && pi < p.max_pages) page = p.table[b * p.table_row + pi];
  if (!p.path) count = n1 - n0;
  bool bad = n0 < 0 || n1 < n0 || n1 > p.Nq || len < 0 || count < 0 || count > p.max_rows;
  if (bad) count = 0;
  const int rows = min(count - first, p.rows_per_cta);
  if (int(threadIdx.x) < rows) {
    if (node < 0 || node >= n1 - n0 || page < 0 || page >= p.num_pages) {
      page = -1;   // nothing is written for this row
      bad = true;
    }
    src_node[threadIdx.x] = int64_t(n0) + node;
    dst_page[threadIdx.x] = page;
    dst_slot[threadIdx.x] = int(t & ((1 << p.page_shift) - 1));
  }
  if (bad && p.status) atomicCAS(p.status, 0, SPLITKV_ERR_INVALID_ARG);
  if (rows <= 0) return;
  __syncthreads();
  const int per_row = p.Hkv * p.vecs;
  const int total = rows * per_row;
  const char* kb = p.kb + layer * p.kb_s[0];
  const char* vb = p.vb + layer * p.vb_s[0];
  char* kc = p.kc + layer * p.kc_s[0];
  char* vc = p.vc + layer * p.vc_s[0];
  for (int i0 = threadIdx.x; i0 < total; i0 += kThreads * kUnroll) {
    uint4 x[kUnroll], y[kUnroll];
    int64_t kd[kUnroll], vd[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = i0 + u * kThreads;
      kd[u] = -1;
      if (j < total) {
        const int r = j / per_row, rem = j - r * per_row;
        const int h = rem / p.vecs, c = (rem - h * p.vecs) * 16;
        if (dst_page[r] >= 0) {
          x[u] = __ldg(reinterpret_cast<const uint4*>(kb + src_node[r] * p.kb_s[1] + h * p.kb_s[2] + c));
          y[u] = __ldg(reinterpret_cast<const uint4*>(vb + src_node[r] * p.vb_s[1] + h * p.vb_s[2] + c));
          kd[u] = dst_page[r] * p.kc_s[1] + dst_slot[r] * p.kc_s[2] + h * p.kc_s[3] + c;
          vd[u] = dst_page[r] * p.vc_s[1] + dst_slot[r] * p.vc_s[2] + h * p.vc_s[3] + c;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (kd[u] >= 0) {
        *reinterpret_cast<uint4*>(kc + kd[u]) = x[u];
        *reinterpret_cast<uint4*>(vc + vd[u]) = y[u];
      }
    }
  }
}

bool strides_ok(const void* ptr, const int64_t* s, int n, int64_t es) {
  if (!splitkv::ptr_aligned(ptr, 16) || !ptr) return false;
  for (int i = 0; i < n; ++i)
    if (s[i] < 0 || s[i] > (int64_t(1) << 44) || (s[i] * es) % 16) return false;
  return true;
}

}  // namespace

extern "C" int splitkv_tree_commit(const splitkv_commit_args* a, void* stream) {
  if (!a) return SPLITKV_ERR_INVALID_ARG;
  if (a->num_layers < 0 || a->num_seqs < 0 || a->num_nodes < 0 || a->max_rows < 0 || a->num_kv_heads < 1 ||
      a->head_dim < 1 || a->head_dim > 65536 || a->num_kv_heads > 65536 || a->num_pages < 0 || a->max_pages < 0)
    return SPLITKV_ERR_INVALID_ARG;
  if (a->page_size < 1 || a->page_size > 65536 || (a->page_size & (a->page_size - 1))) return SPLITKV_ERR_INVALID_ARG;
  if (a->elem_bytes != 2 && a->elem_bytes != 4 && a->elem_bytes != 1) return SPLITKV_ERR_INVALID_ARG;
  if ((int64_t(a->head_dim) * a->elem_bytes) % 16) return SPLITKV_ERR_UNSUPPORTED;
  if (a->num_layers == 0 || a->num_seqs == 0 || a->max_rows == 0 || a->num_nodes == 0) return SPLITKV_OK;
  if (a->num_layers > 65535 || a->num_seqs > 65535) return SPLITKV_ERR_UNSUPPORTED;
  // (the kernel counts a CTA's 16-byte vectors in 32 bits, and steps past the last of them)
  if (int64_t(a->num_kv_heads) * a->head_dim * a->elem_bytes / 16 * kMaxRows > 0x7fffffff - kThreads * kUnroll)
    return SPLITKV_ERR_UNSUPPORTED;
  const int64_t es = a->elem_bytes;
  if (!strides_ok(a->kb, a->kb_stride, 3, es) || !strides_ok(a->vb, a->vb_stride, 3, es) ||
      !strides_ok(a->k_cache, a->k_stride, 4, es) || !strides_ok(a->v_cache, a->v_stride, 4, es))
    return SPLITKV_ERR_INVALID_ARG;
  if (!a->node_ptr || !a->page_table || !a->context_lens || (a->path && !a->count)) return SPLITKV_ERR_INVALID_ARG;
  if (!splitkv::all_aligned4(a->node_ptr, a->page_table, a->context_lens, a->path, a->count, a->status) ||
      a->table_stride < 0 || (a->path && a->path_stride < 0))
    return SPLITKV_ERR_INVALID_ARG;
  // A row that is read while another CTA writes it would be either's: the new keys and values lie apart from both caches,
  // and the caches from each other.
  const int64_t row = int64_t(a->head_dim) * es, L = a->num_layers, H = a->num_kv_heads;
  const auto fresh = [&](const void* ptr, const int64_t* s) {
    return splitkv::Strided{ptr, row, 3, {L, a->num_nodes, H}, {s[0] * es, s[1] * es, s[2] * es}};
  };
  const auto cache = [&](const void* ptr, const int64_t* s) {
    return splitkv::Strided{ptr, row, 4, {L, a->num_pages, a->page_size, H}, {s[0] * es, s[1] * es, s[2] * es, s[3] * es}};
  };
  const splitkv::Strided kb = fresh(a->kb, a->kb_stride), vb = fresh(a->vb, a->vb_stride);
  const splitkv::Strided kc = cache(a->k_cache, a->k_stride), vc = cache(a->v_cache, a->v_stride);
  if (!splitkv::apart(kb, kc) || !splitkv::apart(kb, vc) || !splitkv::apart(vb, kc) || !splitkv::apart(vb, vc) ||
      !splitkv::apart(kc, vc))
    return SPLITKV_ERR_INVALID_ARG;
  CommitParams p;
  p.kb = static_cast<const char*>(a->kb);
  p.vb = static_cast<const char*>(a->vb);
  p.kc = static_cast<char*>(a->k_cache);
  p.vc = static_cast<char*>(a->v_cache);
  for (int i = 0; i < 3; ++i) {
    p.kb_s[i] = a->kb_stride[i] * es;
    p.vb_s[i] = a->vb_stride[i] * es;
  }
  for (int i = 0; i < 4; ++i) {
    p.kc_s[i] = a->k_stride[i] * es;
    p.vc_s[i] = a->v_stride[i] * es;
  }
  p.node_ptr = a->node_ptr;
  p.path = a->path;
  p.count = a->count;
  p.table = a->page_table;
  p.lens = a->context_lens;
  p.path_row = a->path_stride;
  p.table_row = a->table_stride;
  p.status = a->status;
  p.B = a->num_seqs;
  p.Nq = a->num_nodes;
  p.max_rows = a->max_rows;
  p.num_pages = a->num_pages;
  p.max_pages = a->max_pages;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a->page_size) ++p.page_shift;
  p.Hkv = a->num_kv_heads;
  p.vecs = int(int64_t(a->head_dim) * es / 16);
  // Path rows of a CTA: few when few CTAs would run (the copy is then one CTA's latency),
  // many when the grid fills the GPU anyway.
  // (Without a path no sequence has more rows than there are nodes, however loose the caller's bound.)
  const int64_t groups = int64_t(a->num_layers) * a->num_seqs;
  const int64_t most = a->path || a->max_rows < a->num_nodes ? a->max_rows : a->num_nodes;
  int rows = kMaxRows;
  while (rows > 2 && groups * ((most + rows - 1) / rows) < 296) rows /= 2;
  p.rows_per_cta = rows;
  const dim3 grid(unsigned((most + rows - 1) / rows), unsigned(a->num_seqs), unsigned(a->num_layers));
  tree_commit_kernel<<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SPLITKV_OK : SPLITKV_ERR_CUDA;
}
