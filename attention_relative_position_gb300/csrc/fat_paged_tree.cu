// fat_paged_tree.cu -- the maps of trees of drafted tokens: from every node's parent its key position and
// the bits of its path, which attention over the paged cache (fat_paged_tree_attn) and the rotary positions
// of the appended rows go by.
//
//   depth_j = 0 where the parent is -1 (the node follows the cached context), else depth_parent + 1;
//   path_j = {j} and the parent's path; position_j = seqlens_k - nodes + depth_j.
//
// A block per request: its parents in shared memory, a thread per node that walks up to the root. Parents
// come before their children, so the path's bits are met from the highest word of the row to the lowest,
// one word in a register at a time. Tens of kilobytes: bound by the launch and by the longest path (a
// step of the walk is one read of shared memory).
#include <algorithm>
#include <cstdint>

#include "fat_attn_internal.cuh"

namespace fat {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxNodes = 4096;
constexpr int kPadBlocks = 4;  // blocks that clear the rows behind the last request

struct TreeParams {
  int total, n, max_nodes, words;
  const int32_t *parents, *cu, *lk;
  int32_t *pos;
  uint32_t *mask;
  int *err;
};

__global__ void __launch_bounds__(kThreads) fat_paged_tree_plan_kernel(const TreeParams p) {
  extern __shared__ int16_t up[];  // [max_nodes]
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= p.n) {  // rows behind the last request
    const int end = __ldg(p.cu + p.n);
    if (end < 0 || end > p.total) return;
    const int b = blockIdx.x - p.n;
    for (long long r = end + (long long)b * kThreads + tid; r < p.total; r += kPadBlocks * kThreads)
      p.pos[r] = 0;
    const long long last = (long long)p.total * p.words;
    for (long long i = (long long)end * p.words + b * kThreads + tid; i < last;
         i += kPadBlocks * kThreads)
      p.mask[i] = 0u;
    return;
  }
  const int sq = __ldg(p.cu + blockIdx.x), eq = __ldg(p.cu + blockIdx.x + 1);
  const int lk = __ldg(p.lk + blockIdx.x), m = eq - sq;
  if (sq < 0 || eq < sq || eq > p.total) {  // corrupt: no rows of its own
    if (tid == 0) atomicOr(p.err, FAT_DEVERR_SEQLENS);
    return;
  }
  const bool ok = m <= p.max_nodes && lk >= m;
  if (!ok && tid == 0) atomicOr(p.err, FAT_DEVERR_SEQLENS);
  if (ok)
    for (int j = tid; j < m; j += kThreads) {
      int u = __ldg(p.parents + sq + j);
      if (u < -1 || u >= j) {
        atomicOr(p.err, FAT_DEVERR_INDEX);
        u = -1;
      }
      up[j] = (int16_t)u;
    }
  __syncthreads();
  for (int j = tid; j < m; j += kThreads) {
    uint32_t *row = p.mask + (size_t)(sq + j) * p.words;
    int w = p.words - 1, depth = -1;
    if (ok) {
      for (; w > j >> 5; --w) row[w] = 0u;
      uint32_t bits = 0;
      for (int a = j; a >= 0; a = up[a]) {
        for (; w > a >> 5; --w) {
          row[w] = bits;
          bits = 0;
        }
        bits |= 1u << (a & 31);
        ++depth;
      }
      row[w--] = bits;
    }
    for (; w >= 0; --w) row[w] = 0u;
    p.pos[sq + j] = ok ? lk - m + depth : 0;
  }
}

struct Ints {
  const int32_t *p;
  long long n;
};
bool share_memory(const Ints &a, const Ints &b) {
  return a.n > 0 && b.n > 0 && a.p < b.p + b.n && b.p < a.p + a.n;
}
bool odd4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace
}  // namespace fat

using namespace fat;

extern "C" int fat_paged_tree_plan(const fat_tree_shape_t *sh, const int32_t *parents,
                                   const int32_t *cu_seqlens_q, const int32_t *seqlens_k,
                                   int32_t *positions, int32_t *tree_mask) {
  if (!sh) return FAT_EINVAL_NULL;
  if (sh->total_q < 0 || sh->num_seqs < 0 || sh->max_seqlen_q < 0 || sh->mask_words < 0 ||
      sh->mask_words < (sh->max_seqlen_q + 31LL) / 32)
    return FAT_EINVAL_SHAPE;
  if (sh->max_seqlen_q > kMaxNodes || sh->num_seqs > (1 << 24)) return FAT_EUNSUPPORTED;
  if (sh->total_q == 0) return FAT_OK;
  if (!cu_seqlens_q || !positions || (sh->mask_words > 0 && !tree_mask) ||
      (sh->num_seqs > 0 && (!seqlens_k || !parents)))
    return FAT_EINVAL_NULL;
  if (odd4(parents) || odd4(cu_seqlens_q) || odd4(seqlens_k) || odd4(positions) || odd4(tree_mask))
    return FAT_EINVAL_SHAPE;
  const long long T = sh->total_q, n = sh->num_seqs;
  const Ints arrays[5] = {{positions, T}, {tree_mask, T * sh->mask_words}, {parents, T},
                          {cu_seqlens_q, n + 1}, {seqlens_k, n}};
  for (int i = 0; i < 2; ++i)
    for (int j = i + 1; j < 5; ++j)
      if (share_memory(arrays[i], arrays[j])) return FAT_EINVAL_SHAPE;
  TreeParams p{};
  const int rc = device_error_address(&p.err);
  if (rc) return rc;
  p.total = sh->total_q;
  p.n = sh->num_seqs;
  p.max_nodes = sh->max_seqlen_q;
  p.words = sh->mask_words;
  p.parents = parents;
  p.cu = cu_seqlens_q;
  p.lk = seqlens_k;
  p.pos = positions;
  p.mask = reinterpret_cast<uint32_t *>(tree_mask);
  return launch_dependent("paged tree plan launch", fat_paged_tree_plan_kernel,
                          dim3((unsigned)(sh->num_seqs + kPadBlocks)), kThreads,
                          (size_t)sh->max_seqlen_q * 2, static_cast<cudaStream_t>(sh->stream), p);
}
