// fat_paged_tree.cu -- the maps of trees of drafted tokens: from every node's parent its key position and
// the bits of its path, which attention over the paged cache (fat_paged_tree_attn) and the rotary positions
// of the appended rows go by.
//
//   depth_j = 0 where the parent is -1 (the node follows the cached context), else depth_parent + 1;
//   path_j = {j} and the parent's path; position_j = seqlens_k - nodes + depth_j.
//
// A warp per request, 32 nodes at a time, a lane each. Within such a group the paths are closed by doubling
// (five rounds: a lane's bits take in those of the lane at the end of its path so far, and the path gets twice
// as long); what lies before the group is the row of the node that the path enters it from, written earlier by
// the same warp. Kilobytes to a megabyte: bound by the launch and by a group's chain of shuffles and loads.
#include <algorithm>
#include <cstdint>

#include "fat_attn_internal.cuh"

namespace fat {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxNodes = 4096;

struct TreeParams {
  int total, n, max_nodes, words;
  const int32_t *parents, *cu, *lk;
  int32_t *pos;
  uint32_t *mask;
  int *err;
};

__global__ void __launch_bounds__(kThreads) fat_paged_tree_plan_kernel(const TreeParams p) {
  __shared__ int16_t depth_s[kThreads / 32][kMaxNodes];
  grid_dep_launch();
  grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gtid = blockIdx.x * kThreads + threadIdx.x, gthreads = gridDim.x * kThreads;
  {  // rows behind the last request
    const int end = __ldg(p.cu + p.n);
    if (end >= 0) {
      for (long long r = end + (long long)gtid; r < p.total; r += gthreads) p.pos[r] = 0;
      for (long long i = (long long)end * p.words + gtid; i < (long long)p.total * p.words; i += gthreads)
        p.mask[i] = 0u;
    }
  }
  const int i = blockIdx.x * (kThreads / 32) + warp;
  if (i >= p.n) return;
  const int sq = __ldg(p.cu + i), eq = __ldg(p.cu + i + 1), lk = __ldg(p.lk + i), m = eq - sq;
  if (sq < 0 || eq < sq || eq > p.total) {  // corrupt: no rows of its own
    if (lane == 0) atomicOr(p.err, FAT_DEVERR_SEQLENS);
    return;
  }
  uint32_t *rows = p.mask + (size_t)sq * p.words;
  if (m > p.max_nodes || lk < m) {
    if (lane == 0) atomicOr(p.err, FAT_DEVERR_SEQLENS);
    for (int j = lane; j < m; j += 32) p.pos[sq + j] = 0;
    for (long long j = lane; j < (long long)m * p.words; j += 32) rows[j] = 0u;
    return;
  }
  int16_t *depth = depth_s[warp];
  int next = lane < m ? __ldg(p.parents + sq + lane) : -1;
  for (int j0 = 0; j0 < m; j0 += 32) {
    const int j = j0 + lane;
    int parent = next;
    if (j + 32 < m) next = __ldg(p.parents + sq + j + 32);
    if (j < m && (parent < -1 || parent >= j)) {
      atomicOr(p.err, FAT_DEVERR_INDEX);
      parent = -1;
    }
    if (j >= m) parent = -1;
    // bits: the part of the path within the group; up: where it goes on (a lane, or none)
    uint32_t bits = 1u << lane;
    int up = parent >= j0 ? parent - j0 : -1, enter = parent;  // enter: the node before the group, or -1
#pragma unroll
    for (int s = 0; s < 5; ++s) {
      const int from = up < 0 ? lane : up;
      const uint32_t b = __shfl_sync(0xffffffffu, bits, from);
      const int u = __shfl_sync(0xffffffffu, up, from), e = __shfl_sync(0xffffffffu, enter, from);
      if (up >= 0) {
        bits |= b;
        enter = e;
        up = u;
      }
    }
    if (j < m) {
      uint32_t *row = rows + (size_t)j * p.words;
      const uint32_t *before = rows + (size_t)max(enter, 0) * p.words;
      const int g = j0 >> 5;
      for (int w = 0; w < g; ++w) row[w] = enter >= 0 ? before[w] : 0u;
      row[g] = bits;
      for (int w = g + 1; w < p.words; ++w) row[w] = 0u;
      const int d = __popc(bits) + (enter >= 0 ? depth[enter] : 0);
      depth[j] = (int16_t)d;
      p.pos[sq + j] = lk - m + d - 1;
    }
    __syncwarp();  // the rows are read by the groups behind them
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
  // a warp per request, and for the rows behind them at least as many threads as one in eight rows
  const long long warps = std::max<long long>(sh->num_seqs, sh->total_q / 256);
  const int blocks = (int)std::min<long long>((warps + kThreads / 32 - 1) / (kThreads / 32), 1 << 22);
  return launch_dependent("paged tree plan launch", fat_paged_tree_plan_kernel,
                          dim3((unsigned)std::max(blocks, 1)), kThreads, 0,
                          static_cast<cudaStream_t>(sh->stream), p);
}
