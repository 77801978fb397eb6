// fat_paged_attn.cu -- attention of new tokens over a paged key/value cache: per row (query, head)
// softmax(scale * q K^T + bias) V over the row's visible keys, whose pages a block table lists.
//
// One warp per row walks its keys 32 at a time: lane i takes the dot product with key i (bias and
// mask applied), the maximum and sum are running ones, and the lanes then own head_dim / 32
// channels each for P V.
#include <algorithm>
#include <cstdint>

#include "fat_attn_internal.cuh"

namespace fat {
namespace {

struct PagedParams {
  int total_q, n, max_q, max_k, hq, hkv, group, width, log2_page, num_pages;
  long long page_stride, tok_stride, head_stride;
  const __nv_bfloat16 *q, *k, *v;
  const int32_t *table, *cu, *lk;
  BiasParams bias;
  int causal;
  float scale_log2;
  __nv_bfloat16 *out;
  float *lse;
  int *err;
};

template <int D>
__global__ void __launch_bounds__(128) fat_paged_rows_kernel(const PagedParams p) {
  constexpr int CPL = D / 32;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x;
  const int h = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (h >= p.hq) return;
  int lo = 0, hi = p.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.cu + mid) <= row)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int sq = __ldg(p.cu + lo), eq = __ldg(p.cu + lo + 1), lk = __ldg(p.lk + lo);
  if (row < sq || row >= eq) return;
  if (sq < 0 || eq > p.total_q || eq - sq > p.max_q || lk < 0 || lk > p.max_k ||
      lk > ((long long)p.width << p.log2_page)) {
    if (lane == 0) atomicOr(p.err, FAT_DEVERR_SEQLENS);
    return;
  }
  const int qpos = lk - (eq - sq) + (row - sq), hk = h / p.group;
  const int nk = p.causal ? min(lk, qpos + 1) : lk;
  const float slope = p.bias.slopes ? __ldg(p.bias.slopes + h) * kLog2e : 0.f;
  const __nv_bfloat16 *q = p.q + ((size_t)row * p.hq + h) * D;
  float m = -INFINITY, l = 0.f, o[CPL];
  for (int c = 0; c < CPL; ++c) o[c] = 0.f;
  for (int k0 = 0; k0 < nk; k0 += 32) {
    const int key = k0 + lane;
    long long off = -1;
    float x = -INFINITY;
    if (key < nk) {
      const int page = __ldg(p.table + (size_t)lo * p.width + (key >> p.log2_page));
      float dot = 0.f;
      if ((unsigned)page < (unsigned)p.num_pages) {
        off = page * p.page_stride + (key & ((1 << p.log2_page) - 1)) * p.tok_stride +
              hk * p.head_stride;
        for (int c = 0; c < D; ++c)
          dot = fmaf(__bfloat162float(q[c]), __bfloat162float(p.k[off + c]), dot);
      } else {
        atomicOr(p.err, FAT_DEVERR_PAGES);
      }
      const int delta = key - qpos;
      x = dot * p.scale_log2;
      if (p.bias.table)
        x += __ldg(p.bias.table + (size_t)t5_bucket_dev(delta, p.bias) * p.hq + h) * kLog2e;
      x -= slope * (float)(delta < 0 ? -delta : delta);
    }
    float mx = x;
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    const float mn = fmaxf(m, mx);
    const float corr = m == -INFINITY ? 0.f : ex2(m - mn);
    const float pr = x == -INFINITY ? 0.f : ex2(x - mn);
    m = mn;
    l = l * corr + pr;
    for (int c = 0; c < CPL; ++c) o[c] *= corr;
    for (int j = 0; j < min(32, nk - k0); ++j) {
      const float pj = __shfl_sync(0xffffffffu, pr, j);
      const long long oj = __shfl_sync(0xffffffffu, off, j);
      if (oj >= 0)
        for (int c = 0; c < CPL; ++c)
          o[c] = fmaf(pj, __bfloat162float(p.v[oj + lane * CPL + c]), o[c]);
    }
  }
  for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
  const float inv = l > 0.f ? 1.0f / l : 0.f;
  for (int c = 0; c < CPL; ++c)
    p.out[((size_t)row * p.hq + h) * D + lane * CPL + c] = __float2bfloat16(o[c] * inv);
  if (lane == 0 && p.lse)
    p.lse[(size_t)h * p.total_q + row] = l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
}

int check_shape(const fat_paged_shape_t *sh, const fat_paged_cache_t *c) {
  if (!sh || !c) return FAT_EINVAL_NULL;
  if (sh->total_q < 0 || sh->num_seqs < 0 || sh->max_seqlen_q < 0 || sh->max_seqlen_k < 0 ||
      sh->num_heads_q <= 0 || sh->table_width < 0 || c->num_heads <= 0 ||
      sh->num_heads_q % c->num_heads)
    return FAT_EINVAL_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return FAT_EINVAL_SHAPE;
  if ((long long)sh->total_q * sh->num_heads_q * c->head_dim > (1LL << 40)) return FAT_EINVAL_SHAPE;
  if (sh->num_heads_q > 65535 || sh->num_seqs > 65535 || sh->num_heads_q / c->num_heads > 128)
    return FAT_EUNSUPPORTED;
  return FAT_OK;
}

bool odd(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

}  // namespace
}  // namespace fat

using namespace fat;

extern "C" {

size_t fat_paged_attn_workspace_size(const fat_paged_shape_t *sh, const fat_paged_cache_t *cache) {
  if (check_shape(sh, cache)) return 0;
  return 0;
}

int fat_paged_attn(const fat_paged_shape_t *sh, const fat_paged_cache_t *cache, const void *q,
                   const int32_t *block_table, const int32_t *cu_seqlens_q,
                   const int32_t *seqlens_k, const float *bias_table, int num_buckets,
                   int max_distance, int bidirectional, const float *alibi_slopes, int causal,
                   float softmax_scale, void *workspace, size_t workspace_bytes, void *out,
                   float *lse) {
  int rc = check_shape(sh, cache);
  if (rc) return rc;
  int lg = 0;
  fat_paged_cache_t cc;
  rc = check_paged_cache(cache, &cc, &lg);
  if (rc) return rc;
  cache = &cc;
  PagedParams p{};
  rc = make_bias_params(&p.bias, bias_table, num_buckets, max_distance, bidirectional, alibi_slopes);
  if (rc) return rc;
  const int group = sh->num_heads_q / cache->num_heads;
  if (bias_table && (p.bias.sat_pos + p.bias.sat_neg > 8192 || num_buckets * group > 4096))
    return FAT_EUNSUPPORTED;
  if (sh->total_q == 0 || sh->num_seqs == 0 || sh->max_seqlen_q == 0) return FAT_OK;
  if (!q || !cu_seqlens_q || !seqlens_k || !out || (sh->table_width > 0 && !block_table))
    return FAT_EINVAL_NULL;
  const size_t need = fat_paged_attn_workspace_size(sh, cache);
  if (need && !workspace) return FAT_EINVAL_NULL;
  if (odd(q, 16) || odd(out, 16) || odd(lse, 16) || odd(bias_table, 16) || odd(alibi_slopes, 16) ||
      odd(block_table, 4) || odd(cu_seqlens_q, 4) || odd(seqlens_k, 4) || odd(workspace, 256) ||
      workspace_bytes < need)
    return FAT_EINVAL_SHAPE;
  rc = device_error_address(&p.err);
  if (rc) return rc;
  p.total_q = sh->total_q;
  p.n = sh->num_seqs;
  p.max_q = sh->max_seqlen_q;
  p.max_k = sh->max_seqlen_k;
  p.hq = sh->num_heads_q;
  p.hkv = cache->num_heads;
  p.group = group;
  p.width = sh->table_width;
  p.log2_page = lg;
  p.num_pages = cache->num_pages;
  p.page_stride = cache->stride_page;
  p.tok_stride = cache->stride_token;
  p.head_stride = cache->stride_head;
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.k = static_cast<const __nv_bfloat16 *>(cache->k);
  p.v = static_cast<const __nv_bfloat16 *>(cache->v);
  p.table = block_table;
  p.cu = cu_seqlens_q;
  p.lk = seqlens_k;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = softmax_scale * kLog2e;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  const dim3 grid(sh->total_q, (sh->num_heads_q + 3) / 4);
  const cudaStream_t s = static_cast<cudaStream_t>(sh->stream);
  if (cache->head_dim == 64)
    fat_paged_rows_kernel<64><<<grid, 128, 0, s>>>(p);
  else
    fat_paged_rows_kernel<128><<<grid, 128, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return FAT_OK;
  set_last_error("paged attention launch", (int)e, cudaGetErrorString(e));
  return FAT_ECUDA;
}

}  // extern "C"
