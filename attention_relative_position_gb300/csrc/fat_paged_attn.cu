// fat_paged_attn.cu -- attention of new tokens over a paged key/value cache: per row (query, head)
// softmax(scale * q K^T + bias) V over the row's visible keys, whose pages a block table lists.
// Argument checks, the choice of kernels, and the merge of items that share boundaries cut.
//
// A request goes to the kernel that fits its rows (queries x group heads): at most 16 to the few-row
// kernel, more to the tile kernel. Only the device knows the lengths, so a call whose bounds allow
// both launches both, the second beside the first, and each skips the other's requests.
#include <algorithm>
#include <cstdint>

#include "fat_paged.cuh"

namespace fat {
namespace {

// ---- merge of cut items -------------------------------------------------------------------------
// A chain is an item's parts in the order of their CTAs: part 1 of the CTA in which it begins, then
// part 0 of the following ones up to the one in which it ends. One block per (CTA, kMergeRows rows)
// whose CTA begins a chain; kMergeWarps warps share each row's parts, every lane owning D / 32
// channels. Reads chain x (D + 2) x 4 bytes per row from L2, writes a row of out: bound by the
// latency of the chain (a few parts, or all CTAs' when one long item fills the grid).
constexpr int kMergeRows = 2, kMergeWarps = 4;

template <int ROWS, int D>
__global__ void __launch_bounds__(kMergeRows *kMergeWarps * 32)
    fat_paged_merge_kernel(const __grid_constant__ PagedParams p, const int ctas) {
  constexpr int CPL = D / 32;
  __shared__ float acc_s[kMergeRows][kMergeWarps][D];
  __shared__ float2 st_s[kMergeRows][kMergeWarps];
  grid_dep_wait();
  const int c = blockIdx.x;
  const PartRecord rec = *part_record(p.part, c, 1);
  if (!rec.valid || blockIdx.y * kMergeRows >= rec.rows) return;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) / kMergeRows;
  const int rs = (threadIdx.x >> 5) % kMergeRows;
  // parts 1 .. n - 1 lie in CTAs c + 1 .. c + n - 1
  int n = 1;
  for (int i0 = 1;; i0 += 32) {
    const int i = c + i0 + lane;
    const unsigned end = __ballot_sync(0xffffffffu, i >= ctas || part_record(p.part, i, 0)->ends ||
                                                        !part_record(p.part, i, 0)->valid);
    if (end) {
      n = min(i0 + __ffs(end), ctas - c);
      break;
    }
  }
  for (int r0 = blockIdx.y * kMergeRows; r0 < rec.rows; r0 += gridDim.y * kMergeRows) {
    const int r = r0 + rs;
    float m = -INFINITY, l = 0.f, o[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) o[k] = 0.f;
    if (r < rec.rows) {
#pragma unroll 4
      for (int i = w; i < n; i += kMergeWarps) {
        const int which = i == 0 ? 1 : 0;
        const float2 st = *reinterpret_cast<const float2 *>(
            part_stats<ROWS, D>(p.part, ctas, c + i, which) + r * 2);
        const float *src = part_rows<ROWS, D>(p.part, ctas, c + i, which) + r * D + lane * CPL;
        float v[CPL];
        if constexpr (CPL == 4) {
          const float4 t = *reinterpret_cast<const float4 *>(src);
          v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
        } else {
          const float2 t = *reinterpret_cast<const float2 *>(src);
          v[0] = t.x, v[1] = t.y;
        }
        const float mn = fmaxf(m, st.x);
        const float fo = m == -INFINITY ? 0.f : ex2(m - mn);
        const float fn = st.x == -INFINITY ? 0.f : ex2(st.x - mn);
        l = l * fo + st.y * fn;
#pragma unroll
        for (int k = 0; k < CPL; ++k) o[k] = o[k] * fo + v[k] * fn;
        m = mn;
      }
    }
    __syncthreads();  // the rows before have been read
#pragma unroll
    for (int k = 0; k < CPL; ++k) acc_s[rs][w][lane * CPL + k] = o[k];
    if (lane == 0) st_s[rs][w] = make_float2(m, l);
    __syncthreads();
    if (w != 0 || r >= rec.rows) continue;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int i = 0; i < kMergeWarps; ++i) M = fmaxf(M, st_s[rs][i].x);
#pragma unroll
    for (int k = 0; k < CPL; ++k) o[k] = 0.f;
#pragma unroll
    for (int i = 0; i < kMergeWarps; ++i) {
      const float2 st = st_s[rs][i];
      const float f = st.x == -INFINITY ? 0.f : ex2(st.x - M);
      L += st.y * f;
#pragma unroll
      for (int k = 0; k < CPL; ++k) o[k] += acc_s[rs][i][lane * CPL + k] * f;
    }
    const float inv = L > 0.f ? 1.0f / L : 0.f;
    const int q = r / p.group, h = rec.hk * p.group + (r - q * p.group);
    const size_t row = (size_t)rec.row0 + q;
    __nv_bfloat16 *dst = p.out + (row * p.hq + h) * D + lane * CPL;
    if constexpr (CPL == 4)
      *reinterpret_cast<uint2 *>(dst) =
          make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    else
      *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(o[0] * inv, o[1] * inv);
    if (lane == 0 && p.lse != nullptr)
      p.lse[(size_t)h * p.total_q + row] = L > 0.f ? (M + __log2f(L)) * kLn2 : -INFINITY;
  }
}

template <int ROWS, int D>
int launch_merge(const PagedParams &p, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas, std::min(ROWS / kMergeRows, 16));
  cfg.blockDim = dim3(kMergeRows * kMergeWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fat_paged_merge_kernel<ROWS, D>, p, ctas);
  if (e == cudaSuccess) return FAT_OK;
  set_last_error("paged merge launch", (int)e, cudaGetErrorString(e));
  return FAT_ECUDA;
}

// The kernels a call launches and their partial rows' places in the workspace. When every request
// has exactly max_seqlen_q queries (as the totals say), one kernel takes them all.
struct Plan {
  bool few, tile, split;
  size_t few_off, bytes;
};
Plan make_plan(const fat_paged_shape_t *sh, const fat_paged_cache_t *c) {
  Plan l{};
  const long long rows = (long long)sh->max_seqlen_q * (sh->num_heads_q / c->num_heads);
  l.tile = rows > kFewRows;
  l.few = !l.tile || (long long)sh->num_seqs * sh->max_seqlen_q != sh->total_q;
  l.split = sh->max_seqlen_k > kWholeKeys;
  if (!l.split) return l;
  if (l.tile) l.few_off = (part_floats(paged_tile_ctas(), kTileRows, c->head_dim) * 4 + 255) & ~(size_t)255;
  l.bytes = l.few_off + (l.few ? part_floats(paged_few_ctas(), kFewRows, c->head_dim) * 4 : 0);
  return l;
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
  return make_plan(sh, cache).bytes;
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
  if (bias_table && (p.bias.sat_pos + p.bias.sat_neg > kMaxBiasSpan || num_buckets * group > kMaxBiasEntries))
    return FAT_EUNSUPPORTED;
  if (sh->total_q == 0 || sh->num_seqs == 0 || sh->max_seqlen_q == 0) return FAT_OK;
  if (!q || !cu_seqlens_q || !seqlens_k || !out || (sh->table_width > 0 && !block_table))
    return FAT_EINVAL_NULL;
  const Plan plan = make_plan(sh, cache);
  const size_t need = plan.bytes;
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
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.table = block_table;
  p.cu = cu_seqlens_q;
  p.lk = seqlens_k;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = softmax_scale * kLog2e;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  runtime_knobs(&p.timeout_ns, &p.debug_flags);
  p.few_rows = kFewRows;
  const int d = cache->head_dim;
  const cudaStream_t s = static_cast<cudaStream_t>(sh->stream);
  p.split = plan.split;
  PagedParams pf = p;
  p.part = static_cast<float *>(workspace);
  pf.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + plan.few_off);
  if (plan.tile) {
    rc = launch_paged_tile(p, *cache, s);
    if (rc) return rc;
  }
  if (plan.few) {
    rc = launch_paged_few(pf, *cache, s, plan.tile);
    if (rc) return rc;
  }
  if (!plan.split) return FAT_OK;
  if (plan.tile) {
    rc = d == 64 ? launch_merge<kTileRows, 64>(p, paged_tile_ctas(), s)
                 : launch_merge<kTileRows, 128>(p, paged_tile_ctas(), s);
    if (rc) return rc;
  }
  if (plan.few)
    rc = d == 64 ? launch_merge<kFewRows, 64>(pf, paged_few_ctas(), s)
                 : launch_merge<kFewRows, 128>(pf, paged_few_ctas(), s);
  return rc;
}

}  // extern "C"
