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
// part 0 of the following ones up to the one in which it ends. kTileBlocks or kFewBlocks blocks per
// CTA that begins a chain; a task is 32 lanes' rows (16 rows x 2 for the few-row kernel's items) by
// kMergeCh channels, a lane owning one row's: every load of a warp is a run of 16-byte quads of
// consecutive rows. Chains of a few parts: a warp per task, the parts' loads in flight together.
// Long chains (one context over most of the grid): the block's warps share a task's parts and add
// their sums through shared memory. Reads chain x (D + 2) x 4 bytes per row from L2; bound by the
// latency of three dependent loads, so registers are kept to four blocks per SM (2 to 3 us at the end
// of a call).
constexpr int kMergeWarps = 8;
constexpr int kLongChain = 16;  // parts from which the warps of a block share a task
constexpr int kMergeBatch = 4;  // parts whose loads a lane has in flight
constexpr int kMergeCh = 8;
constexpr int kTileBlocks = 8, kFewBlocks = 2;

template <int ROWS, int D>
__device__ __forceinline__ void merge_chain(const PagedParams &p, float *part, int ctas, int c,
                                            int y, int ny, float (*sum_s)[kMergeCh + 2][32]) {
  constexpr int RL = ROWS < 32 ? ROWS : 32;        // rows side by side in a warp
  constexpr int CH = kMergeCh;                     // channels per lane
  constexpr int RG = ROWS / RL, CG = D / CH / (32 / RL);  // tasks: row groups x channel groups
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const PartRecord rec = *part_record(part, c, 1);
  // parts 1 .. n - 1 lie in CTAs c + 1 .. c + n - 1 (the first records are loaded beside rec)
  int n = 1;
  for (int i0 = 1;; i0 += 32) {
    const int i = c + i0 + lane;
    int2 next = make_int2(0, 0);  // valid, ends
    if (i < ctas) next = *reinterpret_cast<const int2 *>(part_record(part, i, 0));
    if (!rec.valid) return;
    const unsigned end = __ballot_sync(0xffffffffu, !next.x || next.y);
    if (end) {
      n = min(i0 + __ffs(end), ctas - c);
      break;
    }
  }
  const bool shared = n > kLongChain;
  const int first = shared ? y : y * kMergeWarps + w;
  const int step = shared ? ny : ny * kMergeWarps;
  for (int task = first; task < RG * CG; task += step) {  // the same count for all warps if shared
    const int r = (task / CG) * RL + lane % RL;
    const int q0 = ((task % CG) * (32 / RL) + lane / RL) * (CH / 4);  // first quad of channels
    float m = -INFINITY, l = 0.f, o[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) o[k] = 0.f;
    if (r < rec.rows) {
      const int i_step = shared ? kMergeWarps : 1;
      for (int i0 = shared ? w : 0; i0 < n; i0 += kMergeBatch * i_step) {
        float2 st[kMergeBatch];  // the loads of several parts first, then their sums
        float4 v[kMergeBatch][CH / 4];
#pragma unroll
        for (int b = 0; b < kMergeBatch; ++b) {
          const int i = i0 + b * i_step;
          st[b] = make_float2(-INFINITY, 0.f);
          if (i < n) {
            const int which = i == 0 ? 1 : 0;
            st[b] = *reinterpret_cast<const float2 *>(
                part_stats<ROWS, D>(part, ctas, c + i, which) + r * 2);
            float *rows = part_rows<ROWS, D>(part, ctas, c + i, which);
#pragma unroll
            for (int k = 0; k < CH / 4; ++k) v[b][k] = *part_quad<ROWS>(rows, r, q0 + k);
          }
        }
#pragma unroll
        for (int b = 0; b < kMergeBatch; ++b) {
          if (st[b].x == -INFINITY && st[b].y == 0.f) continue;  // no key here (a NaN's sum is NaN)
          const float mn = fmaxf(m, st[b].x);
          const float fo = m == -INFINITY ? 0.f : ex2(m - mn), fn = ex2(st[b].x - mn);
          l = l * fo + st[b].y * fn;
#pragma unroll
          for (int k = 0; k < CH / 4; ++k) {
            o[4 * k] = o[4 * k] * fo + v[b][k].x * fn;
            o[4 * k + 1] = o[4 * k + 1] * fo + v[b][k].y * fn;
            o[4 * k + 2] = o[4 * k + 2] * fo + v[b][k].z * fn;
            o[4 * k + 3] = o[4 * k + 3] * fo + v[b][k].w * fn;
          }
          m = mn;
        }
      }
    }
    if (shared) {
      __syncthreads();  // the task before has been read
#pragma unroll
      for (int k = 0; k < CH; ++k) sum_s[w][k][lane] = o[k];
      sum_s[w][CH][lane] = m;
      sum_s[w][CH + 1][lane] = l;
      __syncthreads();
      if (w != 0) continue;
      for (int i = 1; i < kMergeWarps; ++i) {
        const float mi = sum_s[i][CH][lane], mn = fmaxf(m, mi);
        const float fo = m == -INFINITY ? 0.f : ex2(m - mn);
        const float fn = mi == -INFINITY ? 0.f : ex2(mi - mn);
        l = l * fo + sum_s[i][CH + 1][lane] * fn;
#pragma unroll
        for (int k = 0; k < CH; ++k) o[k] = o[k] * fo + sum_s[i][k][lane] * fn;
        m = mn;
      }
    }
    if (r >= rec.rows) continue;
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const int q = r / p.group, h = rec.hk * p.group + (r - q * p.group);
    const size_t row = (size_t)rec.row0 + q;
    *reinterpret_cast<uint4 *>(p.out + (row * p.hq + h) * D + q0 * 4) =
        make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                   pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
    if (q0 == 0 && p.lse != nullptr)
      p.lse[(size_t)h * p.total_q + row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
  }
}

// Blocks [0, tile_ctas * kTileBlocks) merge the tile kernel's items, the others the few-row kernel's.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32, 4)
    fat_paged_merge_kernel(const __grid_constant__ PagedParams p, float *tile_part, int tile_ctas,
                           float *few_part, int few_ctas) {
  __shared__ float sum_s[kMergeWarps][kMergeCh + 2][32];
  grid_dep_launch();
  grid_dep_wait();
  int b = blockIdx.x;
  if (b < tile_ctas * kTileBlocks) {
    merge_chain<kTileRows, D>(p, tile_part, tile_ctas, b / kTileBlocks, b % kTileBlocks,
                              kTileBlocks, sum_s);
  } else {
    b -= tile_ctas * kTileBlocks;
    merge_chain<kFewRows, D>(p, few_part, few_ctas, b / kFewBlocks, b % kFewBlocks, kFewBlocks,
                             sum_s);
  }
}

template <int D>
int launch_merge(const PagedParams &p, float *tile_part, int tile_ctas, float *few_part,
                 int few_ctas, cudaStream_t stream) {
  return launch_dependent("paged merge launch", fat_paged_merge_kernel<D>,
                          dim3((unsigned)(tile_ctas * kTileBlocks + few_ctas * kFewBlocks)),
                          kMergeWarps * 32, 0, stream, p, tile_part, tile_ctas, few_part, few_ctas);
}

// The kernels a call launches and their partial rows' places in the workspace. Bounds that allow
// few rows only need one kernel. A total of num_seqs * max_seqlen_q rows says that the requests most
// likely have max_seqlen_q queries each: then the tile kernel alone takes every request, whatever its
// rows, which saves the other one's launch. If it is padding instead, a single token pays for a tile;
// a caller of padded steps gives another total. Tile kernel alone against both, 32 heads over 4, us:
//   32 x 4 tokens over 1000 .. 4000 keys 74.7 / 80.6 (head_dim 64: 38.0 / 44.0), 8 x 64 over 200 .. 900
//   21.9 / 26.5 (18.8 / 23.1), 2 x 1024 over 4000 .. 8000 172.6 / 178.4 (129.9 / 134.4);
//   padded: 32 single tokens over 1000 .. 4000 keys 70.0 / 38.1 (41.0 / 20.2), 8 over 200 .. 900 21.8 /
//   16.6 (14.6 / 10.8).
struct Plan {
  bool few, tile, split;
  size_t few_off, bytes;
};
size_t tile_part_bytes(int d) {
  return (part_floats(paged_tile_ctas(), kTileRows, d) * 4 + 255) & ~(size_t)255;
}
size_t few_part_bytes(int d) { return part_floats(paged_few_ctas(), kFewRows, d) * 4; }
Plan make_plan(const fat_paged_shape_t *sh, const fat_paged_cache_t *c) {
  Plan l{};
  const long long rows = (long long)sh->max_seqlen_q * (sh->num_heads_q / c->num_heads);
  l.tile = rows > kFewRows;
  l.few = !l.tile || (long long)sh->num_seqs * sh->max_seqlen_q != sh->total_q;
  l.split = sh->max_seqlen_k >
            (l.tile ? kWholeKeys : kWholeStages * few_stage_tokens(c->head_dim));
  if (!l.split) return l;
  if (l.tile) l.few_off = tile_part_bytes(c->head_dim);
  l.bytes = l.few_off + (l.few ? few_part_bytes(c->head_dim) : 0);
  return l;
}

// What every call within the bounds can do with: of two plans' partial rows a smaller call may need
// those that the larger one does not (single tokens cut contexts that a chunk leaves whole, and a call
// of padded rows launches both kernels), so each kernel's are counted wherever some call needs them.
size_t workspace_bound(const fat_paged_shape_t *sh, const fat_paged_cache_t *c) {
  const long long rows = (long long)sh->max_seqlen_q * (sh->num_heads_q / c->num_heads);
  size_t bytes = 0;
  if (rows > kFewRows && sh->max_seqlen_k > kWholeKeys) bytes += tile_part_bytes(c->head_dim);
  if (sh->max_seqlen_k > kWholeStages * few_stage_tokens(c->head_dim))
    bytes += few_part_bytes(c->head_dim);
  return bytes;
}

int check_shape(const fat_paged_shape_t *sh, const fat_paged_cache_t *c) {
  if (!sh || !c) return FAT_EINVAL_NULL;
  if (sh->total_q < 0 || sh->num_seqs < 0 || sh->max_seqlen_q < 0 || sh->max_seqlen_k < 0 ||
      sh->num_heads_q <= 0 || sh->table_width < 0 || c->num_heads <= 0 ||
      sh->num_heads_q % c->num_heads)
    return FAT_EINVAL_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return FAT_EINVAL_SHAPE;
  if ((long long)sh->total_q * sh->num_heads_q * c->head_dim > (1LL << 40)) return FAT_EINVAL_SHAPE;
  if (sh->num_heads_q > 65535 || sh->num_seqs > 65535 || sh->num_heads_q / c->num_heads > 128 ||
      sh->max_seqlen_k > (1 << 30))
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
  return workspace_bound(sh, cache);
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
  if (!rc) rc = check_page_strides(cc);
  if (rc) return rc;
  cache = &cc;
  PagedParams p{};
  rc = make_bias_params(&p.bias, bias_table, num_buckets, max_distance, bidirectional, alibi_slopes);
  if (rc) return rc;
  const int group = sh->num_heads_q / cache->num_heads;
  if (bias_table && (p.bias.sat_pos + p.bias.sat_neg > kMaxBiasSpan ||
                     num_buckets * group > kMaxBiasEntries))
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
  p.few_rows = plan.few ? kFewRows : 0;
  p.both = plan.few && plan.tile;
  p.sms = paged_tile_ctas();
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
    rc = launch_paged_few(pf, *cache, s);
    if (rc) return rc;
  }
  if (!plan.split) return FAT_OK;
  const int tile_ctas = plan.tile ? paged_tile_ctas() : 0, few_ctas = plan.few ? paged_few_ctas() : 0;
  return d == 64 ? launch_merge<64>(p, p.part, tile_ctas, pf.part, few_ctas, s)
                 : launch_merge<128>(p, p.part, tile_ctas, pf.part, few_ctas, s);
}

}  // extern "C"
