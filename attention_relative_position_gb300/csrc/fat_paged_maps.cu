// fat_paged_maps.cu -- what a serving step does around attention over a paged key/value cache: the
// step's maps (block tables, slots, positions) from the requests' lengths, rotary positions at
// explicit positions, and the new key/value rows written into their slots.
//
//   plan: request i holds ctx_i cached tokens and brings new_i; with page size s it has
//         ceil(ctx_i / s) pages and needs ceil((ctx_i + new_i) / s) of them. The missing ones come
//         from a list of free pages in request order (exclusive prefix sums of the needs), and
//         token j of request i goes to slot table[i][(ctx_i + j) / s] * s + (ctx_i + j) % s.
//   rows: y = a (x cos p - x' sin p, x sin p + x' cos p) for the channel pairs of the rotated part
//         of each head, p = position * rate of the pair; the other channels are copied.
#include <algorithm>
#include <array>
#include <cmath>
#include <cstdint>

#include "fat_attn_internal.cuh"

namespace fat {
namespace {

// ---- plan ---------------------------------------------------------------------------------------
// A few hundred kilobytes at most: bound by the latency of one launch and of the scan. Every block
// scans all lengths by itself (they are read from L2; a separate scan launch would cost more than
// the repeated reads) and then takes its share of the tokens and pages, finding each one's request
// by binary search over the prefix sums in shared memory. Requests are taken kPlanTile at a time.
// 64 requests with a token each: 3.7 us (3.4 from a graph); 1000 requests with 47 K tokens: 5.0 (4.7).
constexpr int kPlanThreads = 256;
constexpr int kPlanPer = 4;  // consecutive requests per thread
constexpr int kPlanTile = kPlanThreads * kPlanPer;

struct PlanParams {
  int n, log2_page, num_pages, width, num_free, max_tokens;
  const int32_t *ctx, *add, *free_pages;
  int32_t *table, *cu, *lk, *pos, *slots, *counts;
  int *err;
};

struct PlanPair {
  long long tok, page;
};
__device__ __forceinline__ PlanPair plan_add(PlanPair a, PlanPair b) {
  return PlanPair{a.tok + b.tok, a.page + b.page};
}

// The last index i in [0, m) with start[i] <= x (start[0] <= x): among requests without tokens the
// last one, which is the one that holds x.
__device__ __forceinline__ int plan_find(const int *start, int m, int x) {
  int lo = 0, hi = m - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) fat_paged_plan_kernel(const PlanParams p) {
  __shared__ int tok_s[kPlanTile];   // first token of each request of the tile
  __shared__ int page_s[kPlanTile];  // first free-list index of each request
  __shared__ int ctx_s[kPlanTile];   // cached tokens; -1 - ctx: a request that takes no pages
  __shared__ PlanPair warp_s[kPlanThreads / 32];
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gtid = blockIdx.x * kPlanThreads + tid, gthreads = gridDim.x * kPlanThreads;
  const int page_mask = (1 << p.log2_page) - 1;
  const long long row_tokens = (long long)p.width << p.log2_page;
  PlanPair base{0, 0};
  for (int i0 = 0; i0 < p.n; i0 += kPlanTile) {
    const int m = min(kPlanTile, p.n - i0);
    int c[kPlanPer], a[kPlanPer], need[kPlanPer];
    PlanPair sum{0, 0};
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      const int i = tid * kPlanPer + k;
      c[k] = i < m ? __ldg(p.ctx + i0 + i) : 0;
      a[k] = i < m ? __ldg(p.add + i0 + i) : 0;
    }
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      if (c[k] < 0 || a[k] < 0) {
        if (blockIdx.x == 0) atomicOr(p.err, FAT_DEVERR_SEQLENS);
        c[k] = a[k] = 0;
      }
      const long long all = (long long)c[k] + a[k];
      const bool fits = all <= row_tokens;
      if (!fits && blockIdx.x == 0) atomicOr(p.err, FAT_DEVERR_PAGES);
      need[k] = fits ? (int)(((all + page_mask) >> p.log2_page) -
                             (((long long)c[k] + page_mask) >> p.log2_page))
                     : 0;
      if (!fits) c[k] = -1 - c[k];
      sum.tok += a[k];
      sum.page += need[k];
    }
    PlanPair inc = sum;  // inclusive over the warp, then over the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, inc.tok, o);
      const long long g = __shfl_up_sync(0xffffffffu, inc.page, o);
      if (lane >= o) inc = plan_add(inc, PlanPair{t, g});
    }
    __syncthreads();  // the previous tile's shared arrays are no longer read
    if (lane == 31) warp_s[warp] = inc;
    __syncthreads();
    PlanPair at = base, total = base;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) at = plan_add(at, warp_s[w]);
      total = plan_add(total, warp_s[w]);
    }
    at.tok += inc.tok - sum.tok;
    at.page += inc.page - sum.page;
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      const int i = tid * kPlanPer + k;
      if (i < m) {
        tok_s[i] = (int)min(at.tok, (long long)p.max_tokens);
        page_s[i] = (int)min(at.page, 0x7fffffffLL);
        ctx_s[i] = c[k];
        if (blockIdx.x == 0) {
          const long long ctx = c[k] < 0 ? -1 - (long long)c[k] : c[k];
          p.cu[i0 + i] = (int)min(at.tok, (long long)p.max_tokens);
          p.lk[i0 + i] = (int)min(ctx + a[k], 0x7fffffffLL);
        }
      }
      at.tok += a[k];
      at.page += need[k];
    }
    __syncthreads();
    // the tile's tokens
    const int t_end = (int)min(total.tok, (long long)p.max_tokens);
    for (long long t = min(base.tok, (long long)p.max_tokens) + gtid; t < t_end; t += gthreads) {
      const int i = plan_find(tok_s, m, (int)t);
      const bool fits = ctx_s[i] >= 0;
      const int ctx = fits ? ctx_s[i] : -1 - ctx_s[i];
      const int pos = (int)min((long long)ctx + ((int)t - tok_s[i]), 0x7fffffffLL);
      int slot = -1;
      if (fits) {
        const int col = pos >> p.log2_page, have = (int)(((long long)ctx + page_mask) >> p.log2_page);
        int page;
        if (col < have) {  // the last page it already holds
          page = p.table[(size_t)(i0 + i) * p.width + col];
        } else {
          const long long f = (long long)page_s[i] + (col - have);
          page = f < p.num_free ? __ldg(p.free_pages + f) : -1;
        }
        if ((unsigned)page < (unsigned)p.num_pages)
          slot = (page << p.log2_page) + (pos & page_mask);
        else
          atomicOr(p.err, FAT_DEVERR_PAGES);
      }
      p.pos[t] = pos;
      p.slots[t] = slot;
    }
    // the tile's new pages
    const long long f_end = min(total.page, 0x7fffffffLL);
    for (long long f = base.page + gtid; f < f_end; f += gthreads) {
      const int i = plan_find(page_s, m, (int)f);
      const int have = (int)(((long long)ctx_s[i] + page_mask) >> p.log2_page);
      int page = f < p.num_free ? __ldg(p.free_pages + f) : -1;
      if ((unsigned)page >= (unsigned)p.num_pages) {
        page = -1;
        atomicOr(p.err, FAT_DEVERR_PAGES);
      }
      p.table[(size_t)(i0 + i) * p.width + have + (f - page_s[i])] = page;
    }
    base = total;
  }
  const int tokens = (int)min(base.tok, (long long)p.max_tokens);
  if (gtid == 0) {
    if (base.tok > p.max_tokens) atomicOr(p.err, FAT_DEVERR_SEQLENS);
    p.cu[p.n] = tokens;
    p.counts[0] = (int)min(base.page, 0x7fffffffLL);
    p.counts[1] = (int)min(base.tok, 0x7fffffffLL);
  }
  for (long long t = (long long)tokens + gtid; t < p.max_tokens; t += gthreads) {  // padding
    p.pos[t] = 0;
    p.slots[t] = -1;
  }
}

// ---- rows ---------------------------------------------------------------------------------------
// Memory bound: every row is read and written once. A thread takes one (token, unit) position,
// computes its cosines and sines once (while its first rows are on their way) and turns that unit of
// a run of heads (all heads share them), kRowBatch heads' loads in flight together. A unit is one
// 16-byte chunk (pairs 2i, 2i + 1 lie inside it), or with the halves layout two chunks, i and
// i + rotary_dim / 2, that turn together; what is not rotated goes chunk by chunk. Few tokens: the
// heads are split over more threads (the run length is launch_rows' choice), since a decode step's
// rows are bound by latency. Small blocks end more evenly: 16383 x 16 x 128 in 22.9 us (5.9 TB/s)
// against 25.1 with 256 threads and half as many of them; 131072 x 12 x 64 in 59.3 us (6.8 TB/s, the
// measured copy rate); 37 x 32 x 128 in 2.9 us (2.4 from a graph), the latency of a launch and three
// dependent loads.
// Angles as in fat_rope_apply: position * rate mod one turn in 64-bit integers, exact at any
// position, its top 24 bits through sincospif.
constexpr int kRowThreads = 128;
constexpr int kRowBatch = 4;

struct RowSeg {
  const uint16_t *src;
  uint16_t *dst;
  long long src_tok, src_head, dst_tok, dst_head;  // element strides
  int heads;
  int rotate;
  int to_slots;  // dst is a cache: the token's slot gives its row
};
struct RowParams {
  RowSeg seg[3];
  int nseg, tokens, units, pair_units, half_chunks, all_heads, run;  // run: heads per thread
  int log2_page;
  long long page_stride, num_slots;
  float sign;
  const int32_t *positions, *slots;
  int *err;
  fat_rope_t rope;
};

__device__ __forceinline__ uint4 rotate_pairs(uint4 v, const float2 (&cs)[8]) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&w[k]));
    w[k] = pack_bf16x2(a.x * cs[k].x - a.y * cs[k].y, a.x * cs[k].y + a.y * cs[k].x);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void rotate_halves(uint4 &u, uint4 &v, const float2 (&cs)[8]) {
  uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&a[k]));
    const float2 y = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&b[k]));
    const float2 c0 = cs[2 * k], c1 = cs[2 * k + 1];
    a[k] = pack_bf16x2(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
    b[k] = pack_bf16x2(x.x * c0.y + y.x * c0.x, x.y * c1.y + y.y * c1.x);
  }
  u = make_uint4(a[0], a[1], a[2], a[3]);
  v = make_uint4(b[0], b[1], b[2], b[3]);
}

template <bool PAIRS>
__global__ void __launch_bounds__(kRowThreads) fat_rows_kernel(const __grid_constant__ RowParams p) {
  grid_dep_wait();
  const long long i = (long long)blockIdx.x * kRowThreads + threadIdx.x;
  const int t = (int)(i / p.units), u = (int)(i - (long long)t * p.units);
  if (t >= p.tokens) return;
  const bool turned = u < p.pair_units;
  const bool two = !PAIRS && turned;
  const int chunk = (PAIRS || turned) ? u : u + p.pair_units;
  // this thread's heads: `left` of them, of all segments in a row, from head h0 of segment sg on
  int sg = 0, h0 = blockIdx.y * p.run, left = min(p.run, p.all_heads - h0);
  while (h0 >= p.seg[sg].heads) h0 -= p.seg[sg++].heads;
  int n = min(left, p.seg[sg].heads - h0);  // of them in this segment
  const uint16_t *src =
      p.seg[sg].src + (long long)t * p.seg[sg].src_tok + h0 * p.seg[sg].src_head + chunk * 8;
  uint4 lo[kRowBatch], hi[kRowBatch];
  auto load = [&]() {
    const long long step = p.seg[sg].src_head;
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b)
      if (b < n) {
        lo[b] = *reinterpret_cast<const uint4 *>(src + b * step);
        if (two) hi[b] = *reinterpret_cast<const uint4 *>(src + b * step + p.half_chunks * 8);
      }
  };
  // The first heads' rows are on their way while the angles are computed.
  load();
  float2 cs[8];
  if (turned) {
    // negative positions wrap in two's complement: still exact modulo one turn
    const unsigned long long pos = (unsigned long long)(long long)__ldg(p.positions + t);
#pragma unroll
    for (int k = 0; k < (PAIRS ? 4 : 8); ++k) {
      const unsigned long long turns = pos * p.rope.rate[u * (PAIRS ? 4 : 8) + k];
      const float frac = (float)(uint32_t)(turns >> 40) * (1.0f / 16777216.0f);
      float sn, cn;
      sincospif(2.0f * frac, &sn, &cn);
      cs[k] = make_float2(cn * p.rope.amplitude, sn * p.sign * p.rope.amplitude);
    }
  }
  while (true) {
    const RowSeg &s = p.seg[sg];
    long long row = (long long)t * s.dst_tok;
    bool keep = true;
    if (s.to_slots) {
      const int slot = __ldg(p.slots + t);
      const int page = slot >> p.log2_page;
      row = (long long)page * p.page_stride +
            (long long)(slot - (page << p.log2_page)) * s.dst_tok;
      keep = slot >= 0 && slot < p.num_slots;
      if (slot >= p.num_slots) atomicOr(p.err, FAT_DEVERR_INDEX);
    }
    uint16_t *dst = s.dst + row + h0 * s.dst_head + chunk * 8;
    const bool turn = turned && s.rotate;
    left -= n;
    while (keep) {
#pragma unroll
      for (int b = 0; b < kRowBatch; ++b)
        if (b < n) {
          if (turn) {
            if constexpr (PAIRS)
              lo[b] = rotate_pairs(lo[b], cs);
            else
              rotate_halves(lo[b], hi[b], cs);
          }
          *reinterpret_cast<uint4 *>(dst + b * s.dst_head) = lo[b];
          if (two) *reinterpret_cast<uint4 *>(dst + b * s.dst_head + p.half_chunks * 8) = hi[b];
        }
      if ((n -= kRowBatch) <= 0) break;
      src += kRowBatch * s.src_head;
      dst += kRowBatch * s.dst_head;
      load();
    }
    if (left <= 0) break;
    ++sg;
    h0 = 0;
    n = min(left, p.seg[sg].heads);
    src = p.seg[sg].src + (long long)t * p.seg[sg].src_tok + chunk * 8;
    load();
  }
}

bool odd16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool odd4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
// A stride of rows that are accessed 16 bytes at a time
bool bad_stride(long long s) { return s < 0 || (s & 7) != 0; }

struct Ints {
  const int32_t *p;
  long long count;
};
bool share_memory(const Ints &a, const Ints &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.count > 0 && b.count > 0 && x < y + 4 * (uintptr_t)b.count &&
         y < x + 4 * (uintptr_t)a.count;
}

// Whether rows of d elements at every combination of three indexes lie apart: from the smallest stride
// on, each one is at least what the indexes before it span (an index of one value spans nothing).
struct Extent {
  long long stride, count;
};
bool rows_apart(int d, std::array<Extent, 3> e) {
  std::sort(e.begin(), e.end(), [](const Extent &a, const Extent &b) { return a.stride < b.stride; });
  double span = d;
  for (const Extent &x : e) {
    if (x.count <= 1) continue;
    if ((double)x.stride < span) return false;
    span += (double)x.stride * (double)(x.count - 1);
  }
  return true;
}

int check_rope(const fat_rope_t *r, int head_dim) {
  if (r->rotary_dim < 16 || r->rotary_dim % 16 || r->rotary_dim > 2 * FAT_ROPE_MAX_PAIRS ||
      r->rotary_dim > head_dim)
    return FAT_EINVAL_SHAPE;
  return FAT_OK;
}

// head_dim, the rotation (null: rows are copied) and the segments are set: fill in the rest and
// launch. A thread takes all heads of its position when the positions alone give every SM
// kRowThreadsPerSm threads, else a run of at least kRowBatch of them.
constexpr int kRowThreadsPerSm = 2048;
int launch_rows(RowParams &p, const fat_rope_t *rope, int head_dim, cudaStream_t stream) {
  if (rope) {
    p.rope = *rope;
  } else {
    p.rope.rotary_dim = 0;
    p.rope.interleaved = 1;
    p.rope.amplitude = 1.f;
  }
  const bool pairs = p.rope.interleaved != 0;
  const int chunks = head_dim / 8;
  p.half_chunks = p.rope.rotary_dim / 16;
  p.pair_units = pairs ? p.rope.rotary_dim / 8 : p.half_chunks;
  p.units = pairs ? chunks : chunks - p.half_chunks;
  p.all_heads = 0;
  for (int i = 0; i < p.nseg; ++i) p.all_heads += p.seg[i].heads;
  const long long sms = sm_count() > 0 ? sm_count() : 152;
  const long long positions = (long long)p.tokens * p.units;
  const long long want = std::max<long long>(1, sms * kRowThreadsPerSm / positions);  // runs
  const long long runs =
      std::min<long long>(std::min<long long>(want, (p.all_heads + kRowBatch - 1) / kRowBatch), 65535);
  p.run = (int)(((p.all_heads + runs - 1) / runs + kRowBatch - 1) / kRowBatch * kRowBatch);
  const long long blocks = (positions + kRowThreads - 1) / kRowThreads;
  if (blocks > 0x7fffffffLL || (p.all_heads + p.run - 1) / p.run > 65535) return FAT_EUNSUPPORTED;
  const dim3 grid((unsigned)blocks, (unsigned)((p.all_heads + p.run - 1) / p.run));
  return launch_dependent("rotary / append rows launch",
                          pairs ? fat_rows_kernel<true> : fat_rows_kernel<false>, grid, kRowThreads,
                          0, stream, p);
}

}  // namespace

int check_paged_cache(const fat_paged_cache_t *in, fat_paged_cache_t *c, int *log2_page) {
  if (!in || !in->k || !in->v) return FAT_EINVAL_NULL;
  *c = *in;
  if (c->num_pages <= 0 || c->num_heads <= 0 || c->head_dim <= 0 || c->head_dim % 8)
    return FAT_EINVAL_SHAPE;
  int lg = 0;
  while (lg < 16 && (1 << lg) < c->page_size) ++lg;
  if (c->page_size < 16 || c->page_size != (1 << lg)) return FAT_EINVAL_SHAPE;
  if ((long long)c->num_pages * c->page_size > 0x7fffffffLL) return FAT_EINVAL_SHAPE;
  // a stride over one entry says nothing
  if (c->num_heads == 1) c->stride_head = c->stride_token;
  if (c->num_pages == 1)
    c->stride_page = std::max(c->stride_token * c->page_size, c->stride_head * c->num_heads);
  if (odd16(c->k) || odd16(c->v) || bad_stride(c->stride_page) || bad_stride(c->stride_token) ||
      bad_stride(c->stride_head))
    return FAT_EINVAL_SHAPE;
  // rows of different heads, tokens and pages lie apart
  if (c->stride_token < c->head_dim || c->stride_head < c->head_dim ||
      c->stride_page < c->head_dim ||
      !rows_apart(c->head_dim, {{{c->stride_token, c->page_size},
                                 {c->stride_head, c->num_heads},
                                 {c->stride_page, c->num_pages}}}))
    return FAT_EINVAL_SHAPE;
  *log2_page = lg;
  return FAT_OK;
}

}  // namespace fat

using namespace fat;

extern "C" {

int fat_paged_plan(const fat_plan_shape_t *sh, const int32_t *ctx_lens, const int32_t *new_lens,
                   const int32_t *free_pages, int32_t *block_table, int32_t *cu_seqlens_q,
                   int32_t *seqlens_k, int32_t *positions, int32_t *slots, int32_t *counts) {
  if (!sh || !cu_seqlens_q || !counts) return FAT_EINVAL_NULL;
  if (sh->num_seqs < 0 || sh->num_pages <= 0 || sh->table_width < 0 || sh->num_free < 0 ||
      sh->max_tokens < 0)
    return FAT_EINVAL_SHAPE;
  if (sh->num_seqs > 0 && (!ctx_lens || !new_lens || !seqlens_k)) return FAT_EINVAL_NULL;
  if (sh->num_seqs > 0 && sh->table_width > 0 && !block_table) return FAT_EINVAL_NULL;
  if (sh->max_tokens > 0 && (!positions || !slots)) return FAT_EINVAL_NULL;
  if (sh->num_free > 0 && !free_pages) return FAT_EINVAL_NULL;
  int lg = 0;
  while (lg < 16 && (1 << lg) < sh->page_size) ++lg;
  if (sh->page_size < 16 || sh->page_size != (1 << lg)) return FAT_EINVAL_SHAPE;
  if ((long long)sh->num_pages * sh->page_size > 0x7fffffffLL) return FAT_EINVAL_SHAPE;
  if (odd4(ctx_lens) || odd4(new_lens) || odd4(free_pages) || odd4(block_table) ||
      odd4(cu_seqlens_q) || odd4(seqlens_k) || odd4(positions) || odd4(slots) || odd4(counts))
    return FAT_EINVAL_SHAPE;
  // every block reads the lengths and the free list while others write: no result lies over them
  const long long n = sh->num_seqs, T = sh->max_tokens;
  const Ints arrays[9] = {{block_table, n * sh->table_width}, {cu_seqlens_q, n + 1}, {seqlens_k, n},
                          {positions, T}, {slots, T}, {counts, 2}, {ctx_lens, n}, {new_lens, n},
                          {free_pages, sh->num_free}};
  for (int i = 0; i < 6; ++i)
    for (int j = i + 1; j < 9; ++j)
      if (share_memory(arrays[i], arrays[j])) return FAT_EINVAL_SHAPE;
  PlanParams p{};
  int rc = device_error_address(&p.err);
  if (rc) return rc;
  p.n = sh->num_seqs;
  p.log2_page = lg;
  p.num_pages = sh->num_pages;
  p.width = sh->table_width;
  p.num_free = sh->num_free;
  p.max_tokens = sh->max_tokens;
  p.ctx = ctx_lens;
  p.add = new_lens;
  p.free_pages = free_pages;
  p.table = block_table;
  p.cu = cu_seqlens_q;
  p.lk = seqlens_k;
  p.pos = positions;
  p.slots = slots;
  p.counts = counts;
  const int sms = sm_count() > 0 ? sm_count() : 152;
  // a block for every 256 tokens or requests, two per SM at most: a thread's tokens are looked up one
  // after the other (47 K tokens of 1000 requests from a graph: 4.7 us, with a quarter of the blocks 6.6)
  const int units = std::max(sh->max_tokens, sh->num_seqs);
  const int blocks = std::max(1, std::min(2 * sms, (units + 255) / 256));
  return launch_dependent("paged plan launch", fat_paged_plan_kernel, dim3((unsigned)blocks),
                          kPlanThreads, 0, static_cast<cudaStream_t>(sh->stream), p);
}

int fat_rope_init(fat_rope_t *r, int rotary_dim, int interleaved, double base, double factor,
                  double low_turns, double high_turns, double original_length, double amplitude) {
  if (!r) return FAT_EINVAL_NULL;
  if (rotary_dim < 16 || rotary_dim % 16 || rotary_dim > 2 * FAT_ROPE_MAX_PAIRS)
    return FAT_EINVAL_SHAPE;
  if (!(base > 1.0) || !std::isfinite(base) || !(factor > 0.0) || !std::isfinite(factor) ||
      !((float)amplitude > 0.f) || !std::isfinite((float)amplitude) || !(original_length >= 0.0) ||
      !std::isfinite(original_length))
    return FAT_EINVAL_SHAPE;
  if (original_length > 0.0 &&
      (!(low_turns >= 0.0) || !(high_turns > low_turns) || !std::isfinite(high_turns)))
    return FAT_EINVAL_SHAPE;
  fat_rope_t made{};
  made.rotary_dim = rotary_dim;
  made.interleaved = interleaved ? 1 : 0;
  made.amplitude = (float)amplitude;
  const double two_pi = 6.283185307179586476925286766559;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double turns = std::pow(base, -2.0 * i / rotary_dim) / two_pi;  // per position
    double keep = 0.0;
    if (original_length > 0.0)
      keep = std::min(1.0, std::max(0.0, (original_length * turns - low_turns) /
                                             (high_turns - low_turns)));
    turns = turns * keep + turns * (1.0 - keep) / factor;
    if (!std::isfinite(turns)) return FAT_EINVAL_SHAPE;  // a factor next to zero
    const double scaled = std::ldexp(turns - std::floor(turns), 64);
    made.rate[i] = scaled >= 18446744073709551615.0 ? ~0ull : (unsigned long long)scaled;
  }
  *r = made;
  return FAT_OK;
}

int fat_rope_embed(const fat_rope_shape_t *sh, const fat_rope_t *rope, const void *x, void *y,
                   const int32_t *positions, int inverse) {
  if (!sh || !rope) return FAT_EINVAL_NULL;
  if (sh->tokens < 0 || sh->num_heads <= 0 || sh->head_dim <= 0 || sh->head_dim % 8)
    return FAT_EINVAL_SHAPE;
  int rc = check_rope(rope, sh->head_dim);
  if (rc) return rc;
  if (sh->tokens == 0) return FAT_OK;
  if (!x || !y || !positions) return FAT_EINVAL_NULL;
  if (odd16(x) || odd16(y) || odd4(positions) || bad_stride(sh->x_stride_token) ||
      bad_stride(sh->x_stride_head) || bad_stride(sh->y_stride_token) ||
      bad_stride(sh->y_stride_head))
    return FAT_EINVAL_SHAPE;
  // rows of y lie apart; in place, every row stays where it is
  if (!rows_apart(sh->head_dim, {{{sh->y_stride_head, sh->num_heads},
                                  {sh->y_stride_token, sh->tokens},
                                  {0, 1}}}))
    return FAT_EINVAL_SHAPE;
  if (x == y && ((sh->tokens > 1 && sh->x_stride_token != sh->y_stride_token) ||
                 (sh->num_heads > 1 && sh->x_stride_head != sh->y_stride_head)))
    return FAT_EINVAL_SHAPE;
  RowParams p{};
  p.seg[0] = RowSeg{static_cast<const uint16_t *>(x), static_cast<uint16_t *>(y),
                    sh->x_stride_token, sh->x_stride_head, sh->y_stride_token, sh->y_stride_head,
                    sh->num_heads, 1, 0};
  p.nseg = 1;
  p.tokens = sh->tokens;
  p.sign = inverse ? -1.f : 1.f;
  p.positions = positions;
  return launch_rows(p, rope, sh->head_dim, static_cast<cudaStream_t>(sh->stream));
}

int fat_paged_append(const fat_append_shape_t *sh, const fat_paged_cache_t *cache,
                     const fat_rope_t *rope, const void *q, const void *k, const void *v,
                     const int32_t *positions, const int32_t *slots, void *q_out) {
  if (!sh || !cache) return FAT_EINVAL_NULL;
  int lg = 0;
  fat_paged_cache_t cc;
  int rc = check_paged_cache(cache, &cc, &lg);
  if (rc) return rc;
  cache = &cc;
  if (sh->tokens < 0 || (q && sh->num_heads_q <= 0)) return FAT_EINVAL_SHAPE;
  if (rope) {
    rc = check_rope(rope, cache->head_dim);
    if (rc) return rc;
  }
  if ((q == nullptr) != (q_out == nullptr)) return FAT_EINVAL_NULL;
  if (sh->tokens == 0) return FAT_OK;
  if (!k || !v || !slots || (rope && !positions)) return FAT_EINVAL_NULL;
  const int d = cache->head_dim, H = cache->num_heads;
  if (odd16(q) || odd16(k) || odd16(v) || odd16(q_out) || odd4(positions) || odd4(slots) ||
      bad_stride(sh->k_stride_token) || bad_stride(sh->k_stride_head) ||
      bad_stride(sh->v_stride_token) || bad_stride(sh->v_stride_head))
    return FAT_EINVAL_SHAPE;
  if (q && (bad_stride(sh->q_stride_token) || bad_stride(sh->q_stride_head)))
    return FAT_EINVAL_SHAPE;
  const long long qd = (long long)sh->num_heads_q * d;
  if (q && q == q_out && ((sh->tokens > 1 && sh->q_stride_token != qd) ||
                          (sh->num_heads_q > 1 && sh->q_stride_head != d)))
    return FAT_EINVAL_SHAPE;
  RowParams p{};
  rc = device_error_address(&p.err);
  if (rc) return rc;
  const int turn = rope ? 1 : 0;
  p.seg[0] = RowSeg{static_cast<const uint16_t *>(k), static_cast<uint16_t *>(cache->k),
                    sh->k_stride_token, sh->k_stride_head, cache->stride_token,
                    cache->stride_head, H, turn, 1};
  p.seg[1] = RowSeg{static_cast<const uint16_t *>(v), static_cast<uint16_t *>(cache->v),
                    sh->v_stride_token, sh->v_stride_head, cache->stride_token,
                    cache->stride_head, H, 0, 1};
  p.nseg = 2;
  if (q) {
    p.seg[2] = RowSeg{static_cast<const uint16_t *>(q), static_cast<uint16_t *>(q_out),
                      sh->q_stride_token, sh->q_stride_head, qd, d, sh->num_heads_q, turn, 0};
    p.nseg = 3;
  }
  p.tokens = sh->tokens;
  p.sign = 1.f;
  p.positions = positions;
  p.slots = slots;
  p.log2_page = lg;
  p.page_stride = cache->stride_page;
  p.num_slots = (long long)cache->num_pages << lg;
  return launch_rows(p, rope, d, static_cast<cudaStream_t>(sh->stream));
}

}  // extern "C"
