// fat_paged.cuh -- what the kernels of paged attention share: their parameters, the division of a
// ragged batch into equal shares of work, and the layout of the partial rows that shares leave.
//
// Division. The lengths are known on the device only. An item is (request, key/value head) for the
// few-row kernel and (request, key/value head, block of queries) for the tile kernel; its cost is
// the number of key stages its rows see (at least 1). All items in order form one line of total
// cost U, and CTA c of G takes the stretch [c, c + 1) * max(ceil(U / G), min_share): every SM gets
// the same number of stages whatever the lengths are. An item cut by a boundary leaves, in each
// CTA that holds a part, unnormalised fp32 rows with their maximum and sum; a CTA has at most two
// such parts (its first item's end or middle, its last item's beginning), so the workspace depends
// on the grid alone, and a second grid merges them in the order of the CTAs (no atomics: the result
// does not depend on timing).
#pragma once
#include "fat_attn_internal.cuh"

namespace fat {

constexpr int kMaxBiasSpan = 8192;     // sat_neg + sat_pos of a bias table, at most
constexpr int kMaxBiasEntries = 4096;  // buckets x group, at most: larger tables are not tested

struct PagedParams {
  int total_q, n, max_q, max_k, hq, hkv, group, width, log2_page, num_pages, head_outer;
  const __nv_bfloat16 *q;
  const int32_t *table, *cu, *lk;
  BiasParams bias;
  int causal;
  float scale_log2;
  __nv_bfloat16 *out;
  float *lse;
  int *err;
  long long timeout_ns;
  int debug_flags;
  int few_rows;   // requests with at most this many rows (queries x group) are the few-row kernel's
                  // (0: the tile kernel takes all)
  int both;       // the call launches both kernels: they share the SMs (see share_find)
  int sms;
  int split;      // 0: items are not cut (each goes to the CTA in whose share it begins)
  float *part;    // partial rows of this kernel's grid (see PartLayout)
  // Trees (null: a request's queries follow one another): query j sees the keys before the request's
  // first query and those further ones whose bit is set in its row of `mask`, and sits at key position
  // pos[row], as does the key that it brings.
  const int32_t *pos;
  const uint32_t *mask;
  int mask_words;
};

// A request as the kernels see it.
struct PagedDoc {
  int sq, lq, lk;
  bool ok;
};
template <bool TREE>
__device__ __forceinline__ PagedDoc paged_doc(const PagedParams &p, int i) {
  PagedDoc d;
  d.sq = __ldg(p.cu + i);
  const int eq = __ldg(p.cu + i + 1);
  d.lk = __ldg(p.lk + i);
  d.ok = d.sq >= 0 && eq >= d.sq && eq <= p.total_q && eq - d.sq <= p.max_q && d.lk >= 0 &&
         d.lk <= p.max_k && d.lk <= ((long long)p.width << p.log2_page) &&
         (!TREE || d.lk >= eq - d.sq);
  d.lq = eq - d.sq;
  return d;
}

// Trees: the key position of row `row` of a request whose first query is at `shift` (its last key at
// lk - 1): what lies outside is taken as the nearest end.
__device__ __forceinline__ int tree_pos(const PagedParams &p, int row, int shift, int lk) {
  return min(max(__ldg(p.pos + row), shift), lk - 1);
}
// The bits of keys n .. n + 31 behind the first query's for a row of the mask (n < 0: keys before it, which
// every row sees); bits at or beyond lim are 0.
__device__ __forceinline__ uint32_t tree_bits(const PagedParams &p, const uint32_t *row, int n,
                                              int lim) {
  if (n <= -32) return lim >= 32 ? 0xffffffffu : lim <= 0 ? 0u : (1u << lim) - 1u;
  const int i = n >> 5;  // -1 for n in -32 .. -1
  const uint32_t lo = i < 0 ? 0xffffffffu : i < p.mask_words ? __ldg(row + i) : 0u;
  const uint32_t hi = i + 1 < p.mask_words ? __ldg(row + i + 1) : 0u;
  const uint32_t b = __funnelshift_r(lo, hi, n & 31);
  return lim >= 32 ? b : lim <= 0 ? 0u : b & ((1u << lim) - 1u);
}

// ---- costs --------------------------------------------------------------------------------------
// Few-row kernel: stages of 8 KB of keys and values for every key/value head, and kFewItem for the
// fixed costs of an item (its first loads, the merge of its warps). From a graph, in us, for a cost of
// 1 / 5 / 10 / 20: drafted tokens 30.1 / 26.5 / 25.0 / 24.8, mixed step 59.4 / 56.8 / 53.8 / 50.8, 64
// requests of 1 to 1024 tokens over 500 to 8000 keys (32 heads over 8 of 128 channels) 219 / 217 / 212 /
// 217, decode 100.9 / 100.2 / 98.8 / 99.2.
__host__ __device__ constexpr int few_stage_tokens(int d) { return 2048 / d; }
constexpr int kFewItem = 10;
__host__ __device__ inline int few_item_cost(int stages) { return stages + kFewItem; }
template <int D>
struct FewCost {
  const PagedParams &p;
  __device__ long long operator()(const PagedDoc &d) const {
    if ((long long)d.lq * p.group > p.few_rows) return 0;
    constexpr int KT = few_stage_tokens(D);
    return (long long)p.hkv * few_item_cost((d.lk + KT - 1) / KT);
  }
};

// Tile kernel: one block of queries of a request: tokens [q0, q0 + ntok), one or two tiles, the key
// tiles that its rows see, its cost in (Q tile, key tile) pairs, kTileItem of them for the fixed costs
// of an item (its first loads, its rows written). From a graph, in us, for a cost of 1 / 2 / 5 / 10: 2 x
// 1500 first tokens 88.9 / 84.6 / 79.8 / 80.0, 8 chunks of 32 to 64 tokens over 500 to 2000 keys 33.0 /
// 32.7 / 30.9 / 32.0, 4 T5 chunks of 512 over 2048 to 4096 at head_dim 64 70.2 / 67.7 / 66.6 / 67.5.
constexpr int kTileItem = 5;
struct TileBlock {
  int q0, ntok, nkv, tiles, cost;
};
__device__ __forceinline__ TileBlock tile_block(const PagedDoc &d, int b, int tq, int blk,
                                                int causal) {
  TileBlock t;
  t.q0 = b * blk;
  t.ntok = min(d.lq - t.q0, blk);
  t.tiles = t.ntok > tq ? 2 : 1;
  t.nkv = (d.lk + 127) >> 7;
  if (causal) {
    const int last = d.lk - d.lq + t.q0 + t.ntok - 1;  // key position of the last row
    t.nkv = last < 0 ? 0 : min(t.nkv, (last >> 7) + 1);
  }
  t.cost = kTileItem + t.tiles * t.nkv;
  return t;
}
__device__ __forceinline__ long long tile_head_cost(const PagedDoc &d, int tq, int blk,
                                                    int causal) {
  long long c = 0;
  for (int b = 0; b * blk < d.lq; ++b) c += tile_block(d, b, tq, blk, causal).cost;
  return c;
}
struct TileCost {
  const PagedParams &p;
  int tq, blk;  // tokens per tile and per block
  __device__ long long operator()(const PagedDoc &d) const {
    return (long long)d.lq * p.group <= p.few_rows ? 0
                                                   : p.hkv * tile_head_cost(d, tq, blk, p.causal);
  }
};

// SMs n of the tile kernel when a call launches both kernels, so that they end together: with its
// total a and the other's b in stages of the few-row kernel (a pair of tiles weighs kPairStages:
// 0.96 us against 0.11 us of an SM at head_dim 128, measured) and its start longer by kStartStages,
// kStartStages + a / n = b / (sms - n). Each kernel has at least one SM. From a graph, in us: 24 decode
// steps beside a chunk of 384 tokens, 300 .. 6000 keys, 57 where shares in proportion to the totals alone
// gave 62. At head_dim 64, for a pair's weight of 3 / 5 / 8: 40 requests of 1 to 256 tokens with T5 bias
// 39.7 / 38.6 / 39.6, 48 of 1 to 768 tokens over 500 to 8000 keys 136 / 125 / 117.
constexpr float kPairStages = 9.f, kPairStages64 = 5.f, kStartStages = 80.f;
template <int D>
__device__ __forceinline__ int tile_sms(const PagedParams &p, long long tile_total,
                                        long long few_total) {
  if (!p.both || few_total == 0) return p.sms;
  if (tile_total == 0) return 0;
  const float a = (D == 128 ? kPairStages : kPairStages64) * (float)tile_total;
  const float N = (float)p.sms, c = kStartStages * N - a - (float)few_total;
  const float n = 2.f * a * N / (sqrtf(c * c + 4.f * kStartStages * a * N) - c);
  return min(max((int)(n + 0.5f), 1), p.sms - 1);
}

// ---- partial rows -------------------------------------------------------------------------------
// Per CTA: two records (part 0: its first item, begun by an earlier CTA; part 1: its last item,
// begun here and continued by the next CTA), then for each record [D / 4][rows][4] unnormalised rows
// (four channels of consecutive rows side by side: the threads that write and merge them hold a row
// each, and their 16-byte accesses line up) and [rows][2] (maximum in log2 units, sum).
struct PartRecord {
  int valid;   // this part exists
  int ends;    // the item ends in this CTA
  int row0;    // first row of q and out of the item's block (token), and its key/value head
  int hk;
  int rows;    // packed rows (token-major, the group's heads inside)
  int pos;     // tree kernel: which part of how many
  int parts;
  int pad;
};
__host__ __device__ inline size_t part_records_floats(int ctas) {
  return (size_t)ctas * 2 * sizeof(PartRecord) / 4;
}
__host__ __device__ inline size_t part_floats(int ctas, int rows, int d) {
  return part_records_floats(ctas) + (size_t)ctas * 2 * rows * (d + 2);
}
__device__ __forceinline__ PartRecord *part_record(float *part, int cta, int which) {
  return reinterpret_cast<PartRecord *>(part) + cta * 2 + which;
}
template <int ROWS, int D>
__device__ __forceinline__ float *part_rows(float *part, int ctas, int cta, int which) {
  return part + part_records_floats(ctas) + (size_t)(cta * 2 + which) * ROWS * D;
}
// channels 4 c4 .. 4 c4 + 3 of a row
template <int ROWS>
__device__ __forceinline__ float4 *part_quad(float *rows, int row, int c4) {
  return reinterpret_cast<float4 *>(rows) + (size_t)c4 * ROWS + row;
}
template <int ROWS, int D>
__device__ __forceinline__ float *part_stats(float *part, int ctas, int cta, int which) {
  return part + part_records_floats(ctas) + (size_t)ctas * 2 * ROWS * D +
         (size_t)(cta * 2 + which) * ROWS * 2;
}

// ---- this CTA's stretch -------------------------------------------------------------------------
constexpr int kShareDocs = 64;  // requests staged in shared memory from the stretch's first on

struct Share {
  long long lo, hi;  // this CTA's stretch; lo >= hi: none
  int doc;           // the request in which it begins
  long long off;     // cost of that request before lo
};

// Scratch of share_find, and the staged requests.
template <int NT>
struct ShareSmem {
  long long wsum[NT / 32 + 1];
  long long off;
  int doc;
  int sq[kShareDocs], lq[kShareDocs], lk[kShareDocs];
};

// a / b for a >= 0: by a 32-bit division wherever a has 32 bits (the 64-bit one is a long routine).
__device__ __forceinline__ long long div_small(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

template <int NT>
__device__ __forceinline__ long long share_scan(long long v, ShareSmem<NT> &s, long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  __syncthreads();
  if (lane == 31) s.wsum[warp] = inc;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += s.wsum[w];
    all += s.wsum[w];
  }
  *total = all;
  return before + inc - v;
}

// Find this CTA's stretch (all NT threads of the block; cost(doc) is the request's cost in this
// kernel, other(doc) in the other one, 0 for requests that are not theirs; ctas(total, other total)
// is the number of CTAs that share the line), report corrupt requests once, stage the requests the
// stretch may hold. Up to NT requests, one per thread, are read once; more are read again to find
// the stretch's first.
template <int NT, bool TREE, typename CostFn, typename OtherFn, typename CtasFn>
__device__ __forceinline__ Share share_find(const PagedParams &p, int min_share, const CostFn &cost,
                                            const OtherFn &other, CtasFn ctas, ShareSmem<NT> &s) {
  const int tid = threadIdx.x;
  const bool small = p.n <= NT;
  Share r;
  PagedDoc d{0, 0, 0, false};
  if (tid < p.n) d = paged_doc<TREE>(p, tid);
  long long first, total, before, other_total = 0;
  if (p.both) {
    long long mine = d.ok && d.lq > 0 ? other(d) : 0;
    for (int i = tid + NT; i < p.n; i += NT) {
      const PagedDoc e = paged_doc<TREE>(p, i);
      if (e.ok && e.lq > 0) mine += other(e);
    }
    share_scan<NT>(mine, s, &other_total);
  }
  first = d.ok && d.lq > 0 ? cost(d) : 0;
  {
    long long mine = first;
    for (int i = tid + NT; i < p.n; i += NT) {
      const PagedDoc e = paged_doc<TREE>(p, i);
      if (!e.ok && blockIdx.x == 0) atomicOr(p.err, FAT_DEVERR_SEQLENS);
      if (e.ok && e.lq > 0) mine += cost(e);
    }
    before = share_scan<NT>(small ? first : mine, s, &total);
  }
  const int G = ctas(total, other_total);
  if (tid < p.n && !d.ok && blockIdx.x == 0) atomicOr(p.err, FAT_DEVERR_SEQLENS);
  r.lo = r.hi = r.off = 0;
  r.doc = 0;
  if ((int)blockIdx.x >= G || total == 0) return r;
  const long long share = max(div_small(total + G - 1, G), (long long)min_share);
  r.lo = blockIdx.x * share;
  r.hi = min(total, r.lo + share);
  if (r.lo >= r.hi) return r;
  if (small) {
    if (r.lo >= before && r.lo < before + first) {
      s.doc = tid;
      s.off = r.lo - before;
    }
    __syncthreads();
    const int i = tid - s.doc;
    if (i >= 0 && i < kShareDocs) {
      s.sq[i] = d.sq;
      s.lq[i] = d.ok ? d.lq : 0;
      s.lk[i] = d.lk;
    }
  } else {
    long long base = 0;
    for (int i0 = 0;; i0 += NT) {  // the stretch begins in one of the requests: this ends
      long long c = 0, chunk;
      if (i0 + tid < p.n) {
        const PagedDoc e = paged_doc<TREE>(p, i0 + tid);
        c = e.ok && e.lq > 0 ? cost(e) : 0;
      }
      before = share_scan<NT>(c, s, &chunk);
      if (r.lo >= base + before && r.lo < base + before + c) {
        s.doc = i0 + tid;
        s.off = r.lo - (base + before);
      }
      base += chunk;
      if (r.lo < base || i0 + NT >= p.n) break;  // the same for every thread
    }
    __syncthreads();
    for (int i = tid; i < kShareDocs; i += NT) {
      PagedDoc e{0, 0, 0, false};
      if (s.doc + i < p.n) e = paged_doc<TREE>(p, s.doc + i);
      s.sq[i] = e.sq;
      s.lq[i] = e.ok ? e.lq : 0;
      s.lk[i] = e.lk;
    }
  }
  __syncthreads();
  r.doc = s.doc;
  r.off = s.off;
  return r;
}

template <bool TREE, int NT>
__device__ __forceinline__ PagedDoc share_doc(const PagedParams &p, const ShareSmem<NT> &s,
                                              int first_doc, int doc) {
  const int i = doc - first_doc;
  if (i < kShareDocs) return PagedDoc{s.sq[i], s.lq[i], s.lk[i], s.lq[i] > 0};
  PagedDoc d = paged_doc<TREE>(p, doc);
  d.ok = d.ok && d.lq > 0;
  return d;
}

// ---- launchers ----------------------------------------------------------------------------------
constexpr int kFewRows = 16;  // rows of the few-row kernel's items
int paged_few_ctas();
constexpr int kTileRows = 256;  // packed rows of the tile kernel's items, at most
int paged_tile_ctas();
// Whether items are cut: contexts of at most so many keys (the few-row kernel's: stages) are computed by
// one CTA each, which costs less than the merge grid. Whole against cut, in us:
//   few rows, head_dim 64, 12 heads: 500 keys 7.4 / 8.2 (16 requests 8.2 / 11.0), 1000 keys 10.3 / 8.9;
//   head_dim 128, 8 requests, 32 heads over 8: 250 keys 9.3 / 10.4, 500 keys 12.2 / 11.5;
//   chunks of 64 tokens, 32 heads over 8: 1000 keys 23.3 / 24.5 (32 chunks, head_dim 64: 38 / 43), 2000
//   keys 37.2 / 28.2.
// A call that launches both kernels goes by the tile kernel's figure for both of them.
constexpr int kWholeStages = 24, kWholeKeys = 1024;
int launch_paged_few(const PagedParams &p, const fat_paged_cache_t &c, cudaStream_t stream);
int launch_paged_tile(const PagedParams &p, const fat_paged_cache_t &c, cudaStream_t stream);
// Trees: items of `rows` (64 or 128) rows.
int launch_paged_mid(const PagedParams &p, const fat_paged_cache_t &c, int rows, cudaStream_t stream);

}  // namespace fat
