// fat_paged_tile.cu -- attention over a paged cache for requests with more rows than the few-row
// kernel takes: chunks of a prompt, drafted tokens of large groups.
//
// Rows are packed: the group's heads of a query lie side by side (row = token * group + head), so
// every key/value tile is read once for all heads of its group, and a chunk of a few tokens fills a
// tile. An item is (request, key/value head, up to two tiles of floor(128 / group) tokens); one
// persistent CTA per SM takes an equal share of all key tiles (fat_paged.cuh) and walks its items:
//   warps 0-7   two softmax warpgroups, one row per thread (a TMEM lane): logits, bias, mask, running
//               maximum (moved only when it grows by more than 2^32), P as bf16 into tensor memory;
//   warp 8      producer: Q by one TMA box per 64 channels ([tokens][group heads]), K and V tiles of
//               128 tokens page by page (a lane per page, its number fetched a tile ahead);
//   warps 9-10  MMA issuers, one per softmax warpgroup: S = Q K^T, O += P V (tcgen05, TMEM);
//   warp 11     values behind a request's last key are zeroed in its last tile (a page may hold
//               anything there, and 0 * NaN is NaN).
// An item of two tiles gives each warpgroup its own rows, both over every key tile (the copies are
// shared, one warpgroup's softmax overlaps the other's products). An item of one tile gives both the
// same rows and every other key tile each, and adds the two results at the end through tensor
// memory: a short chunk over a long context keeps both busy as well.
// Key tiles go from the last one backwards: the first holds each row's largest linear bias, so the
// maximum rarely moves afterwards.
//
// Bound by the softmax warpgroups' own work (head_dim 128: 0.74 us of each half of 64 keys, and 0.22 us
// between two halves; the tensor pipe is busy half of the time): a chunk of 2048 tokens over 18432 keys,
// 16 heads over 8, in 252 us (1165 TFLOP/s, 0.60 of the measured peak).
// A call's first steps are slow (the first copies, and instructions that come from L2 a line at a
// time): a block's first step begins 5 to 7 us after the block, the second 6 to 11 us later where other
// kernels ran before (4 to 7 behind the same call), the third 3 to 6 (2 to 3), from then on one every
// 1.7 to 1.9.
// P is rounded to bf16, the operand type that P V shares with V, as in the packed forward: an error of
// 2^-8 of a row's sum of |weight x value| at most (relative to 64 bits 0.0022 in all, the output's own
// rounding 0.0017). The second bf16 part that the few-row kernel adds would take half as many products
// again and tensor memory that head_dim 128 does not have.
#include <algorithm>
#include <cstdint>

#include "fat_paged.cuh"

namespace fat {
namespace {

constexpr int kThreads = 384;
constexpr int kWarpProd = 8, kWarpMma = 9, kWarpTail = 11;
constexpr int kMinShare = 4;  // cost units (a key tile of one Q tile) a CTA takes at least

struct TileItem {
  int doc, hk, row0;      // row0: token of q and out
  int q0, ntok, tiles;    // tokens of the request, tiles (0: the end of the list)
  int lk, shift;          // shift: key position of the request's first query
  int j0, j1;             // key tiles taken here: key tile nkv - 1 - j for j in [j0, j1)
  int nkv;
  int begins, ends;
};
// The producer walks the share and hands its items to the other roles through this ring.
constexpr int kItems = 4;
template <int D>
struct TileCfg {
  static constexpr int DB = D / 64;
  static constexpr int BLK = 128 * 128;    // 128 rows x 64 bf16
  static constexpr int TILE = DB * BLK;
  static constexpr int NS = D == 64 ? 4 : 2;  // K and V stages (a power of two)
  static constexpr int NS_LOG2 = D == 64 ? 2 : 1;
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = OFF_K + NS * TILE;
  static constexpr int OFF_BAR = OFF_V + NS * TILE;
  static constexpr int OFF_STATS = OFF_BAR + 512;            // float2 [128]
  static constexpr int OFF_ITEMS = OFF_STATS + 1024;
  static constexpr int OFF_SHARE = OFF_ITEMS + ((kItems * (int)sizeof(TileItem) + 15) & ~15);
  static constexpr int OFF_THR = OFF_SHARE + (int)sizeof(ShareSmem<kThreads>);
  static constexpr int OFF_ROWS = (OFF_THR + kMaxThresholds * 4 + 127) & ~127;  // 2 KB per softmax warp
  static constexpr int OFF_LUT = OFF_ROWS + 8 * 2048;
  static_assert((2 + 4 * NS + 20 + 2 * kItems) * 8 + 8 <= 448, "barrier block");
  static_assert(OFF_LUT + kMaxBiasSpan + 512 + 1024 <= kSmemLimit, "shared memory");
  static constexpr int REG_SM = 224, REG_OTHER = 56;
  static constexpr int REGS_NEEDED = 256 * REG_SM + 128 * REG_OTHER;
  static_assert(REGS_NEEDED <= kThreads * ((65536 / kThreads) & ~7), "register split");
  // TMEM columns: S_t at 128 t, O_t behind them.
  // d 64: P_t has columns of its own, so that the next S_t is computed while P_t is still read.
  // d 128: there is no room for that. S_t comes in two halves of 64 keys: step g of a tile has its
  // first 64 keys' S in half g % 2 and the others' in the other half; P of both (bf16 pairs, 64
  // columns) is written over the first. The second half is free again once it has been read, so the
  // next step's first S is computed before this step's P V is complete, and the warpgroup finds it when
  // it comes back; P V of the first half runs beside the second half's softmax (1.92 us a step of two
  // tiles; 2.07 with P V in one, 2.75 with S whole). With d 64 the halves' own costs are
  // higher than what they save (106 us against 91 on 2 x 1024 queries over 8192 keys, 16 heads).
  static constexpr bool SEP_P = D == 64;
  static constexpr int SCOLS = SEP_P ? 128 : 64;  // columns of S that are computed and read at once
  static constexpr uint32_t COL_O = 256, O_STRIDE = D;
  static constexpr uint32_t COL_P = COL_O + 2 * O_STRIDE;
  static constexpr uint32_t TMEM_COLS = 512;
  static_assert(COL_P + (SEP_P ? 128 : 0) <= TMEM_COLS, "TMEM column budget");
  static constexpr uint32_t IDESC_S = idesc_bf16_f32(128, SCOLS, 0, 0);
  static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, 0, 1);
};

struct TileWalk {
  const PagedParams &p;
  const ShareSmem<kThreads> &sm;
  int tq, blk, first_doc, doc, hk, b;
  long long left;
  int off;
  __device__ TileWalk(const PagedParams &pp, const ShareSmem<kThreads> &s, const TileCost &c,
                      const Share &sh)
      : p(pp), sm(s), tq(c.tq), blk(c.blk), first_doc(sh.doc), doc(sh.doc), b(0),
        left(sh.hi - sh.lo) {
    const PagedDoc d = share_doc(p, sm, doc, doc);
    const long long per = tile_head_cost(d, tq, blk, p.causal);
    hk = (int)div_small(sh.off, per);
    long long rest = sh.off - hk * per;
    for (int c; rest >= (c = tile_block(d, b, tq, blk, p.causal).cost); rest -= c) ++b;
    off = (int)rest;
  }
  __device__ bool next(TileItem &it) {
    while (left > 0 && doc < p.n) {
      const PagedDoc d = share_doc(p, sm, first_doc, doc);
      if (!d.ok || (long long)d.lq * p.group <= p.few_rows) {
        ++doc;
        hk = b = 0;
        continue;
      }
      const TileBlock t = tile_block(d, b, tq, blk, p.causal);
      const int o = off;
      off = 0;
      const int take = (int)min(left, (long long)(t.cost - o));
      left -= take;
      it.doc = doc;
      it.hk = hk;
      it.row0 = d.sq + t.q0;
      it.q0 = t.q0;
      it.ntok = t.ntok;
      it.tiles = t.tiles;
      it.lk = d.lk;
      it.shift = d.lk - d.lq;
      it.nkv = t.nkv;
      ++b;
      if (b * blk >= d.lq) {
        b = 0;
        if (++hk == p.hkv) {
          hk = 0;
          ++doc;
        }
      }
      if (!p.split) {  // whole items: the one that begins earlier is another CTA's
        if (o > 0) continue;
        it.j0 = 0;
        it.j1 = t.nkv;
        it.begins = it.ends = true;
        return true;
      }
      // the fixed part of the cost comes first, before the key tiles
      it.j0 = (max(o - kTileItem, 0) + t.tiles - 1) / t.tiles;
      it.j1 = (max(o + take - kTileItem, 0) + t.tiles - 1) / t.tiles;
      it.begins = it.j0 == 0;
      it.ends = o + take == t.cost;
      if (it.j0 == it.j1 && !(t.nkv == 0 && it.ends)) continue;  // no key tile of it lies here
      it.ends = it.j1 == t.nkv;
      return true;
    }
    return false;
  }
};
// Positions j0 + first, j0 + first + step, ... of an item that Q tile t multiplies: both tiles every
// one, or (a single tile, shared) alternating.
__device__ __forceinline__ int item_first(const TileItem &it, int t) { return it.tiles == 2 ? 0 : t; }
__device__ __forceinline__ int item_step(const TileItem &it) { return it.tiles == 2 ? 1 : 2; }
__device__ __forceinline__ int item_count(const TileItem &it, int t) {
  const int n = it.j1 - it.j0;
  return it.tiles == 2 ? n : (n + 1 - t) >> 1;
}

// COLS columns of the S row turned into logits where they stand: scale, bias and mask (columns from
// lim on), chunk by chunk in a rolled loop. For the few tiles near the diagonal (and, with d 64, those
// that the mask cuts): they pay a second pass over tensor memory rather than a variant of the whole
// softmax code, of which a call's first use of 6 KB costs 3 us of instruction fetches.
//   NEAR: bias = table[lut[j]] - slope |delta0 + j|;  else rowc + kk * j.
template <int COLS, bool NEAR>
__device__ __forceinline__ void tile_edge(uint32_t tS, float scale_log2, float rowc, float kk,
                                          const uint8_t *lut, const float *tab, int tab_stride,
                                          float slope, int delta0, int lim) {
#pragma unroll 1
  for (int c = 0; c < COLS; c += 32) {
    uint32_t x[32];
    tmem_ld32(tS + c, x);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float b;
      if (NEAR) {
        b = -slope * fabsf((float)(delta0 + c + i));
        if (tab != nullptr) b = fmaf(__ldg(tab + lut[c + i] * tab_stride), kLog2e, b);
      } else {
        b = fmaf(kk, (float)(c + i), rowc);
      }
      const float v = fmaf(__uint_as_float(x[i]), scale_log2, b);
      x[i] = __float_as_uint(c + i < lim ? v : -INFINITY);
    }
    tmem_st32(tS + c, x);
  }
  tmem_st_wait();
}

// 32 CHUNKS columns of the S row from tensor memory as logits x (log2 units):
// S * scale + rowc + kk * j, columns from lim on masked; returns the row's maximum.
template <int CHUNKS, bool LINEAR, bool MASK>
__device__ __forceinline__ float tile_logits(uint32_t tS, uint32_t (&x)[CHUNKS][32],
                                             float scale_log2, float rowc, float kk, int lim) {
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) tmem_ld32_issue(tS + c * 32, x[c]);
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) tmem_ld32_fence(x[c]);
  const uint64_t sl2 = f2_pack(scale_log2, scale_log2);
  const uint64_t rc2 = f2_pack(rowc, rowc);
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const int j = c * 32 + i;
      const uint64_t b2 =
          LINEAR ? f2_pack(fmaf(kk, (float)j, rowc), fmaf(kk, (float)(j + 1), rowc)) : rc2;
      float v0, v1;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1])), sl2, b2),
                v0, v1);
      if (MASK) {
        v0 = (j < lim) ? v0 : -INFINITY;
        v1 = (j + 1 < lim) ? v1 : -INFINITY;
      }
      x[c][i] = __float_as_uint(v0);
      x[c][i + 1] = __float_as_uint(v1);
      mx[(i >> 1) & 3] = fmax3(mx[(i >> 1) & 3], v0, v1);
    }
  }
  return fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
}

// P = 2^(x - sub) of those columns as bf16 pairs into tensor memory, with their fp32 sum.
template <int CHUNKS, bool SUB>
__device__ __forceinline__ void tile_exp(const uint32_t (&x)[CHUNKS][32], uint64_t sub2, uint32_t tP,
                                         uint64_t (&sum2)[4]) {
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float a = __uint_as_float(x[c][2 * i]), b = __uint_as_float(x[c][2 * i + 1]);
      if (SUB) f2_unpack(f2_sub(f2_pack(a, b), sub2), a, b);
      a = ex2(a);
      b = ex2(b);
      pk[i] = pack_bf16x2(a, b);
      sum2[i & 3] = f2_add(sum2[i & 3], f2_pack(a, b));
    }
    tmem_st16(tP + c * 16, pk);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    fat_paged_tile_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v,
                          const __grid_constant__ PagedParams p) {
  using C = TileCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.group, tq = 128 / G, RT = tq * G;  // tokens and rows of a tile
  uint8_t *sQ = sm, *sK = sm + C::OFF_K, *sV = sm + C::OFF_V;
  auto &share_s = *reinterpret_cast<ShareSmem<kThreads> *>(sm + C::OFF_SHARE);
  uint64_t *q_full = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR);
  uint64_t *q_empty = q_full + 1;
  uint64_t *k_full = q_empty + 1;
  uint64_t *v_full = k_full + C::NS;
  uint64_t *k_empty = v_full + C::NS;
  uint64_t *v_empty = k_empty + C::NS;
  uint64_t *s_full = v_empty + C::NS;  // [tile][half]
  uint64_t *p_ready = s_full + 4;      // [tile][half]
  uint64_t *o_half = p_ready + 4;      // [2] each from here on; d 128: the first half's P V is complete
  uint64_t *o_ready = o_half + 2;
  uint64_t *s_read = o_ready + 2;  // S (d 128: the step's second half of it) has been read
  uint64_t *o_free = s_read + 2;
  uint64_t *mma_done = o_free + 2;
  uint64_t *merge_ready = mma_done + 2;
  uint64_t *tail = merge_ready + 1;  // a last tile's values have arrived (before they are zeroed)
  uint64_t *item_full = tail + 1;    // [kItems] each
  uint64_t *item_empty = item_full + kItems;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(item_empty + kItems);
  TileItem *items = reinterpret_cast<TileItem *>(sm + C::OFF_ITEMS);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  Watchdog *wdp = reinterpret_cast<Watchdog *>(sm + C::OFF_BAR + 448);
  int *thr_s = reinterpret_cast<int *>(sm + C::OFF_THR);
  uint8_t *lut = sm + C::OFF_LUT;
  grid_dep_wait();
  grid_dep_launch();  // the few-row kernel may start: what this call reads is complete
  if (p.split && tid < 2) part_record(p.part, blockIdx.x, tid)->valid = 0;
  for (int i = tid; i < p.bias.n_thr; i += kThreads) thr_s[i] = p.bias.thr[i];
  const TileCost cost{p, tq, 2 * tq};
  const Share share = share_find<kThreads>(
      p, kMinShare, cost, FewCost<D>{p},
      [&](long long mine, long long other) { return tile_sms<D>(p, mine, other); }, share_s);
  if (share.lo >= share.hi) return;

  if (warp == kWarpProd && lane == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);  // one release per issuer and item
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(v_full + s, 1);
      mbar_init(k_empty + s, 2);  // two commits: one per issuer, or both by the one that used it
      mbar_init(v_empty + s, 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full + 2 * t, 1);
      mbar_init(s_full + 2 * t + 1, 1);
      mbar_init(p_ready + 2 * t, 128);
      mbar_init(p_ready + 2 * t + 1, 128);
      mbar_init(o_half + t, 1);
      mbar_init(o_ready + t, 1);
      mbar_init(s_read + t, 128);
      mbar_init(o_free + t, 128);
      mbar_init(mma_done + t, 1);
    }
    mbar_init(merge_ready, 128);
    mbar_init(tail, 1);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(item_full + i, 1);
      mbar_init(item_empty + i, 11);  // eight softmax warps, two issuers, the tail warp
    }
    *abort_flag = 0;
    *wdp = Watchdog{abort_flag, p.err, FAT_DEVERR_TIMEOUT_FWD, p.timeout_ns};
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  // rows of the Q tiles that no token fills (group does not divide 128): zeros, never overwritten
  for (int i = tid; i < 2 * C::DB * (128 - RT) * 8; i += kThreads) {
    const int blk = i / ((128 - RT) * 8), rest = i % ((128 - RT) * 8);
    *reinterpret_cast<uint4 *>(sQ + blk * C::BLK + RT * 128 + rest * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  if (p.bias.table != nullptr)
    for (int i = tid; i < p.bias.lut_len; i += kThreads)
      lut[i] = (uint8_t)t5_bucket_staged(p.bias.lut_lo + i, p.bias, thr_s);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Watchdog &wd = *wdp;
  if (warp >= kWarpProd) regs_dec<C::REG_OTHER>();
  // item i of the list, for the roles that read it (a whole warp, or the issuers' threads alone)
  auto item_wait = [&](int i) {
    return mbar_wait(item_full + (i & (kItems - 1)), (i / kItems) & 1, wd);
  };
  auto item_done = [&](int i) { mbar_arrive(item_empty + (i & (kItems - 1))); };

  if (warp == kWarpProd) {
    // ------------------------------------------------------------------ producer
    const int kbox = min(128, 1 << p.log2_page), pieces = 128 / kbox;
    TileWalk walk(p, share_s, cost, share);
    TileItem it;
    uint32_t J = 0;      // K/V stream position
    int ni = 0;          // items with keys
    uint32_t last_tail = 0;
    bool any_tail = false, ok = !(p.debug_flags & 1);  // test hook: no copies, the waits run out
    for (int i = 0; ok; ++i) {
      const bool last = !walk.next(it);
      if (i >= kItems) {
        ok = warp_wait(item_empty + (i & (kItems - 1)), (i / kItems - 1) & 1, wd);
        if (!ok) break;
      }
      if (last) it.tiles = 0;
      if (lane == 0) {
        items[i & (kItems - 1)] = it;
        mbar_arrive(item_full + (i & (kItems - 1)));
      }
      if (last) break;
      const int n = it.j1 - it.j0;
      if (n == 0) continue;
      // this lane's page of key tile kt (the next one's is fetched while this one's copies go out)
      auto fetch = [&](int kt) -> int {
        const int tok = kt * 128 + lane * kbox;
        return (lane < pieces && tok < it.lk)
                   ? __ldg(p.table + (size_t)it.doc * p.width + (tok >> p.log2_page))
                   : 0;
      };
      int kt = it.nkv - 1 - it.j0;
      int page = fetch(kt);
      // The item's Q. It is free once both issuers have released it, which also means that every K
      // tile of the items before has been used. Their V tiles have arrived too before Q is loaded:
      // an issuer that finds Q full then knows every stage's phases of earlier items to be over,
      // also of stages that only the other one used, and tells the phases of its own by their parity.
      auto load_q = [&](uint32_t before) {  // before: K/V positions of earlier items
        if (ni > 0) ok = warp_wait(q_empty, (ni - 1) & 1, wd);
        for (uint32_t k = 1; ok && k <= min(before, (uint32_t)C::NS); ++k)
          ok = warp_wait(v_full + ((before - k) & (C::NS - 1)), ((before - k) >> C::NS_LOG2) & 1, wd);
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(q_full, (uint32_t)RT * 128 * C::DB * it.tiles);
          for (int t = 0; t < it.tiles; ++t)
            for (int b = 0; b < C::DB; ++b)
              tma_load_3d(&tm_q, q_full, sQ + t * C::TILE + b * C::BLK, 64 * b, it.hk * G,
                          it.row0 + t * tq);
        }
        ++ni;
      };
      // With two stages (d 128) the first K would only wait as well; with four it is loaded first.
      if (C::NS == 2) load_q(J);
      if (!ok) break;
      for (int jj = 0; jj < n; ++jj, --kt, ++J) {
        const int s = J & (C::NS - 1);
        const uint32_t u = J >> C::NS_LOG2;
        const int tok = kt * 128 + lane * kbox;
        const int nvalid = min(pieces, (it.lk - kt * 128 + kbox - 1) / kbox);
        const bool issue = lane < nvalid;
        if (issue && (unsigned)page >= (unsigned)p.num_pages) {
          atomicOr(p.err, FAT_DEVERR_PAGES);
          page = p.num_pages;  // just outside: filled with zeros
        }
        const int in = tok & ((1 << p.log2_page) - 1);
        const int c1 = p.head_outer ? in : it.hk, c2 = p.head_outer ? it.hk : in;
        const int cur = page;
        if (jj + 1 < n) page = fetch(kt - 1);
        const uint32_t bytes = (uint32_t)nvalid * kbox * 128 * C::DB;
        if (u > 0 && !(ok = warp_wait(k_empty + s, (u - 1) & 1, wd))) break;
        if (lane == 0) mbar_arrive_expect_tx(k_full + s, bytes);
        __syncwarp();
        if (issue)
          for (int b = 0; b < C::DB; ++b)
            tma_load_4d(&tm_k, k_full + s, sK + s * C::TILE + b * C::BLK + lane * kbox * 128, 64 * b,
                        c1, c2, cur);
        if (C::NS > 2 && jj == 0) {
          load_q(J);
          if (!ok) break;
        }
        if (u > 0 && !(ok = warp_wait(v_empty + s, (u - 1) & 1, wd))) break;
        // a request's last tile: its values complete on `tail`, and warp 11 arrives on v_full
        uint64_t *vbar = v_full + s;
        if (kt * 128 + 128 > it.lk) {
          if (any_tail && J - last_tail < (uint32_t)C::NS) {  // the one before has been passed on
            const uint32_t sl = last_tail & (C::NS - 1), ul = last_tail >> C::NS_LOG2;
            if (!(ok = warp_wait(v_full + sl, ul & 1, wd))) break;
          }
          any_tail = true;
          last_tail = J;
          vbar = tail;
        }
        if (lane == 0) mbar_arrive_expect_tx(vbar, bytes);
        __syncwarp();
        if (issue)
          for (int b = 0; b < C::DB; ++b)
            tma_load_4d(&tm_v, vbar, sV + s * C::TILE + b * C::BLK + lane * kbox * 128, 64 * b, c1,
                        c2, cur);
      }
      if (!ok) break;
    }
    // After a wait ran out, copies may still be on their way: give them time to land before the
    // block exits (a stage's barrier alone does not tell which of its phases they belong to).
    if (*abort_flag) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
  } else if (warp == kWarpMma || warp == kWarpMma + 1) {
    // ------------------------------------------------------------------ MMA issuers
    const int t = warp - kWarpMma;
    if (lane == 0) {
      const uint32_t dS = tmem + 128 * t, dO = tmem + C::COL_O + C::O_STRIDE * t;
      const uint64_t dKd = sw128_desc(smem_u32(sK), 16, 1024);
      const uint64_t dVd = sw128_desc(smem_u32(sV), C::BLK, 1024);
      uint32_t J = 0, g = 0;  // stream position, this tile's steps
      int ni = 0, act = 0;    // items with keys, those in which this tile has steps
      bool ok = true;
      for (int i = 0; ok; ++i) {
        if (!(ok = item_wait(i))) break;
        const TileItem it = items[i & (kItems - 1)];
        item_done(i);
        if (it.tiles == 0) break;
        const int n = it.j1 - it.j0;
        if (n == 0) continue;
        const int first = item_first(it, t), step = item_step(it);
        if (first >= n) {  // one key tile: the other issuer's; Q is released without being used
          if (!(ok = mbar_wait(q_full, ni & 1, wd))) break;
          mbar_arrive(q_empty);
          J += n;
          ++ni;
          continue;
        }
        const uint64_t dQd = sw128_desc(smem_u32(sQ) + (it.tiles == 2 ? t * C::TILE : 0), 16, 1024);
        const bool alone = it.tiles == 1;  // each stage is one tile's
        // S of keys SCOLS half .. of position jj, as step gs of this tile
        auto issue_S = [&](int jj, int half, uint32_t gs) {
          const int st = (J + jj) & (C::NS - 1);
          const uint64_t kd = dKd + ((st * C::TILE + half * 64 * 128) >> 4);
          const uint32_t d = C::SEP_P ? dS : dS + 64 * ((gs & 1) ^ half);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * C::BLK + (kk & 3) * 32) >> 4;
            mma_bf16_ss(d, dQd + off, kd + off, C::IDESC_S, kk > 0);
          }
          mma_commit(s_full + 2 * t + half);
          if (C::SEP_P || half == 1) {  // the key tile has been used
            mma_commit(k_empty + st);
            if (alone) mma_commit(k_empty + st);
            if (jj + step >= n) mma_commit(q_empty);  // and so has Q
          }
        };
        auto k_wait = [&](int jj) {
          return mbar_wait(k_full + ((J + jj) & (C::NS - 1)), ((J + jj) >> C::NS_LOG2) & 1, wd);
        };
        ok = mbar_wait(q_full, ni & 1, wd) && k_wait(first);
        if (!ok) break;
        tc_fence_after();
        issue_S(first, 0, g);
        if (!C::SEP_P) issue_S(first, 1, g);
        for (int jj = first; jj < n; jj += step, ++g) {
          const uint32_t jp = J + jj;
          const int s = jp & (C::NS - 1);
          const bool more = jj + step < n;
          const uint64_t vd = dVd + ((s * C::TILE) >> 4);
          const uint32_t aP = C::SEP_P ? tmem + C::COL_P + 64 * t : dS + 64 * (g & 1);
          // O += P V of keys 16 k0 .. 16 k1 - 1
          auto issue_PV = [&](int k0, int k1) {
#pragma unroll
            for (int kk = k0; kk < k1; ++kk)
              mma_bf16_ts(dO, aP + kk * 8, vd + ((kk * 2048) >> 4), C::IDESC_PV,
                          (jj > first || kk > 0) ? 1u : 0u);
          };
          // the first P V overwrites O: the previous item's rows have been read
          auto o_wait = [&]() {
            return jj > first || act == 0 || mbar_wait(o_free + t, (act - 1) & 1, wd);
          };
          auto v_wait = [&]() { return mbar_wait(v_full + s, (jp >> C::NS_LOG2) & 1, wd); };
          if constexpr (!C::SEP_P) {  // the first half's P V
            if (!(ok = v_wait() && mbar_wait(p_ready + 2 * t, g & 1, wd) && o_wait())) break;
            tc_fence_after();
            issue_PV(0, 4);
            mma_commit(o_half + t);
          }
          // the next step's S (d 128: its first half, where this step's second one has been read)
          if (!(ok = mbar_wait(s_read + t, g & 1, wd))) break;
          if (more) {
            if (!(ok = k_wait(jj + step))) break;
            tc_fence_after();
            issue_S(jj + step, 0, g + 1);
          }
          if constexpr (C::SEP_P) {
            if (!(ok = v_wait() && mbar_wait(p_ready + 2 * t, g & 1, wd) && o_wait())) break;
            tc_fence_after();
            issue_PV(0, 8);
          } else {
            if (!(ok = mbar_wait(p_ready + 2 * t + 1, g & 1, wd))) break;
            tc_fence_after();
            issue_PV(4, 8);
          }
          mma_commit(o_ready + t);
          mma_commit(v_empty + s);
          if (alone) mma_commit(v_empty + s);
          // the other half over P, which the products above have read
          if (!C::SEP_P && more) issue_S(jj + step, 1, g + 1);
        }
        J += n;
        ++ni;
        ++act;
      }
      mma_commit(mma_done + t);
      mbar_wait_teardown(mma_done + t, 0, kTeardownNs);
    }
  } else if (warp == kWarpTail) {
    // ------------------------------------------------------------------ values behind the last key
    uint32_t J = 0;
    int nt = 0;
    for (int i = 0;; ++i) {
      if (!__all_sync(0xffffffffu, item_wait(i))) break;
      const TileItem it = items[i & (kItems - 1)];
      __syncwarp();
      if (lane == 0) item_done(i);
      if (it.tiles == 0) break;
      const int n = it.j1 - it.j0;
      if (n == 0) continue;
      const int kt = it.nkv - 1 - it.j0;
      if (kt * 128 + 128 > it.lk) {  // only an item's first position can be the last tile
        if (!warp_wait(tail, nt & 1, wd)) break;
        ++nt;
        const int s = J & (C::NS - 1), row = it.lk - kt * 128;
        for (int b = 0; b < C::DB; ++b)
          for (int k = row * 8 + lane; k < 128 * 8; k += 32)
            *reinterpret_cast<uint4 *>(sV + s * C::TILE + b * C::BLK + k * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_full + s);
      }
      J += n;
    }
  } else {
    // ------------------------------------------------------------------ softmax warpgroups
    regs_inc<C::REG_SM>();
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + 128 * t;
    const uint32_t tO = tmem + lane_off + C::COL_O + C::O_STRIDE * t;
    float2 *stats = reinterpret_cast<float2 *>(sm + C::OFF_STATS);
    const uint32_t scratch = smem_u32(sm + C::OFF_ROWS) + warp * 2048;
    const int rq = r / G, rg = r - rq * G;  // token and head of this row within the tile
    const bool has_slopes = p.bias.slopes != nullptr, has_table = p.bias.table != nullptr;
    uint32_t g = 0, g_other = 0;  // steps of this tile and of the other one
    int merges = 0;
    bool ok = true;
    for (int n_item = 0;; ++n_item) {
      if (n_item > 0) {  // the item before is read no more
        __syncwarp();
        if (lane == 0) item_done(n_item - 1);
      }
      if (ok) ok = __all_sync(0xffffffffu, item_wait(n_item));
      if (!ok) break;
      const TileItem &it = items[n_item & (kItems - 1)];  // read where it is: registers are short
      if (it.tiles == 0) break;
      const int t_row = it.tiles == 2 ? t : 0;           // which tile's rows
      const int ntok = min(it.ntok - t_row * tq, tq);    // its tokens
      const bool valid = rq < ntok && r < RT;
      const int h = it.hk * G + rg;
      const int row = it.row0 + t_row * tq + rq;
      const bool whole = it.begins && it.ends;
      const int which = it.begins ? 1 : 0;
      if (!whole && r == 0 && t == 0) {
        PartRecord *rec = part_record(p.part, blockIdx.x, which);
        rec->valid = 1;
        rec->ends = it.ends;
        rec->row0 = it.row0;
        rec->hk = it.hk;
        rec->rows = it.ntok * G;
      }
      const int steps = item_count(it, t), steps_other = item_count(it, 1 - t);
      if (it.nkv == 0) {  // no key for any row
        if (valid && (it.tiles == 2 || t == 0)) {
          uint4 *dst = reinterpret_cast<uint4 *>(p.out + ((size_t)row * p.hq + h) * D);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse != nullptr) p.lse[(size_t)h * p.total_q + row] = -INFINITY;
        }
        continue;
      }
      // positions: of the tile's first and last row, and of this one (a row without a token: as
      // the last one's)
      const int pos_lo = it.shift + it.q0 + t_row * tq, pos_hi = pos_lo + ntok - 1;
      const int qpos = min(pos_lo + rq, pos_hi);
      const float slope = has_slopes ? __ldg(p.bias.slopes + h) * kLog2e : 0.f;
      const float *tab = has_table ? p.bias.table + h : nullptr;
      float c_pos = 0.f, c_neg = 0.f;
      if (has_table) {
        c_pos = __ldg(tab + lut[p.bias.sat_pos - p.bias.lut_lo] * p.hq) * kLog2e;
        c_neg = __ldg(tab + lut[-p.bias.sat_neg - p.bias.lut_lo] * p.hq) * kLog2e;
      }
      // m: the row's reference, which P is relative to. It is raised (and what was summed so far
      // scaled) only when the row's maximum grows beyond it by more than 2^32: every sum stays far
      // from fp32's and bf16's ends, and the result is exact.
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < steps && ok; ++i) {
        const uint32_t gi = g + i;
        const int jj = item_first(it, t) + i * item_step(it);
        const int ks = 128 * (it.nkv - 1 - it.j0 - jj);
        const bool need_mask = ks + 128 > it.lk || (p.causal && ks + 127 > pos_lo);
        const int lim = min(it.lk - ks, p.causal ? qpos - ks + 1 : 128);
        float rowc = 0.f, kk = 0.f;
        bool near = false;
        if (p.bias.has_bias) {
          const bool far_pos = ks - pos_hi >= p.bias.sat_pos;
          near = !far_pos && ks + 127 - pos_lo > -p.bias.sat_neg;
          kk = far_pos ? -slope : slope;
          rowc = fmaf(kk, (float)(ks - qpos), far_pos ? c_pos : c_neg);
        }
        uint64_t sum2[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) sum2[k] = f2_pack(0.f, 0.f);
        if constexpr (C::SEP_P) {
          const uint32_t tP = tmem + lane_off + C::COL_P + 64 * t;
          ok = warp_wait(s_full + 2 * t, gi & 1, wd);
          if (!ok) break;
          tc_fence_after();
          float scale = p.scale_log2;
          const bool edge = near || need_mask;
          if (edge) {
            const uint8_t *row_lut = lut + (ks - qpos - p.bias.lut_lo);
            if (near)
              tile_edge<128, true>(tS, scale, 0.f, 0.f, row_lut, tab, p.hq, slope, ks - qpos, lim);
            else
              tile_edge<128, false>(tS, scale, rowc, kk, row_lut, tab, p.hq, slope, ks - qpos, lim);
            scale = 1.f;
            rowc = 0.f;
          }
          uint32_t x[4][32];
          const float mx = (has_slopes && !edge)
                               ? tile_logits<4, true, false>(tS, x, scale, rowc, kk, 0)
                               : tile_logits<4, false, false>(tS, x, scale, rowc, 0.f, 0);
          tc_fence_before();
          mbar_arrive(s_read + t);  // S is in registers: the next one may be computed
          if (i == 0) {
            m = mx;
          } else {
            const bool fresh = m == -INFINITY;  // no key of this row so far
            const bool need = fresh ? mx != -INFINITY : mx > m + 32.0f;
            // P and O are still read by the previous P V
            ok = warp_wait(o_ready + t, (gi - 1) & 1, wd);
            if (!ok) break;
            tc_fence_after();
            if (__any_sync(0xffffffffu, need)) {
              const float f = need ? (fresh ? 0.f : ex2(m - mx)) : 1.0f;
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tO + c * 32, o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st32(tO + c * 32, o);
              }
              if (need) {
                l *= f;
                m = mx;
              }
            }
          }
          const float m_use = m == -INFINITY ? 0.f : m;
          tile_exp<4, true>(x, f2_pack(m_use, m_use), tP, sum2);
        } else {
          const uint32_t tP = tS + 64 * (gi & 1);
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            ok = warp_wait(s_full + 2 * t + half, gi & 1, wd);
            if (!ok) break;
            tc_fence_after();
            const uint32_t tH = tS + 64 * ((gi & 1) ^ half);
            const int c0 = 64 * half;
            const float m_ref = m == -INFINITY ? 0.f : m;
            uint32_t x[2][32];
            float mx;
            if (near) {
              tile_edge<64, true>(tH, p.scale_log2, 0.f, 0.f,
                                  lut + (ks + c0 - qpos - p.bias.lut_lo), tab, p.hq, slope,
                                  ks + c0 - qpos, lim - c0);
              mx = tile_logits<2, false, false>(tH, x, 1.f, -m_ref, 0.f, 0);
            } else {
              const float rc = fmaf(kk, (float)c0, rowc) - m_ref;
#define FAT_TILE_LOGITS(LINEAR, MASK) \
  tile_logits<2, LINEAR, MASK>(tH, x, p.scale_log2, rc, kk, lim - c0)
              if (has_slopes)
                mx = need_mask ? FAT_TILE_LOGITS(true, true) : FAT_TILE_LOGITS(true, false);
              else
                mx = need_mask ? FAT_TILE_LOGITS(false, true) : FAT_TILE_LOGITS(false, false);
#undef FAT_TILE_LOGITS
            }
            if (half == 1) {  // it is in registers: the next S may be computed there
              tc_fence_before();
              mbar_arrive(s_read + t);
            }
            float sub = 0.f;  // what the exponentials still subtract
            bool need = false;
            if (m == -INFINITY) {  // no key of this row so far: what was summed is zero
              if (mx != -INFINITY) m = sub = mx;
            } else {
              need = mx > 32.f;
            }
            if (__any_sync(0xffffffffu, need)) {
              const float f = need ? ex2(-mx) : 1.f;
              if (i + half > 0) {  // O, once the products so far are complete
                ok = half == 0 ? warp_wait(o_ready + t, (gi - 1) & 1, wd)
                               : warp_wait(o_half + t, gi & 1, wd);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                  uint32_t o[32];
                  tmem_ld32(tO + c, o);
#pragma unroll
                  for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                  tmem_st32(tO + c, o);
                }
              }
              l *= f;
#pragma unroll
              for (int k = 0; k < 4; ++k) sum2[k] = f2_mul(sum2[k], f2_pack(f, f));
              if (need) {
                m += mx;
                sub = mx;
              }
            }
            if (__any_sync(0xffffffffu, sub != 0.f))
              tile_exp<2, true>(x, f2_pack(sub, sub), tP + 32 * half, sum2);
            else
              tile_exp<2, false>(x, 0, tP + 32 * half, sum2);
            if (half == 0) {  // (the second half's is passed on below)
              tmem_st_wait();
              tc_fence_before();
              mbar_arrive(p_ready + 2 * t);
            }
          }
          if (!ok) break;
        }
        {
          float s0, s1, s2, s3;
          f2_unpack(f2_add(sum2[0], sum2[2]), s0, s1);
          f2_unpack(f2_add(sum2[1], sum2[3]), s2, s3);
          l += (s0 + s1) + (s2 + s3);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_ready + 2 * t + (C::SEP_P ? 0 : 1));
      }
      // ---- the item's rows
      g += steps;
      g_other += steps_other;
      if (steps == 0) continue;  // one key tile: the other warpgroup's
      if (ok) ok = warp_wait(o_ready + t, (g - 1) & 1, wd);
      const bool pair = it.tiles == 1 && it.j1 - it.j0 > 1;  // both warpgroups hold these rows
      if (pair && t == 1) {
        if (ok) {
          stats[r] = make_float2(m, l);
          mbar_arrive(merge_ready);
        }
        continue;
      }
      float f0 = 1.f, f1 = 0.f;
      if (pair) {
        if (ok) ok = warp_wait(merge_ready, merges & 1, wd) &&
                     warp_wait(o_ready + 1, (g_other - 1) & 1, wd);
        ++merges;
        if (ok) {
          const float2 st = stats[r];
          const float M = fmaxf(m, st.x);
          f0 = m == -INFINITY ? 0.f : ex2(m - M);
          f1 = st.x == -INFINITY ? 0.f : ex2(st.x - M);
          l = l * f0 + st.y * f1;
          m = M;
        }
      }
      if (!ok) continue;
      tc_fence_after();
      const float inv = whole ? (l == 0.f ? 0.f : 1.0f / l) : 1.f;
      f0 *= inv;
      f1 *= inv;
      const int prow = t_row * RT + r;
      // where this lane stores: rows 8 k + lane / 4 of the warp's, relative to the item's first head
      __nv_bfloat16 *out0 = p.out + ((size_t)(it.row0 + t_row * tq) * p.hq + (size_t)it.hk * G) * D;
      int to[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int rr = (warp & 3) * 32 + 8 * k + (lane >> 2), q = rr / G;
        to[k] = rr < RT && q < ntok ? (q * p.hq + (rr - q * G)) * D : -1;
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        __syncwarp();
        tmem_ld32(tO + c * 32, o);
        if (pair) {
          uint32_t o1[32];
          tmem_ld32(tO + C::O_STRIDE + c * 32, o1);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            o[k] = __float_as_uint(__uint_as_float(o[k]) * f0 + __uint_as_float(o1[k]) * f1);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f0);
        }
        if (whole) {
          // through shared memory, so that a store covers 64 bytes of each of eight rows rather than
          // 16 bytes of 32 (3 us less for an item's 256 rows)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack_bf16x2(__uint_as_float(o[8 * v + 2 * k]),
                                 __uint_as_float(o[8 * v + 2 * k + 1]));
            st_shared_v4(scratch + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4), w[0], w[1], w[2],
                         w[3]);
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rr = 8 * k + (lane >> 2);
            const uint4 w = ld_shared_v4(scratch + rr * 64 +
                                         (((lane & 3) ^ ((rr >> 1) & 3)) << 4));
            if (to[k] >= 0)
              *reinterpret_cast<uint4 *>(out0 + (size_t)to[k] + c * 32 + (lane & 3) * 8) = w;
          }
          __syncwarp();
        } else if (valid) {
          float *part = part_rows<kTileRows, D>(p.part, gridDim.x, blockIdx.x, which);
#pragma unroll
          for (int v = 0; v < 8; ++v)
            *part_quad<kTileRows>(part, prow, c * 8 + v) =
                make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                            __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
        }
      }
      __syncwarp();
      tc_fence_before();
      mbar_arrive(o_free + t);
      if (pair) mbar_arrive(o_free + 1);
      if (valid) {
        if (!whole)
          *reinterpret_cast<float2 *>(
              part_stats<kTileRows, D>(p.part, gridDim.x, blockIdx.x, which) + prow * 2) =
              make_float2(m, l);
        else if (p.lse != nullptr)
          p.lse[(size_t)h * p.total_q + row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D>
int launch_t(const PagedParams &p, const fat_paged_cache_t &c, cudaStream_t stream) {
  using C = TileCfg<D>;
  PagedParams pp = p;
  CUtensorMap mq, mk, mv;
  const int kbox = std::min(128, 1 << p.log2_page);
  int rc = make_tmap_pages(&mk, c.k, c, kbox, &pp.head_outer);
  if (!rc) rc = make_tmap_pages(&mv, c.v, c, kbox, &pp.head_outer);
  if (rc) return rc;
  if (make_tmap_rows(&mq, p.q, p.total_q, p.hq, D, p.group, 128 / p.group)) return FAT_ECUDA;
  const size_t smem = 1024 + C::OFF_LUT + (p.bias.table ? (size_t)((p.bias.lut_len + 15) & ~15) : 0);
  if (prepare_kernel((const void *)fat_paged_tile_kernel<D>, smem, kThreads, C::REGS_NEEDED))
    return FAT_ECUDA;
  return launch_dependent("paged tile kernel launch", fat_paged_tile_kernel<D>,
                          dim3((unsigned)paged_tile_ctas()), kThreads, smem, stream, mq, mk, mv, pp);
}

}  // namespace

int paged_tile_ctas() { return sm_count() > 0 ? sm_count() : 152; }

int launch_paged_tile(const PagedParams &p, const fat_paged_cache_t &c, cudaStream_t stream) {
  return c.head_dim == 64 ? launch_t<64>(p, c, stream) : launch_t<128>(p, c, stream);
}

}  // namespace fat
