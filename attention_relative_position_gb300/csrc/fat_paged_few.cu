// fat_paged_few.cu -- attention over a paged cache for requests with few rows: a decode step, a few
// drafted tokens, a group's heads over their key/value head (queries x group heads <= 16 rows).
//
// The work is one read of the requests' keys and values; the rows ride along. A CTA (two per SM)
// takes an equal share of all key stages (fat_paged.cuh); a stage is 8 KB of keys and values (16
// tokens at head_dim 128, 32 at 64). Four warps compute, each on stages of its own from a ring of
// three; four more fill the rings, one each, by TMA (boxes of 16 rows x 64 channels, of 32 where
// stage and page hold as many, 128-byte swizzle), the page numbers of many stages loaded at once.
// One warp for the four rings, a lane each, put a stage off every 0.9 us, and short contexts waited
// for it: one token over 500 keys 9.4 us against 7.4. What is copied is marked to leave L2 first: a
// request reads it once (24 x 5 drafted tokens over 127 MB 33.2 us without, 30.5 with). Pages that
// requests share (a common prefix) are found in L2 all the same: 32 tokens over one prefix of 4000 keys,
// 32 heads over 8 of 128 channels, 49 us, over 32 contexts of their own 89.
// Per stage and warp: S = Q K^T for 16 rows with warp-level matrix products (Q in registers), bias
// and mask, a running maximum that moves only when it grows by more than 2^32, P in registers as a sum
// of two bf16 numbers, O += P V. (With one, the error against 64 bits is 0.0022 where the output's own
// rounding, and the decode kernel over packed keys with its fp32 weights, leave 0.0016.) Up to 8 rows
// the second parts take the fragment's other 8 rows and cost no products; with more, every P V is done
// twice. One part against two, in us: one token over 500 keys 7.5 / 7.7, decode of 32 requests 102.0 /
// 102.5, drafted tokens (15 rows) 30.6 / 31.8, mixed step 56 / 59.
// Warp-level products suffice here: with 16 of 128 rows of a tcgen05 tile filled, its round trip
// through tensor memory would cost more than the 32 or 48 products of a stage.
// A short item (two stages at most) is one warp's; the warps of a longer one merge their rows in
// shared memory once. Items cut by the share boundaries leave partial rows for the merge grid.
// Bound by HBM: one token for each of 32 requests over 1024 .. 4096 keys, 64 heads over 16 of 128
// channels, 602 MB in 102 us with the merge (5.9 TB/s, 0.87 of a copy's rate). Short calls are bound by
// their start: 1.2 us to the shares, 0.9 to the first copy, 0.7 to its arrival, 0.6 a stage, 1.0 for
// the merge of the warps (one token over 500 keys, 7.6 us from a graph).
#include <algorithm>
#include <cstdint>

#include "fat_paged.cuh"

namespace fat {
namespace {

constexpr int kWarps = 4;          // computing warps
constexpr int kThreads = 2 * kWarps * 32;
// registers of a thread: 128 at launch (two CTAs per SM), then split unevenly
constexpr int kProdRegs = 64, kCompRegs = 192;
constexpr int kRegsNeeded = kThreads / 2 * (kProdRegs + kCompRegs);  // a build with fewer is refused
static_assert(kRegsNeeded <= kThreads * 128, "what the block is launched with");
constexpr int kRing = 3;           // stages per warp
constexpr int kShortStages = 2;    // items of at most this many stages are one warp's
constexpr int kMinShare = 8;       // stages a CTA takes at least

template <int D>
struct FewCfg {
  static constexpr int KT = few_stage_tokens(D);  // tokens per stage
  static constexpr int DB = D / 64;              // 64-channel blocks
  static constexpr int LOG2_KT = D == 64 ? 5 : 4;
  static constexpr int PIECE = 16 * 128;         // 16 rows x 64 channels
  static constexpr int PIECES = KT / 16;         // of these per 64-channel block
  static constexpr int BLK = KT * 128;           // one 64-channel block of a stage
  static constexpr int TILE = DB * BLK;          // K or V of a stage
  static constexpr int STAGE = 2 * TILE;
  static constexpr int OFF_MERGE = kWarps * kRing * STAGE;
  static constexpr int OFF_STATS = OFF_MERGE + kWarps * (kWarps - 1) * 2 * 32 * 16;
  static constexpr int OFF_BAR = OFF_STATS + kWarps * kFewRows * 2 * 4;
  static constexpr int OFF_THR = OFF_BAR + 2 * kWarps * kRing * 8 + 64;
  static constexpr int OFF_SHARE = OFF_THR + kMaxThresholds * 4;
  static constexpr int OFF_LUT = OFF_SHARE + (int)sizeof(ShareSmem<kThreads>);
  // bucket bytes of the deltas -sat_neg .. sat_pos (up to 2.2 KB two CTAs fit on an SM, beyond that
  // one: saturation distances of a thousand keys each way still fit)
  static int bytes(const BiasParams &b) {
    return OFF_LUT + (b.table ? (b.sat_neg + b.sat_pos + 1 + 15) & ~15 : 0);
  }
  static_assert(OFF_LUT + kMaxBiasSpan + 16 + 1024 <= kSmemLimit, "shared memory");
  static_assert(STAGE == 8192 && KT == 1 << LOG2_KT, "a stage is 8 KB");
};

// Two weights (at most 2^32) as bf16 pairs hi + lo: what is left is below 2^-16 of them.
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16x2(a, b);
  const float2 r = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&hi));
  lo = pack_bf16x2(a - r.x, b - r.y);
}

// The items of a share in order.
struct FewItem {
  int doc, hk, sq, lq, lk, nst;  // nst: stages of the item (0: no keys)
  int s0, s1;                    // the stages taken here
  bool begins, ends;
};
template <int D>
struct FewWalk {
  const PagedParams &p;
  const ShareSmem<kThreads> &sm;
  int first_doc, doc, hk;
  long long left;  // cost still to take
  int off;         // cost of the current item that lies before the stretch
  __device__ bool next(FewItem &it) {
    while (left > 0 && doc < p.n) {
      const PagedDoc d = share_doc(p, sm, first_doc, doc);
      if (!d.ok || (long long)d.lq * p.group > p.few_rows) {
        ++doc;
        hk = 0;
        continue;
      }
      constexpr int KT = FewCfg<D>::KT;
      it.nst = (d.lk + KT - 1) / KT;
      const int cost = few_item_cost(it.nst);
      const int o = off;
      off = 0;
      const int take = (int)min(left, (long long)(cost - o));
      left -= take;
      it.doc = doc;
      it.hk = hk;
      it.sq = d.sq;
      it.lq = d.lq;
      it.lk = d.lk;
      if (++hk == p.hkv) {
        hk = 0;
        ++doc;
      }
      if (!p.split) {  // whole items: the one that begins earlier is another CTA's
        if (o > 0) continue;
        it.s0 = 0;
        it.s1 = it.nst;
        it.begins = it.ends = true;
        return true;
      }
      // the fixed part of the cost comes first, before the stages
      it.s0 = max(o - kFewItem, 0);
      it.s1 = max(o + take - kFewItem, 0);
      it.begins = it.s0 == 0;
      it.ends = o + take == cost;
      if (it.s0 == it.s1 && !(it.nst == 0 && it.ends)) continue;  // a boundary before its stages
      return true;
    }
    return false;
  }
};

// The stages of one warp, in order: of a short item all (items take turns over the warps), of a
// longer one every kWarps-th, continuing the turn of the item before.
template <int D>
struct FewStages {
  FewWalk<D> walk;
  FewItem it;
  int s, step;   // next stage of `it` and the distance to the one after
  int turn;      // stages dealt so far, modulo kWarps
  int shorts;    // short items so far
  __device__ explicit FewStages(const FewWalk<D> &w) : walk(w), s(0), step(1), turn(0), shorts(0) {}
  // The next item with its first stage for `warp` (s >= it.s1: none of its stages).
  __device__ bool item(int warp) {
    if (!walk.next(it)) return false;
    if (it.s1 - it.s0 <= kShortStages) {
      s = (shorts & (kWarps - 1)) == warp ? it.s0 : it.s1;
      step = 1;
      ++shorts;
    } else {
      s = it.s0 + ((warp - turn) & (kWarps - 1));
      step = kWarps;
      turn = (turn + it.s1 - it.s0) & (kWarps - 1);
    }
    return true;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    fat_paged_few_kernel(const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ PagedParams p) {
  using C = FewCfg<D>;
  constexpr int KT = C::KT, NT = KT / 8;  // key groups of 8
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto &share_s = *reinterpret_cast<ShareSmem<kThreads> *>(sm + C::OFF_SHARE);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR);  // full, then empty, [warp][ring]
  volatile int *abort_flag =
      reinterpret_cast<volatile int *>(sm + C::OFF_BAR + 2 * kWarps * kRing * 8);
  int *thr_s = reinterpret_cast<int *>(sm + C::OFF_THR);
  float *stats = reinterpret_cast<float *>(sm + C::OFF_STATS);  // [warps][16][2]
  grid_dep_launch();
  if (tid == 0) *abort_flag = 0;
  if (tid < 2 * kWarps * kRing) {
    mbar_init(bars + tid, 1);
    fence_mbar_init();
  }
  if (tid == kThreads - 32) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  for (int i = tid; i < p.bias.n_thr; i += kThreads) thr_s[i] = p.bias.thr[i];
  // Beside the tile kernel, which has waited for the work before it, nothing is waited for here.
  if (!p.both) grid_dep_wait();
  if (p.split && tid < 2) {
    PartRecord *r = part_record(p.part, blockIdx.x, tid);
    r->valid = 0;
  }
  const FewCost<D> cost{p};
  const Share sh = share_find<kThreads>(
      p, kMinShare, cost, TileCost{p, 128 / p.group, 2 * (128 / p.group)},
      [&](long long mine, long long other) {
        return 2 * (p.sms - (p.both ? tile_sms<D>(p, other, mine) : 0));
      },
      share_s);
  if (sh.lo >= sh.hi) {
    grid_dep_wait();
    return;
  }
  const Watchdog wd{abort_flag, p.err, FAT_DEVERR_TIMEOUT_FWD, p.timeout_ns};
  const PagedDoc d0 = share_doc(p, share_s, sh.doc, sh.doc);
  const int cost0 = few_item_cost((d0.lk + KT - 1) / KT);
  const int hk0 = (int)div_small(sh.off, cost0);
  const FewWalk<D> start{p, share_s, sh.doc, sh.doc, hk0, sh.hi - sh.lo,
                         (int)(sh.off - (long long)hk0 * cost0)};

  if (warp >= kWarps) {
    // ------------------------------------------------------------------ producers
    // Warp kWarps + w fills warp w's ring. It waits on that ring alone: a warp that waits for the
    // others at the end of an item must not hold up their copies.
    regs_dec<kProdRegs>();
    const int w = warp - kWarps;
    uint8_t *ring = sm + w * kRing * C::STAGE;
    uint64_t *full = bars + w * kRing, *empty = bars + (kWarps + w) * kRing;
    const int log2_box = min(p.log2_page, C::LOG2_KT);  // rows of a copy
    const uint64_t once = l2_evict_first();  // a request's keys and values are read once
    const int in_mask = (1 << p.log2_page) - 1;
    FewStages<D> ahead(start);
    int slot = 0, phase = 1;
    bool ok = !(p.debug_flags & 1);  // test hook: no copies, the waits run out
    while (ok && ahead.item(w)) {
      const FewItem &it = ahead.it;
      if (ahead.s >= it.s1) continue;
      // The page numbers of the item's next kBatch stages, lane PIECES j + i those of stage j's
      // rows 16 i: loaded a batch ahead.
      constexpr int kBatch = 32 / C::PIECES;
      const int32_t *row = p.table + (size_t)it.doc * p.width;
      auto pages = [&](int s) {
        const int tok =
            (s + (lane / C::PIECES) * ahead.step) * KT + (lane & (C::PIECES - 1)) * 16;
        return tok < it.lk ? __ldg(row + (tok >> p.log2_page)) : 0;
      };
      int mine = pages(ahead.s), coming = 0;
      {  // the item's queries (a row per two lanes) and bias table rows, towards L1
        const int h0 = it.hk * p.group, all = it.s1 - it.s0 >= kWarps ? kWarps : 1;
        const int r = lane >> 1, q = r / p.group;
        if (q < it.lq && (D == 128 || (lane & 1) == 0))
          prefetch_l1(p.q + ((size_t)(it.sq + q) * p.hq + h0 + (r - q * p.group)) * D +
                      (lane & 1) * 64);
        if (p.bias.table != nullptr)
          for (int b = lane + (all > 1 ? w : 0) * 32; b < p.bias.nb; b += 32 * all)
            prefetch_l1(p.bias.table + (size_t)b * p.hq + h0);
        if (p.bias.slopes != nullptr && lane == 0) prefetch_l1(p.bias.slopes + h0);
      }
      int j = 0;  // the stage's place in the batch
      for (int s = ahead.s; s < it.s1; s += ahead.step) {
        if (j == 0) coming = pages(s + kBatch * ahead.step);
        if (!(ok = warp_wait(empty + slot, phase, wd))) break;
        const int tok = s * KT, n = min(KT, it.lk - tok);
        int page[C::PIECES];
#pragma unroll
        for (int i = 0; i < C::PIECES; ++i)
          page[i] = __shfl_sync(0xffffffffu, mine, j * C::PIECES + i);
        if (lane == 0) {
          const int copies = (n + (1 << log2_box) - 1) >> log2_box;
          uint8_t *dst = ring + slot * C::STAGE;
          mbar_arrive_expect_tx(full + slot, (copies << log2_box) * 2 * D * 2);
#pragma unroll
          for (int i = 0; i < C::PIECES; ++i) {
            if (i >= copies) break;
            if ((unsigned)page[i] >= (unsigned)p.num_pages) {
              atomicOr(p.err, FAT_DEVERR_PAGES);
              page[i] = p.num_pages;  // just outside: filled with zeros
            }
            const int in = (tok + (i << log2_box)) & in_mask;
            const int c1 = p.head_outer ? in : it.hk, c2 = p.head_outer ? it.hk : in;
#pragma unroll
            for (int b = 0; b < C::DB; ++b) {
              uint8_t *d = dst + i * C::PIECE + b * C::BLK;
              tma_load_4d(&tm_k, full + slot, d, 64 * b, c1, c2, page[i], once);
              tma_load_4d(&tm_v, full + slot, d + C::TILE, 64 * b, c1, c2, page[i], once);
            }
          }
        }
        __syncwarp();
        if (++slot == kRing) {
          slot = 0;
          phase ^= 1;
        }
        if (++j == kBatch) {
          j = 0;
          mine = coming;
        }
      }
    }
    if (*abort_flag) {  // copies may still be on their way: give them time to land
      const uint64_t a = global_timer_ns();
      while (global_timer_ns() - a < 1000000ull) __nanosleep(1000);
    }
    grid_dep_wait();  // as at the end of the other warps
    return;
  }
  regs_inc<kCompRegs>();
  uint8_t *ring = sm + warp * kRing * C::STAGE;
  uint64_t *full = bars + warp * kRing, *empty = bars + (kWarps + warp) * kRing;

  // ---- computation
  FewStages<D> cur(start);
  const int G = p.group;
  const int r0 = lane >> 2, r1 = r0 + 8;  // this thread's rows, keys 2 (lane % 4) + {0, 1} + 8 t
  const bool t5 = p.bias.table != nullptr;
  const bool biased = p.bias.has_bias != 0;
  // bucket of every near delta, one byte each
  uint8_t *lut = sm + C::OFF_LUT;
  const int span = p.bias.sat_neg + p.bias.sat_pos;
  if (t5) {
    for (int i = tid; i <= span; i += kWarps * 32)
      lut[i] = (uint8_t)t5_bucket_staged(i - p.bias.sat_neg, p.bias, thr_s);
    named_bar_sync(1, kWarps * 32);
  }
  const int bucket_pos = t5 ? lut[span] : 0, bucket_neg = t5 ? lut[0] : 0;
  int slot = 0, phase = 0;
  bool ok = true;
  while (cur.item(warp)) {
    const FewItem &it = cur.it;
    const bool shortened = it.s1 - it.s0 <= kShortStages;  // one warp's
    const bool mine = !shortened || ((cur.shorts - 1) & (kWarps - 1)) == warp;
    if (!mine) continue;
    const int rows = it.lq * G, shift = it.lk - it.lq;
    const bool half = rows <= 8;  // rows 8 .. 15 of O take the second parts of rows 0 .. 7
    uint32_t qf[D / 16][4];
    int qpos[2], lim[2], head[2];
    float slope[2], far_pos[2], far_neg[2];
    const int lim_all = p.causal ? min(shift, it.lk - 1) : it.lk - 1;  // every row sees up to here
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int t = 0; t < D / 8; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;

    for (int s = cur.s; s < it.s1; s += cur.step) {
      if (s == cur.s) {  // the item's first stage here
        // Q as the A operand: rows r0, r1, channels 16 kk + 2 (lane % 4) + {0, 1} and + 8
        const __nv_bfloat16 *qb = p.q + ((size_t)it.sq * p.hq + (size_t)it.hk * G) * D;
        const int q0 = r0 / G, q1 = r1 / G;
        const uint32_t *a = reinterpret_cast<const uint32_t *>(
            qb + ((size_t)q0 * p.hq + (r0 - q0 * G)) * D) + (lane & 3);
        const uint32_t *b = reinterpret_cast<const uint32_t *>(
            qb + ((size_t)q1 * p.hq + (r1 - q1 * G)) * D) + (lane & 3);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qf[kk][0] = r0 < rows ? __ldg(a + kk * 8) : 0u;
          qf[kk][1] = r1 < rows ? __ldg(b + kk * 8) : 0u;
          qf[kk][2] = r0 < rows ? __ldg(a + kk * 8 + 4) : 0u;
          qf[kk][3] = r1 < rows ? __ldg(b + kk * 8 + 4) : 0u;
        }
        // per row: query position among the keys, last visible key, bias constants
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = i ? r1 : r0, q = r / G;
          qpos[i] = q + shift;
          head[i] = it.hk * G + (r - q * G);
          lim[i] = p.causal ? min(qpos[i], it.lk - 1) : it.lk - 1;
          slope[i] = p.bias.slopes ? __ldg(p.bias.slopes + head[i]) * kLog2e : 0.f;
          far_pos[i] =
              t5 ? __ldg(p.bias.table + (size_t)bucket_pos * p.hq + head[i]) * kLog2e : 0.f;
          far_neg[i] =
              t5 ? __ldg(p.bias.table + (size_t)bucket_neg * p.hq + head[i]) * kLog2e : 0.f;
        }
      }
      if (ok) ok = warp_wait(full + slot, phase, wd);
      if (ok) {
        const uint8_t *kt = ring + slot * C::STAGE;
        uint8_t *vt = ring + slot * C::STAGE + C::TILE;
        const int k0 = s * KT;
        if (k0 + KT > it.lk) {  // values behind the last key: whatever the page holds, they are 0
          const int first = it.lk - k0;
          for (int i = first * 8 * C::DB + lane; i < KT * 8 * C::DB; i += 32) {
            const int row = i / (8 * C::DB), c = i % (8 * C::DB);
            *reinterpret_cast<uint4 *>(vt + (c >> 3) * C::BLK + row * 128 + (c & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();  // before the next copy into this place
          __syncwarp();
        }
        // S = Q K^T
        float x[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
        const uint32_t ka = smem_u32(kt) + (lane & 7) * 128 + (lane >> 4) * 1024;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ch = ((uint32_t)(((2 * kk) & 7) + ((lane >> 3) & 1)) ^ (lane & 7)) << 4;
#pragma unroll
          for (int t = 0; t < NT; t += 2) {
            uint32_t b[4];
            ldmatrix_x4(ka + (kk >> 2) * C::BLK + t * 1024 + ch, b);
            mma_16x8x16(x[t], qf[kk], b[0], b[1]);
            mma_16x8x16(x[t + 1], qf[kk], b[2], b[3]);
          }
        }
        // logits in log2 units
        const int kb = k0 + 2 * (lane & 3);
        if (!biased) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[t][e] *= p.scale_log2;
        } else if (k0 - (shift + it.lq - 1) >= p.bias.sat_pos ||
                   k0 + KT - 1 - shift <= -p.bias.sat_neg) {  // every delta on one far side
          const bool pos = k0 - (shift + it.lq - 1) >= p.bias.sat_pos;
          const float kk[2] = {pos ? -slope[0] : slope[0], pos ? -slope[1] : slope[1]};
          const float c0[2] = {fmaf(kk[0], (float)(kb - qpos[0]), pos ? far_pos[0] : far_neg[0]),
                               fmaf(kk[1], (float)(kb - qpos[1]), pos ? far_pos[1] : far_neg[1])};
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[t][e] = fmaf(x[t][e], p.scale_log2,
                             fmaf(kk[e >> 1], (float)(8 * t + (e & 1)), c0[e >> 1]));
        } else {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = e >> 1, delta = kb + 8 * t + (e & 1) - qpos[i];
              float b = -slope[i] * fabsf((float)delta);
              if (t5) {
                const int bk = lut[min(max(delta + p.bias.sat_neg, 0), span)];
                b += __ldg(p.bias.table + bk * p.hq + head[i]) * kLog2e;
              }
              x[t][e] = fmaf(x[t][e], p.scale_log2, b);
            }
        }
        if (k0 + KT - 1 > lim_all) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (kb + 8 * t + (e & 1) > lim[e >> 1]) x[t][e] = -INFINITY;
        }
        // the running maximum, moved only when it grows by more than 2^32
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mx[0] = fmax3(mx[0], x[t][0], x[t][1]);
          mx[1] = fmax3(mx[1], x[t][2], x[t][3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        }
        const bool up0 = mx[0] > m[0] + 32.f || (m[0] == -INFINITY && mx[0] > m[0]);
        const bool up1 = !half && (mx[1] > m[1] + 32.f || (m[1] == -INFINITY && mx[1] > m[1]));
        if (__any_sync(0xffffffffu, up0 || up1)) {
          const float f0 = up0 ? ex2(m[0] - mx[0]) : 1.f;
          const float f1 = half ? f0 : up1 ? ex2(m[1] - mx[1]) : 1.f;
          if (up0) m[0] = mx[0];
          if (up1) m[1] = mx[1];
          l[0] *= f0;
          l[1] *= f1;
#pragma unroll
          for (int t = 0; t < D / 8; ++t) {
            o[t][0] *= f0;
            o[t][1] *= f0;
            o[t][2] *= f1;
            o[t][3] *= f1;
          }
        }
        const float s0 = m[0] == -INFINITY ? 0.f : m[0], s1 = m[1] == -INFINITY ? 0.f : m[1];
        // P as two bf16 parts, the weight rounded and what that left (16 bits in all; the sums are of
        // the unrounded weights), O += P V. Up to 8 rows: the second parts are rows 8 .. 15 of the
        // same products. More: products of their own.
        const uint32_t va = smem_u32(vt) + ((lane & 7) + ((lane >> 3) & 1) * 8) * 128;
        auto values = [&](int kk, int t, uint32_t (&b)[4]) {  // of 16 keys, channels 8 t .. 8 t + 15
          ldmatrix_x4_trans(va + (t >> 3) * C::BLK + kk * 2048 +
                                (((uint32_t)((t & 7) + (lane >> 4)) ^ (lane & 7)) << 4), b);
        };
        if (half) {
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk) {
            uint32_t pf[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float a = ex2(x[2 * kk + h][0] - s0), b = ex2(x[2 * kk + h][1] - s0);
              l[0] += a + b;
              split_bf16x2(a, b, pf[2 * h], pf[2 * h + 1]);
            }
#pragma unroll
            for (int t = 0; t < D / 8; t += 2) {
              uint32_t b[4];
              values(kk, t, b);
              mma_16x8x16(o[t], pf, b[0], b[1]);
              mma_16x8x16(o[t + 1], pf, b[2], b[3]);
            }
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float a = ex2(x[2 * kk + h][0] - s0), b = ex2(x[2 * kk + h][1] - s0);
              const float c = ex2(x[2 * kk + h][2] - s1), d = ex2(x[2 * kk + h][3] - s1);
              l[0] += a + b;
              l[1] += c + d;
              split_bf16x2(a, b, hi[2 * h], lo[2 * h]);
              split_bf16x2(c, d, hi[2 * h + 1], lo[2 * h + 1]);
            }
#pragma unroll
            for (int t = 0; t < D / 8; t += 2) {
              uint32_t b[4];
              values(kk, t, b);
              mma_16x8x16(o[t], hi, b[0], b[1]);
              mma_16x8x16(o[t + 1], hi, b[2], b[3]);
              mma_16x8x16(o[t], lo, b[0], b[1]);
              mma_16x8x16(o[t + 1], lo, b[2], b[3]);
            }
          }
        }
        __syncwarp();  // the stage has been read: its place is free for the next copy
        if (lane == 0) mbar_arrive(empty + slot);
      }
      if (++slot == kRing) {
        slot = 0;
        phase ^= 1;
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    if (half) {
#pragma unroll
      for (int t = 0; t < D / 8; ++t) {
        o[t][0] += o[t][2];
        o[t][1] += o[t][3];
      }
    }

    // ---- the item's rows: whole ones to out, cut ones to the workspace
    const bool whole = it.begins && it.ends;
    const int which = it.begins ? 1 : 0;
    if (!whole && (shortened || warp == 0) && lane == 0) {
      PartRecord *rec = part_record(p.part, blockIdx.x, which);
      rec->valid = 1;
      rec->ends = it.ends;
      rec->row0 = it.sq;
      rec->hk = it.hk;
      rec->rows = rows;
    }
    if (shortened) {
      float *po = whole ? nullptr : part_rows<kFewRows, D>(p.part, gridDim.x, blockIdx.x, which);
      float *ps = whole ? nullptr : part_stats<kFewRows, D>(p.part, gridDim.x, blockIdx.x, which);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = i ? r1 : r0;
        if (r >= rows) continue;
        const int q = r / G, h = it.hk * G + (r - q * G), row = it.sq + q;
        if (whole) {
          const float inv = l[i] == 0.f ? 0.f : 1.0f / l[i];
          uint32_t *dst =
              reinterpret_cast<uint32_t *>(p.out + ((size_t)row * p.hq + h) * D) + (lane & 3);
#pragma unroll
          for (int t = 0; t < D / 8; ++t)
            dst[t * 4] = pack_bf16x2(o[t][2 * i] * inv, o[t][2 * i + 1] * inv);
          if ((lane & 3) == 0 && p.lse != nullptr)
            p.lse[(size_t)h * p.total_q + row] =
                l[i] == 0.f ? -INFINITY : (m[i] + __log2f(l[i])) * kLn2;
        } else {
#pragma unroll
          for (int t = 0; t < D / 8; ++t)
            reinterpret_cast<float2 *>(
                part_quad<kFewRows>(po, r, t * 2 + ((lane >> 1) & 1)))[lane & 1] =
                make_float2(o[t][2 * i], o[t][2 * i + 1]);
          if ((lane & 3) == 0) *reinterpret_cast<float2 *>(ps + r * 2) = make_float2(m[i], l[i]);
        }
      }
      continue;
    }
    // Merge of the four warps: each takes a quarter of every 64 channels (16: two of its fragments'
    // blocks of 8) from the other three, which leave theirs, scaled to the common maximum, as they
    // hold them (a thread's rows and columns are the same in every warp: no transposition).
    if ((lane & 3) == 0) {
      *reinterpret_cast<float2 *>(stats + (warp * kFewRows + r0) * 2) = make_float2(m[0], l[0]);
      *reinterpret_cast<float2 *>(stats + (warp * kFewRows + r1) * 2) = make_float2(m[1], l[1]);
    }
    named_bar_sync(1, kWarps * 32);
    float f[2], M[2], L[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i ? r1 : r0;
      M[i] = -INFINITY;
      L[i] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M[i] = fmaxf(M[i], stats[(w * kFewRows + r) * 2]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = *reinterpret_cast<const float2 *>(stats + (w * kFewRows + r) * 2);
        L[i] += v.y * (v.x == -INFINITY ? 0.f : ex2(v.x - M[i]));  // (0 * NaN stays NaN)
      }
      f[i] = m[i] == -INFINITY ? 0.f : ex2(m[i] - M[i]);
    }
    float4 *buf = reinterpret_cast<float4 *>(sm + C::OFF_MERGE);  // [to][from][2][32]
#pragma unroll
    for (int b = 0; b < C::DB; ++b) {
      if (b > 0) named_bar_sync(1, kWarps * 32);  // the block before has been read
      float4 own[2];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const int w = t >> 1, ot = 8 * b + t;
        const float4 v =
            make_float4(o[ot][0] * f[0], o[ot][1] * f[0], o[ot][2] * f[1], o[ot][3] * f[1]);
        if (w == warp)
          own[t & 1] = v;
        else
          buf[((w * (kWarps - 1) + ((warp - w - 1) & (kWarps - 1))) * 2 + (t & 1)) * 32 + lane] = v;
      }
      named_bar_sync(1, kWarps * 32);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        // in the order of the warps, whichever of them adds
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 v =
              w == warp ? own[t]
                        : buf[((warp * (kWarps - 1) + ((w - warp - 1) & (kWarps - 1))) * 2 + t) *
                                  32 + lane];
          a.x += v.x;
          a.y += v.y;
          a.z += v.z;
          a.w += v.w;
        }
        const int ch = 64 * b + 16 * warp + 8 * t + 2 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = i ? r1 : r0;
          const float x = i ? a.z : a.x, y = i ? a.w : a.y;
          if (r >= rows) continue;
          if (whole) {
            const int q = r / G, h = it.hk * G + (r - q * G), row = it.sq + q;
            const float inv = L[i] == 0.f ? 0.f : 1.0f / L[i];
            *reinterpret_cast<uint32_t *>(p.out + ((size_t)row * p.hq + h) * D + ch) =
                pack_bf16x2(x * inv, y * inv);
            if (ch == 0 && p.lse != nullptr)
              p.lse[(size_t)h * p.total_q + row] =
                  L[i] == 0.f ? -INFINITY : (M[i] + __log2f(L[i])) * kLn2;
          } else {
            reinterpret_cast<float2 *>(
                part_quad<kFewRows>(part_rows<kFewRows, D>(p.part, gridDim.x, blockIdx.x, which),
                                    r, ch >> 2))[lane & 1] = make_float2(x, y);
            if (ch == 0)
              *reinterpret_cast<float2 *>(
                  part_stats<kFewRows, D>(p.part, gridDim.x, blockIdx.x, which) + r * 2) =
                  make_float2(M[i], L[i]);
          }
        }
      }
    }
    // (the next merge writes buf only after its first barrier, stats only after this one's last)
  }
  // A grid that was started beside the tile kernel's ends after it, so that the merge grids, which
  // wait for this one, find both complete (returns at once when there is none before).
  grid_dep_wait();
}

template <int D>
int launch_t(const PagedParams &p, const fat_paged_cache_t &c, cudaStream_t stream) {
  PagedParams pp = p;
  CUtensorMap mk, mv;
  const int rows = std::min(1 << pp.log2_page, FewCfg<D>::KT);
  int rc = make_tmap_pages(&mk, c.k, c, rows, &pp.head_outer);
  if (!rc) rc = make_tmap_pages(&mv, c.v, c, rows, &pp.head_outer);
  if (rc) return rc;
  const size_t smem = FewCfg<D>::bytes(p.bias) + 1024;
  if (prepare_kernel((const void *)fat_paged_few_kernel<D>, smem, kThreads, kRegsNeeded))
    return FAT_ECUDA;
  return launch_dependent("paged few-row kernel launch", fat_paged_few_kernel<D>,
                          dim3((unsigned)paged_few_ctas()), kThreads, smem, stream, mk, mv, pp);
}

}  // namespace

int paged_few_ctas() { return 2 * (sm_count() > 0 ? sm_count() : 152); }

int launch_paged_few(const PagedParams &p, const fat_paged_cache_t &c, cudaStream_t stream) {
  return c.head_dim == 64 ? launch_t<64>(p, c, stream) : launch_t<128>(p, c, stream);
}

}  // namespace fat
