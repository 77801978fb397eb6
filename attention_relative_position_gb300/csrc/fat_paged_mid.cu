// fat_paged_mid.cu -- attention of trees of drafted tokens over a paged cache: more rows (queries x group heads
// per key/value head) than the few-row kernel takes, in items of 64 or 128.
//
// As in the few-row kernel the work is one read of the requests' keys and values; 64 or 128 rows make it
// enough for the tensor cores. The rows are the narrow side of both products, so that a step costs what
// its rows need and the softmax keeps every lane busy:
//   S^T = K Q^T (128 keys x R rows), P = 2^(S - reference), O^T += V^T P^T (channels x R rows).
// Two warpgroups of softmax threads share a tile's rows, half of them each. A thread holds one key's logits
// against its group's rows (a TMEM lane); what it subtracts per row, the reference, is a shared number. A
// row's reference is the largest of eight logits of the first tile taken, and is raised to the maximum (O and
// the sums scaled) when a weight would exceed 2^32: a group's 128 threads vote once a tile, and a maximum
// over the keys, across lanes, is formed only then. A thread sums its own key's weights in a register per row
// (unrounded, fp32); the threads' sums are added at an item's end. Key tiles go from the last one backwards,
// from the request's own tokens and the largest linear bias on. P is rounded to bf16, as in the tile kernel
// (outputs 0.0023 off in the mean, 0.0017 with the few-row kernel's two parts, for which shared memory has
// no room beside 128 rows and would take a stage of values beside 64).
// One persistent CTA per SM takes an equal share of all key tiles (fat_paged.cuh); requests of more rows are
// cut into blocks of them (their keys are found in L2 again):
//   warps 0-7  softmax, epilogue, zeros over the values behind the last key;
//   warp 8     Q of an item (64 rows: two buffers) and its key tiles of 128 tokens, a lane per page;
//   warp 9     issues the products; S of two tiles ahead runs beside this tile's softmax (three buffers);
//   warp 10    value tiles (one warp for both put a copy off every 0.45 us).
#include <algorithm>
#include <cstdint>

#include "fat_paged.cuh"

namespace fat {
namespace {

constexpr int kThreads = 384;  // (warp 11 only completes the third warpgroup)
constexpr int kSoftWarps = 8, kWarpK = 8, kWarpMma = 9, kWarpV = 10;
constexpr int kMinShare = 2;  // key tiles a CTA takes at least
constexpr int kItemCost = 2;  // cost of an item beside its key tiles
constexpr float kNoRow = 3e38f;      // reference of a row without a token: its weights are 0
constexpr float kFreshRow = -3e38f;  // of a row that has seen no key: whatever it sees calls for a new one
// From here on a bias (in log2 units) leaves of a logit whole numbers at most, and a reference like it cannot
// say which: rows with such biases for their far keys form logits as one rounded sum each, as long as their
// references are as large, too. That is for parts of items that begin behind the near keys: 64 trees of 12 nodes
// with -1e9 as the far T5 buckets' bias 98 -> 100 us (4000 keys of 128 channels) and 133 -> 147 (8000 of 64).
constexpr float kLargeBias = 16777216.f;
constexpr float kSeen = -2.9e38f;    // logits above this count as seen (biases down to -2e38, times log2 e)

template <int D, int R>
struct MidCfg {
  static constexpr int DB = D / 64;
  static constexpr int BLK = 128 * 128;          // 128 keys x 64 channels
  static constexpr int TILE = DB * BLK;          // K or V of a tile
  // stages of K and of V: what is in flight bounds the rate of the copies
  static constexpr int KS = D == 64 ? 5 : 2, VS = D == 64 ? (R == 64 ? 6 : 4) : R == 64 ? 3 : 2;
  static constexpr int QB = R == 64 ? 2 : 1;     // buffers of Q
  static constexpr int QBLK = R * 128, QTILE = DB * QBLK;
  static constexpr int PBLK = 128 * 128;         // 128 keys x 64 rows
  static constexpr int OFF_V = KS * TILE;
  static constexpr int OFF_Q = OFF_V + VS * TILE;
  static constexpr int OFF_P = OFF_Q + QB * QTILE;
  static constexpr int RW = R / 2;               // rows of a softmax warpgroup
  // registers of a softmax thread and of the others (neither spills; 208 and 88 did in both)
  static constexpr int SOFT_REGS = R == 64 ? 200 : 216, OTHER_REGS = R == 64 ? 104 : 72;
  static constexpr int REGS_NEEDED = 256 * SOFT_REGS + 128 * OTHER_REGS;
  static_assert(REGS_NEEDED <= kThreads * ((65536 / kThreads) & ~7), "register split");
  static constexpr int PB = 1;                   // buffers of P
  static constexpr int SB = 3;                   // and of S
  static constexpr int PTILE = R / 64 * PBLK;
  static constexpr int OFF_ROW = OFF_P + PB * PTILE;
  // per row: slope; bias of a far key at the first query's position less the reference; minus the reference;
  // the reference; sum or factor; int2: position - shift, head; its place in out behind the item's first row
  static constexpr int OFF_SLOPE = OFF_ROW, OFF_FAR = OFF_SLOPE + R * 4, OFF_NREF = OFF_FAR + R * 4;
  static constexpr int OFF_REF = OFF_NREF + R * 4, OFF_FAC = OFF_REF + R * 4, OFF_FARB = OFF_FAC + R * 4;
  static constexpr int OFF_INT = OFF_FARB + R * 4, OFF_OUT = OFF_INT + R * 8;
  static constexpr int OFF_MAX = OFF_OUT + R * 4;  // float [2][8][RW]: maxima
  static constexpr int OFF_BAR = OFF_MAX + 8 * R * 4;
  static constexpr int OFF_THR = OFF_BAR + 320;
  static constexpr int OFF_SHARE = OFF_THR + kMaxThresholds * 4;
  static constexpr int OFF_LUT = (OFF_SHARE + (int)sizeof(ShareSmem<kThreads>) + 15) & ~15;
  static int bytes(const BiasParams &b) {
    return OFF_LUT + (b.table ? (b.sat_neg + b.sat_pos + 1 + 15) & ~15 : 0);
  }
  static_assert((2 * QB + 2 * KS + 2 * VS + 2 * SB + 6) * 8 + 8 <= 320, "barrier block");
  static_assert(OFF_LUT + kMaxBiasSpan + 16 + 1024 <= kSmemLimit, "shared memory");
  static constexpr uint32_t COL_O = SB * R, TMEM_COLS = 4 * R;
  static constexpr uint32_t IDESC_S = idesc_bf16_f32(128, R, 0, 0);
  static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, R, 1, 1);
};

// Blocks of a request's tokens (rows / group each at most) and the tokens of one.
__device__ __forceinline__ int mid_blocks(int lq, int rows, int group, int *per) {
  const int most = rows / group, n = (lq + most - 1) / most;
  *per = (lq + n - 1) / n;
  return n;
}
template <int R>
struct MidCost {
  const PagedParams &p;
  __device__ long long operator()(const PagedDoc &d) const {
    int per;
    return (long long)p.hkv * mid_blocks(d.lq, R, p.group, &per) * (((d.lk + 127) >> 7) + kItemCost);
  }
};
struct NoCost {
  __device__ long long operator()(const PagedDoc &) const { return 0; }
};

struct MidItem {
  int doc, hk, row0, ntok, tok0;  // row0: first token of q and out; tok0: the request's first
  int lk, shift, nkv, j0, j1;     // key tile nkv - 1 - j for j in [j0, j1)
  bool begins, ends;
};
template <int R>
struct MidWalk {
  const PagedParams &p;
  const ShareSmem<kThreads> &sm;
  int first_doc, doc, hk, b;
  long long left;  // cost still to take
  int off;         // cost of the current item that lies before the stretch
  __device__ MidWalk(const PagedParams &pp, const ShareSmem<kThreads> &s, const Share &sh)
      : p(pp), sm(s), first_doc(sh.doc), doc(sh.doc), left(sh.hi - sh.lo) {
    const PagedDoc d = share_doc<true>(p, sm, doc, doc);
    int per;
    const int n = mid_blocks(d.lq, R, p.group, &per), cost = ((d.lk + 127) >> 7) + kItemCost;
    const int item = (int)div_small(sh.off, cost);
    hk = item / n;
    b = item - hk * n;
    off = (int)(sh.off - (long long)item * cost);
  }
  __device__ bool next(MidItem &it) {
    while (left > 0 && doc < p.n) {
      const PagedDoc d = share_doc<true>(p, sm, first_doc, doc);
      if (!d.ok) {
        ++doc;
        hk = b = 0;
        continue;
      }
      int per;
      const int n = mid_blocks(d.lq, R, p.group, &per);
      it.nkv = (d.lk + 127) >> 7;
      const int cost = it.nkv + kItemCost, o = off;
      off = 0;
      const int take = (int)min(left, (long long)(cost - o));
      left -= take;
      it.doc = doc;
      it.hk = hk;
      it.tok0 = d.sq;
      it.row0 = d.sq + b * per;
      it.ntok = min(per, d.lq - b * per);
      it.lk = d.lk;
      it.shift = d.lk - d.lq;
      if (++b == n) {
        b = 0;
        if (++hk == p.hkv) {
          hk = 0;
          ++doc;
        }
      }
      if (!p.split) {  // whole items: the one that begins earlier is another CTA's
        if (o > 0) continue;
        it.j0 = 0;
        it.j1 = it.nkv;
        it.begins = it.ends = true;
        return true;
      }
      // the fixed part of the cost comes first, before the key tiles
      it.j0 = max(o - kItemCost, 0);
      it.j1 = max(o + take - kItemCost, 0);
      it.begins = it.j0 == 0;
      it.ends = o + take == cost;
      if (it.j0 == it.j1) continue;  // a boundary before its tiles (a request has a key at least)
      return true;
    }
    return false;
  }
  // Of the CTAs in which the item has tiles the first one, and their number (stretch: this CTA's on the line of
  // costs; all but the last one's are as long).
  __device__ int first_cta(const MidItem &it, const long long *stretch, int *parts) const {
    const long long tiles = stretch[1] - left - it.j1;  // where the first one lies
    const long long share = blockIdx.x ? div_small(stretch[0], blockIdx.x) : stretch[1];
    const int c = (int)div_small(tiles, share);
    *parts = (int)div_small(tiles + it.nkv - 1, share) + 1 - c;
    return c;
  }
};

// bit j of lane i's word -> bit i of lane j's
__device__ __forceinline__ uint32_t transpose32(uint32_t x, int lane) {
  uint32_t m = 0x0000ffffu;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, s);
    x = (lane & s) ? (x & ~m) | ((y & ~m) >> s) : (x & m) | ((y & m) << s);
    m ^= m << (s >> 1);
  }
  return x;
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1)
    fat_paged_mid_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ PagedParams p) {
  using C = MidCfg<D, R>;
  constexpr int KS = C::KS, VS = C::VS, QB = C::QB, SB = C::SB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto &share_s = *reinterpret_cast<ShareSmem<kThreads> *>(sm + C::OFF_SHARE);
  uint64_t *q_full = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR);  // [QB] each
  uint64_t *q_empty = q_full + QB;
  uint64_t *k_full = q_empty + QB;  // [KS] each
  uint64_t *k_empty = k_full + KS;
  uint64_t *v_full = k_empty + KS;  // [VS] each
  uint64_t *v_empty = v_full + VS;
  uint64_t *s_full = v_empty + VS;  // [SB] each
  uint64_t *s_free = s_full + SB;
  uint64_t *p_ready = s_free + SB;  // [2]
  uint64_t *o_ready = p_ready + 2;  // [2]: a tile's last products are complete: P is free, O is up to date
  uint64_t *o_free = o_ready + 2;
  uint64_t *done = o_free + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int *thr_s = reinterpret_cast<int *>(sm + C::OFF_THR);
  uint8_t *lut = sm + C::OFF_LUT;
  const int G = p.group, tq = R / G, RT = tq * G;  // tokens and rows of a block
  grid_dep_launch();
  if (tid == 0) {
    for (int i = 0; i < QB; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
    }
    for (int i = 0; i < 2 * KS; ++i) mbar_init(k_full + i, 1);
    for (int i = 0; i < 2 * VS; ++i) mbar_init(v_full + i, 1);
    for (int i = 0; i < SB; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(s_free + i, kSoftWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(p_ready + i, kSoftWarps);
      mbar_init(o_ready + i, 1);
    }
    mbar_init(o_free, kSoftWarps);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  for (int i = tid; i < p.bias.n_thr; i += kThreads) thr_s[i] = p.bias.thr[i];
  // rows of the Q buffers that no token fills (group does not divide R): zeros, never overwritten
  for (int i = tid; i < QB * C::DB * (R - RT) * 8; i += kThreads) {
    const int blk = i / ((R - RT) * 8), rest = i % ((R - RT) * 8);
    *reinterpret_cast<uint4 *>(sm + C::OFF_Q + blk * C::QBLK + RT * 128 + rest * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  grid_dep_wait();
  if (p.split && tid < 2) part_record(p.part, blockIdx.x, tid)->valid = 0;
  const Share sh = share_find<kThreads, true>(p, kMinShare, MidCost<R>{p}, NoCost{},
                                              [&](long long, long long) { return p.sms; }, share_s);
  __shared__ long long stretch_s[2];
  if (tid == 0) {
    stretch_s[0] = sh.lo;
    stretch_s[1] = sh.hi;
  }
  if (p.bias.table != nullptr)  // (behind share_find's barriers)
    for (int i = tid; i <= p.bias.sat_neg + p.bias.sat_pos; i += kThreads)
      lut[i] = (uint8_t)t5_bucket_staged(i - p.bias.sat_neg, p.bias, thr_s);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Watchdog wd{abort_flag, p.err, FAT_DEVERR_TIMEOUT_FWD, p.timeout_ns};
  const bool work = sh.lo < sh.hi;
  if (warp >= kSoftWarps) regs_dec<C::OTHER_REGS>();
  if (work) {
    MidWalk<R> walk(p, share_s, sh);
    MidItem it;
    if (warp == kWarpK || warp == kWarpV) {
      // ------------------------------------------------------------------ producers
      const bool keys = warp == kWarpK;
      const int kbox = min(128, 1 << p.log2_page), pieces = 128 / kbox;
      const int in_mask = (1 << p.log2_page) - 1;
      const uint32_t stages = keys ? KS : VS;
      const CUtensorMap *map = keys ? &tm_k : &tm_v;
      uint64_t *full = keys ? k_full : v_full, *empty = keys ? k_empty : v_empty;
      uint8_t *ring = sm + (keys ? 0 : C::OFF_V);
      const uint64_t once = l2_evict_first();  // a request's keys and values are read once
      uint32_t slot = 0, phase = 1;
      int ni = 0;
      bool ok = !(p.debug_flags & 1);  // test hook: no copies, the waits run out
      while (ok && walk.next(it)) {
        const int n = it.j1 - it.j0, qb = ni % QB;
        const int32_t *row = p.table + (size_t)it.doc * p.width;
        auto fetch = [&](int j) -> int {  // this lane's page of the j-th tile
          const int tok = (it.nkv - 1 - it.j0 - j) * 128 + lane * kbox;
          return j < n && lane < pieces && tok < it.lk ? __ldg(row + (tok >> p.log2_page)) : 0;
        };
        int page = fetch(0), next = fetch(1);
        if (keys) {
          if (ni >= QB && !(ok = warp_wait(q_empty + qb, (ni / QB - 1) & 1, wd))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(q_full + qb, (uint32_t)RT * 128 * C::DB);
            for (int b = 0; b < C::DB; ++b)
              tma_load_3d(&tm_q, q_full + qb, sm + C::OFF_Q + qb * C::QTILE + b * C::QBLK, 64 * b,
                          it.hk * G, it.row0);
          }
        } else if (p.bias.table != nullptr) {
          for (int b = lane; b < p.bias.nb; b += 32)
            prefetch_l1(p.bias.table + (size_t)b * p.hq + it.hk * G);
        }
        ++ni;
        for (int j = 0; j < n; ++j) {
          const int after = fetch(j + 2);
          if (!(ok = warp_wait(empty + slot, phase, wd))) break;
          const int kt = it.nkv - 1 - it.j0 - j, tok = kt * 128 + lane * kbox;
          const int nvalid = min(pieces, (it.lk - kt * 128 + kbox - 1) / kbox);
          if (lane == 0) mbar_arrive_expect_tx(full + slot, (uint32_t)nvalid * kbox * 128 * C::DB);
          __syncwarp();
          if (lane < nvalid) {
            if ((unsigned)page >= (unsigned)p.num_pages) {
              atomicOr(p.err, FAT_DEVERR_PAGES);
              page = p.num_pages;  // just outside: filled with zeros
            }
            const int in = tok & in_mask;
            const int c1 = p.head_outer ? in : it.hk, c2 = p.head_outer ? it.hk : in;
            for (int b = 0; b < C::DB; ++b)
              tma_load_4d(map, full + slot, ring + slot * C::TILE + b * C::BLK + lane * kbox * 128, 64 * b, c1,
                          c2, page, once);
          }
          if (++slot == stages) {
            slot = 0;
            phase ^= 1;
          }
          page = next;
          next = after;
        }
      }
      if (*abort_flag) {  // copies may still be on their way: give them time to land
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) __nanosleep(1000);
      }
    } else if (warp == kWarpMma) {
      // ------------------------------------------------------------------ products
      // (the whole warp walks and waits, and an elected lane issues: a lane alone took 0.2 us more a tile)
      {
        uint32_t g = 0;
        int ni = 0;
        bool ok = true;
        while (ok && walk.next(it)) {
          const int n = it.j1 - it.j0, qb = ni % QB;
          const uint64_t dQ = sw128_desc(smem_u32(sm + C::OFF_Q + qb * C::QTILE), 16, 1024);
          auto issue_S = [&](int j) {  // tile j of the item
            const uint32_t gs = g + j, buf = gs % SB, s = gs % KS;
            if (!(ok = warp_wait(k_full + s, (gs / KS) & 1, wd))) return;
            if (gs >= SB && !(ok = warp_wait(s_free + buf, (gs / SB - 1) & 1, wd))) return;
            tc_fence_after();
            const uint64_t dK = sw128_desc(smem_u32(sm + s * C::TILE), 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ss_e(tmem + R * buf, dK + (((kk >> 2) * C::BLK + (kk & 3) * 32) >> 4),
                          dQ + (((kk >> 2) * C::QBLK + (kk & 3) * 32) >> 4), C::IDESC_S, kk > 0);
            mma_commit_e(s_full + buf);
            mma_commit_e(k_empty + s);
            if (j == n - 1) mma_commit_e(q_empty + qb);
          };
          if (!(ok = warp_wait(q_full + qb, (ni / QB) & 1, wd))) break;
          for (int j = 0; ok && j < min(n, SB - 1); ++j) issue_S(j);
          for (int j = 0; ok && j < n; ++j) {
            if (j + SB - 1 < n) issue_S(j + SB - 1);
            const uint32_t s = (g + j) % VS;
            const uint32_t gt = g + j;
            if (!ok || !(ok = warp_wait(v_full + s, (gt / VS) & 1, wd) &&
                              warp_wait(p_ready + (gt & 1), (gt / 2) & 1, wd)))
              break;
            // the first product overwrites O: the previous item's rows have been read
            if (j == 0 && ni > 0 && !(ok = warp_wait(o_free, (ni - 1) & 1, wd))) break;
            tc_fence_after();
            const uint64_t dP =
                sw128_desc(smem_u32(sm + C::OFF_P + ((g + j) % C::PB) * C::PTILE), C::PBLK, 1024);
            // head_dim 64: the channels twice (the second block of 64 is the first again)
            const uint64_t dV =
                sw128_desc(smem_u32(sm + C::OFF_V + s * C::TILE), D == 128 ? C::BLK : 0, 1024);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ss_e(tmem + C::COL_O, dV + ((kk * 2048) >> 4), dP + ((kk * 2048) >> 4), C::IDESC_PV,
                          j > 0 || kk > 0);
            mma_commit_e(v_empty + s);
            mma_commit_e(o_ready + ((g + j) & 1));
          }
          g += n;
          ++ni;
        }
        mma_commit_e(done);
        if (lane == 0) mbar_wait_teardown(done, 0, kTeardownNs);
        __syncwarp();
      }
    } else if (warp < kSoftWarps) {
      // ------------------------------------------------------------------ softmax: thread = key
      regs_inc<C::SOFT_REGS>();
      constexpr int RW = C::RW;
      const int wg = warp >> 2, t = tid & 127, rb = wg * RW, bar = 1 + wg;
      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      // per-row numbers of this group's rows
      float *slope_s = reinterpret_cast<float *>(sm + C::OFF_SLOPE) + rb;
      float *far_s = reinterpret_cast<float *>(sm + C::OFF_FAR) + rb;
      float *nref_s = reinterpret_cast<float *>(sm + C::OFF_NREF) + rb;
      float *ref_s = reinterpret_cast<float *>(sm + C::OFF_REF) + rb;
      float *fac_s = reinterpret_cast<float *>(sm + C::OFF_FAC) + rb;
      float *farb_s = reinterpret_cast<float *>(sm + C::OFF_FARB) + rb;
      int2 *int_s = reinterpret_cast<int2 *>(sm + C::OFF_INT) + rb;
      int *out_s = reinterpret_cast<int *>(sm + C::OFF_OUT) + rb;
      float *max_s = reinterpret_cast<float *>(sm + C::OFF_MAX) + 8 * rb;  // [8][RW]
      const bool t5 = p.bias.table != nullptr, biased = p.bias.has_bias != 0;
      const bool slopes = p.bias.slopes != nullptr;
      const int span = p.bias.sat_neg + p.bias.sat_pos;
      auto set_ref = [&](float r) {  // of row rb + t
        ref_s[t] = r;
        nref_s[t] = -r;
        far_s[t] = farb_s[t] - r;
      };
      auto o_wait = [&](uint32_t i) { return warp_wait(o_ready + (i & 1), (i / 2) & 1, wd); };
      uint32_t g = 0;
      int ni = 0;
      // A group's warps meet at barriers, so none leaves alone: once a wait has run out (ok) a warp waits no
      // more and goes through the motions until a vote ends the loops for all of them.
      bool ok = true;
      for (; ok && walk.next(it); ++ni) {
        const int n = it.j1 - it.j0, rows = it.ntok * G;
        const int mine = min(rows - rb, RW);  // rows of this group (none: it only keeps step)
        int near = 0;  // from this key on logits are formed one by one
        // (all of the group's threads; r: row t's reference, or what it may become)
        auto choose_near = [&](float r) {
          const float far = t < mine ? farb_s[t] : 0.f;
          const bool large = fmaxf(fabsf(far), t < mine ? fabsf(slope_s[t]) * (float)it.lk : 0.f) >= kLargeBias &&
                             fabsf(far) < INFINITY && fmaxf(fabsf(r), far) >= kLargeBias;
          near = named_bar_any(bar, 128, large) ? 0 : it.shift - (biased ? p.bias.sat_neg : 0);
        };
        if (mine > 0) {  // row t's numbers; its position arrives beside the first tile's logits
          const int rt = rb + min(t, mine - 1), q = rt / G, h = it.hk * G + (rt - q * G);
          int pos_in = 0;
          if (t < RW) {
            pos_in = __ldg(p.pos + it.row0 + q);
            prefetch_l1(p.mask + (size_t)(it.row0 + q) * p.mask_words);
          }
          ok = warp_wait(s_full + g % SB, (g / SB) & 1, wd);
          if (t < RW) {
            const int pos = min(max(pos_in, it.shift), it.lk - 1);
            if (pos_in != pos) atomicOr(p.err, FAT_DEVERR_INDEX);
            const float slope = slopes ? __ldg(p.bias.slopes + h) * kLog2e : 0.f;
            const float far = t5 ? __ldg(p.bias.table + (size_t)lut[0] * p.hq + h) * kLog2e : 0.f;
            slope_s[t] = slope;
            farb_s[t] = far - slope * (float)(pos - it.shift);
            int_s[t] = make_int2(pos - it.shift, h);
            out_s[t] = q * p.hq + h;
            set_ref(t < mine ? 0.f : kNoRow);
          }
          choose_near(INFINITY);
        }
        uint64_t sum[RW / 2];  // of this thread's weights, rows 2 i and 2 i + 1
#pragma unroll
        for (int i = 0; i < RW / 2; ++i) sum[i] = 0;
        for (int j = 0; j < n; ++j) {
          const uint32_t gt = g + j, buf = gt % SB;
          const uint32_t tS = tmem + lane_off + R * buf + rb;
          const int k0 = (it.nkv - 1 - it.j0 - j) * 128, key = k0 + t;
          if (ok) ok = warp_wait(s_full + buf, (gt / SB) & 1, wd);
          tc_fence_after();
          if (mine > 0) {
            float scale = p.scale_log2;
            const bool edge = k0 + 128 > near;
            const bool linear = slopes && !edge;
            const float *cst_s = edge ? nref_s : far_s;
            if (edge) {
              // Own keys, or cached ones near them: logits where they stand, masked by the rows' bits. A
              // thread's key is the same for all rows, and so is its position.
              const int key0 = k0 + (warp & 3) * 32;
              const int kp = key < it.shift ? key - it.shift
                                            : tree_pos(p, it.tok0 + min(key, it.lk - 1) - it.shift, it.shift,
                                                       it.lk) - it.shift;
#pragma unroll 1
              for (int c = 0; c < mine; c += 32) {
                const int q = (rb + min(c + lane, mine - 1)) / G;
                const uint32_t see = transpose32(
                    tree_bits(p, p.mask + (size_t)(it.row0 + q) * p.mask_words, key0 - it.shift,
                              it.lk - key0), lane);
                uint32_t x[32];
                tmem_ld32(tS + c, x);
                if (!biased) {
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    x[i] = (see >> i) & 1u ? __float_as_uint(__uint_as_float(x[i]) * scale) : 0xff800000u;
                } else if (R == 64 && k0 + 128 <= it.shift - p.bias.sat_neg) {
                  // far keys, beside large biases (128 rows have no registers left for this form)
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), scale,
                                                fmaf(slope_s[c + i], (float)(key - it.shift), farb_s[c + i])));
                } else {
#pragma unroll
                  for (int i = 0; i < 32; ++i) {
                    const int2 rc = int_s[c + i];
                    const int delta = kp - rc.x;
                    float b = -slope_s[c + i] * fabsf((float)delta);
                    if (t5) {
                      const int bk = lut[min(max(delta + p.bias.sat_neg, 0), span)];
                      b = fmaf(__ldg(p.bias.table + bk * p.hq + rc.y), kLog2e, b);
                    }
                    x[i] = (see >> i) & 1u ? __float_as_uint(fmaf(__uint_as_float(x[i]), scale, b))
                                           : 0xff800000u;
                  }
                }
                tmem_st32(tS + c, x);
              }
              tmem_st_wait();
              scale = 1.f;
            }
            const float delta0 = (float)(key - it.shift);
            // logits of 32 rows less their references, in pairs
            const uint64_t scale2 = f2_pack(scale, scale), delta2 = f2_pack(delta0, delta0);
            auto logits = [&](int c, uint64_t *y) {
              uint32_t x[32];
              tmem_ld32(tS + c, x);
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(cst_s + c + i);
                if (linear) {
                  const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(slope_s + c + i);
                  m.x = f2_fma(k.x, delta2, m.x);
                  m.y = f2_fma(k.y, delta2, m.y);
                }
                y[i / 2] = f2_fma(f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), scale2, m.x);
                y[i / 2 + 1] =
                    f2_fma(f2_pack(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), scale2, m.y);
              }
            };
            uint64_t y[RW / 2];  // of this group's rows
            auto all_logits = [&]() {
#pragma unroll
              for (int c = 0; c < RW; c += 32)
                if (c == 0 || c < mine) logits(c, y + c / 2);
            };
            if (j == 0) {  // references from eight keys of the tile (those that their row sees)
              all_logits();
              if ((t & 15) == 0) {
#pragma unroll
                for (int i = 0; i < RW / 2; i += 2)
                  *reinterpret_cast<ulonglong2 *>(max_s + (t >> 4) * RW + 2 * i) =
                      make_ulonglong2(y[i], y[i + 1]);
              }
              named_bar_sync(bar, 128);
              if (t < mine) {
                float mx = max_s[t];
#pragma unroll
                for (int i = 1; i < 8; ++i) mx = fmaxf(mx, max_s[i * RW + t]);
                set_ref(mx > kSeen ? mx : mx != mx ? 0.f : kFreshRow);  // (a NaN shows in the sum)
              }
              choose_near(t < mine ? ref_s[t] : 0.f);
            }
            all_logits();
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < RW / 2; ++i) {
              if (i >= 16 && mine <= 32) break;
              float a, b;
              f2_unpack(y[i], a, b);
              top = fmax3(top, a, b);
            }
            const bool raise = named_bar_any(bar, 128, top > 32.f || !ok);
            if (raise) {
              if (named_bar_any(bar, 128, !ok)) {
                ok = false;
                break;
              }
              // The rows' maxima over the tile, and new references where they passed 2^32. They are taken from
              // reference 0: a low reference (-3e38 of a row that has seen no key, or of keys with masking
              // biases) has rounded the other keys' logits away.
              if (t < mine) {
                fac_s[t] = ref_s[t];
                set_ref(0.f);
              }
              named_bar_sync(bar, 128);
#pragma unroll 1
              for (int c = 0; c < mine; c += 32) {
                float best = -INFINITY;
                logits(c, y);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  float a, b;
                  f2_unpack(y[i], a, b);
                  a = warp_max_f32(a);
                  b = warp_max_f32(b);
                  if (lane == 2 * i) best = a;
                  if (lane == 2 * i + 1) best = b;
                }
                max_s[(warp & 3) * RW + c + lane] = best;
              }
              named_bar_sync(bar, 128);
              if (t < RW) {
                const float mx = fmaxf(fmaxf(max_s[t], max_s[RW + t]),
                                       fmaxf(max_s[2 * RW + t], max_s[3 * RW + t]));
                float f = 1.f;
                if (t < mine) {
                  const float old = fac_s[t];
                  const bool up = mx > kSeen && mx > old + 32.f;  // (not if mx is NaN: that shows in the sum)
                  if (up) f = ex2(old - mx);
                  set_ref(up ? mx : old);
                }
                fac_s[t] = f;
              }
              choose_near(t < mine ? ref_s[t] : 0.f);
              if (j > 0) {  // what was summed so far
                ok = o_wait(gt - 1);
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < mine; c += 8) {
                  uint32_t a[8];
                  const uint32_t tO = tmem + lane_off + C::COL_O + rb + c;
                  tmem_ld8(tO, a);
#pragma unroll
                  for (int i = 0; i < 8; ++i) a[i] = __float_as_uint(__uint_as_float(a[i]) * fac_s[c + i]);
                  tmem_st8(tO, a);
                }
                tmem_st_wait();
#pragma unroll
                for (int i = 0; i < RW / 2; ++i)
                  sum[i] = f2_mul(sum[i], f2_pack(fac_s[2 * i], fac_s[2 * i + 1]));
              }
              all_logits();
            }
            // P, once the products that read its place are complete
            if (ok && gt >= C::PB) ok = o_wait(gt - C::PB);
            const uint32_t sP = smem_u32(sm + C::OFF_P + (gt % C::PB) * C::PTILE);
#pragma unroll
            for (int c = 0; c < RW; c += 32) {
              if (c > 0 && c >= mine) break;
              uint32_t w[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float a, b;
                f2_unpack(y[c / 2 + i], a, b);
                a = ex2(a);
                b = ex2(b);
                sum[c / 2 + i] = f2_add(sum[c / 2 + i], f2_pack(a, b));
                w[i] = pack_bf16x2(a, b);
              }
              const int r = rb + c;
              const uint32_t at = sP + (r >> 6) * C::PBLK + t * 128;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                st_shared_v4(at + (((((r & 63) >> 3) + i) ^ (t & 7)) << 4), w[4 * i], w[4 * i + 1],
                             w[4 * i + 2], w[4 * i + 3]);
            }
          } else if (ok && gt >= C::PB) {  // a group without rows keeps step: its arrivals count for this tile
            ok = o_wait(gt - C::PB);
          }
          tc_fence_before();
          // values behind the last key: whatever the page holds, they are 0
          if (k0 + 128 > it.lk) {
            const uint32_t v = gt % VS;
            if (ok) ok = warp_wait(v_full + v, (gt / VS) & 1, wd);
            if (ok)
              for (int i = (it.lk - k0) * 8 + tid; i < 1024; i += 256)
#pragma unroll
                for (int c = 0; c < C::DB; ++c)
                  *reinterpret_cast<uint4 *>(sm + C::OFF_V + v * C::TILE + c * C::BLK + i * 16) =
                      make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (ok && lane == 0) {
            mbar_arrive(s_free + buf);
            mbar_arrive(p_ready + (gt & 1));
          }
        }
        g += n;
        // ---- the item's rows: their sums over the threads (beside the last products), then O, whose TMEM
        // lanes are channels. Four lanes trade a 4 x 4 block, after which each has four channels of a row.
        const bool whole = it.begins && it.ends;
        const int which = it.begins ? 1 : 0;
        if (!whole && tid == 0) {
          PartRecord *rec = part_record(p.part, blockIdx.x, which);
          rec->valid = 1;
          rec->ends = it.ends;
          rec->row0 = it.row0;
          rec->hk = it.hk;
          rec->rows = rows;
          rec->pos = (int)blockIdx.x - walk.first_cta(it, stretch_s, &rec->parts);
        }
        if (mine > 0) {
#pragma unroll
          for (int c = 0; c < RW; c += 32) {
            if (c > 0 && c >= mine) break;
            float s[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) f2_unpack(sum[c / 2 + i], s[2 * i], s[2 * i + 1]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)  // lane i ends with row c + i
#pragma unroll
              for (int i = 0; i < o; ++i) {
                const float keep = (lane & o) ? s[i + o] : s[i], give = (lane & o) ? s[i] : s[i + o];
                s[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
              }
            max_s[(warp & 3) * RW + c + lane] = s[0];
          }
          named_bar_sync(bar, 128);
          if (t < mine) {
            const float l = (max_s[t] + max_s[RW + t]) + (max_s[2 * RW + t] + max_s[3 * RW + t]);
            if (whole) {
              fac_s[t] = l == 0.f ? 0.f : 1.0f / l;
              if (p.lse != nullptr)
                p.lse[(size_t)int_s[t].y * p.total_q + it.row0 + (rb + t) / G] =
                    l == 0.f ? -INFINITY : (ref_s[t] + __log2f(l)) * kLn2;
            } else {
              *reinterpret_cast<float2 *>(part_stats<R, D>(p.part, gridDim.x, blockIdx.x, which) +
                                          (rb + t) * 2) = make_float2(l == 0.f ? -INFINITY : ref_s[t], l);
            }
          }
          named_bar_sync(bar, 128);
        }
        if (ok) ok = o_wait(g - 1);
        tc_fence_after();
        const int ch = t & (D - 4), odd = lane & 1, high = lane & 2;
        __nv_bfloat16 *out = p.out + (size_t)it.row0 * p.hq * D + ch;
        float *po = whole ? nullptr : part_rows<R, D>(p.part, gridDim.x, blockIdx.x, which);
#pragma unroll 1
        for (int c = 0; c < mine; c += 16) {
          uint32_t x[16];
          tmem_ld16(tmem + lane_off + C::COL_O + rb + c, x);
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            if (D == 64 && (a & 1) != ((warp >> 1) & 1)) continue;  // (the channels twice: half the rows each)
            const int row = c + 4 * a + (lane & 3);
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(x[4 * a + i]);
            if (whole) {
              const float4 f = *reinterpret_cast<const float4 *>(fac_s + c + 4 * a);
              v[0] *= f.x;
              v[1] *= f.y;
              v[2] *= f.z;
              v[3] *= f.w;
            }
#pragma unroll
            for (int i = 0; i < 4; i += 2) {  // rows i and i + 1: two channels of one of them
              const float got = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], 1);
              const float kept = odd ? v[i + 1] : v[i];
              v[i] = odd ? got : kept;
              v[i + 1] = odd ? kept : got;
            }
            if (whole) {
              const uint32_t w0 = pack_bf16x2(v[0], v[1]), w1 = pack_bf16x2(v[2], v[3]);
              const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? w0 : w1, 2);
              if (row < mine)
                *reinterpret_cast<uint2 *>(out + (size_t)out_s[row] * D) =
                    high ? make_uint2(got, w1) : make_uint2(w0, got);
            } else {
              const float g0 = __shfl_xor_sync(0xffffffffu, high ? v[0] : v[2], 2);
              const float g1 = __shfl_xor_sync(0xffffffffu, high ? v[1] : v[3], 2);
              if (row < mine)
                *part_quad<R>(po, rb + row, ch >> 2) =
                    high ? make_float4(g0, g1, v[2], v[3]) : make_float4(v[0], v[1], g0, g1);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(o_free);
        ok = !named_bar_any(bar, 128, !ok);  // (and out_s has been read: the next item's may be written)
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D, int R>
int launch_t(const PagedParams &p, const fat_paged_cache_t &c, cudaStream_t stream) {
  using C = MidCfg<D, R>;
  PagedParams pp = p;
  CUtensorMap mq, mk, mv;
  const int kbox = std::min(128, 1 << pp.log2_page);
  int rc = make_tmap_pages(&mk, c.k, c, kbox, &pp.head_outer);
  if (!rc) rc = make_tmap_pages(&mv, c.v, c, kbox, &pp.head_outer);
  if (rc) return rc;
  if (make_tmap_rows(&mq, p.q, p.total_q, p.hq, D, p.group, R / p.group)) return FAT_ECUDA;
  const size_t smem = C::bytes(p.bias) + 1024;
  const auto kernel = fat_paged_mid_kernel<D, R>;
  if (prepare_kernel((const void *)kernel, smem, kThreads, C::REGS_NEEDED)) return FAT_ECUDA;
  return launch_dependent("paged tree kernel launch", kernel, dim3((unsigned)paged_tile_ctas()),
                          kThreads, smem, stream, mq, mk, mv, pp);
}

}  // namespace

int launch_paged_mid(const PagedParams &p, const fat_paged_cache_t &c, int rows, cudaStream_t stream) {
  if (c.head_dim == 64) return rows == 64 ? launch_t<64, 64>(p, c, stream) : launch_t<64, 128>(p, c, stream);
  return rows == 64 ? launch_t<128, 64>(p, c, stream) : launch_t<128, 128>(p, c, stream);
}

}  // namespace fat
