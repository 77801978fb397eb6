// fat_linear_ce.cu -- cross-entropy of hidden rows over a vocabulary (the output layer and its loss)
// without keeping the logits, and its gradient.
//
//   z_rv = s h_r . w_v, lse_r = log sum_v exp(z_rv), loss_r = lse_r - z_r,t + zc lse_r^2 (t < 0: 0);
//   with g_r = grad_scale dloss_r: dz_rv = g_r (exp(z_rv - lse_r) (1 + 2 zc lse_r) - [v == t_r]),
//   dh = s dz W, dw = s dz^T H.
//
// The logits exist only as accumulators in tensor memory. Forward: tiles of 256 rows x up to 256
// vocabulary entries; the epilogue leaves the maximum and sum of exponentials of each half of a tile's row
// (8 bytes for up to 128 logits), which a second grid merges. Backward: the vocabulary in pieces; a
// piece's logits are computed again, their gradient goes to the workspace in bf16, and two products take
// it from there: dh += dz W and dw = dz^T H. (One bf16 a value: most gradients are 0.0022 to 0.0025 off in
// the mean where the results' own rounding gives 0.0017; two would double the products.) dz is kept without
// grad_scale and s, which scale the results: bf16 holds the large entries, p - 1 at the targets, best when
// they are next to 1 (with 1 / rows in them all of them round the same way, and so do the results: 251 rows
// 0.0038 off against 0.0017). A launch does the products of one piece and the logits of the next, so that
// its last wave is filled with short tiles.
// Bound by the tensor cores (2, 4 and 2 N V D operations in the three products, 2 in the loss) from some
// 300 rows on, below that by the read of the weights (and the write of their gradient).
//
// One kernel does all products: pairs of CTAs on two SMs, one tcgen05 product of 256 x 256 x 16 for both
// (cta_group::2: each CTA stages half of the rows and half of the columns, so a stage is 32 KB a CTA for
// the work of 64 KB), persistent over a list of tiles:
//   warps 0-7  epilogue, a row (TMEM lane) per thread, each warpgroup half of the columns; two accumulators,
//              so a tile's epilogue runs beside the next tile's products;
//   warp 8     producer: boxes of 64 x 64 elements by TMA, 128-byte swizzle; the same boxes serve
//              operands whose reduction runs along their rows (K-major: hidden rows and weights of the logits,
//              dz of dh) or across them (MN-major: weights of dh, dz and hidden rows of dw);
//   warp 9     issues the products (the pair's first CTA).
// Up to 128 rows (scores of drafted tokens) the weights are the tall side instead: 256 vocabulary entries x
// the rows, a stage holds little but weights, and more of them are on their way.
#include <algorithm>
#include <cstdint>

#include "../../include/fat_attn_debug.h"
#include "fat_attn_internal.cuh"

namespace fat {
namespace {

constexpr int kThreads = 320;
constexpr int kEpiWarps = 8, kWarpProd = 8, kWarpMma = 9;
constexpr int kHalf = 128 * 128;          // one operand's half of a stage: 128 rows x 64 bf16
constexpr int kBuf = 32 * 128;            // staged output of a warp: 32 rows x 128 bytes
constexpr int kTile = 256;                // rows and columns of a pair's tile
constexpr int kColStep = 32;              // a pair's product of 256 rows has 32, 64, .. 256 columns
constexpr int kFewHeadRows = 128;         // forward calls of at most so many rows take the few-row form
constexpr int kMaxPairs = 128;
static_assert(kTile % kColStep == 0 && kFewHeadRows % kColStep == 0, "columns of a product");

// The kernel's forms, and what each has in shared memory.
enum Mode { kForward, kBackward, kFew, kLong };
// The tensor cores cut off what a sum loses at every step, towards zero. The loss adds up at most kChunk
// blocks of 64 channels there, and further ones in fp32 with rounding: kLong is the forward of more
// channels, whose epilogue keeps a tile's logits in registers (lse against 64 bits, 3808 channels: 1.9e-6
// without, 3.5e-7 with; 1024 channels 3.5e-7).
constexpr int kChunk = 16;
template <int MODE>
struct HeadCfg {
  static constexpr int STAGES = MODE == kFew ? 10 : 6;  // at most
  static constexpr int OFF_BUF = MODE == kFew ? 186 * 1024 : STAGES * 2 * kHalf;
  // backward: an output buffer a warp; few rows: targets, and 32 rows of logits a warpgroup
  static constexpr int LD = 132;  // floats from row to row of these
  static constexpr int OFF_ROWS = OFF_BUF + kFewHeadRows * 4;
  static constexpr int OFF_BAR = MODE == kBackward ? OFF_BUF + kEpiWarps * kBuf
                                 : MODE == kFew    ? OFF_ROWS + 2 * 32 * LD * 4
                                                   : OFF_BUF;
  static constexpr int SMEM = OFF_BAR + 320 + 1024;
  static_assert((2 * STAGES + 5) * 8 + 8 <= 320, "barrier block");
  static_assert(SMEM <= kSmemLimit, "shared memory");
};

enum Kind { kLogits, kProb, kDx, kDw };

struct HeadParams {
  int rows, vocab, dim;
  float sl2;               // logit scale in log2 units
  int pairs;               // CTA pairs of the grid
  int bn;                  // columns of a logits tile
  int row_tiles, col_tiles;
  int row_group;           // forward: row tiles that walk the vocabulary together
  // forward
  int stages, stage_bytes; // few rows: stages and their size
  float2 *part;            // [2 col_tiles][rows]: maximum (log2 units), sum (of each half of a tile)
  float *zt;               // [rows]: the target's logit
  const int32_t *target;
  float scale;
  // backward: products of one piece (dz in P, vocabulary entries from v0 on, rows from r0 on)
  int n_dw, n_dx, n_prob;
  int d_tiles, dx_splits, dx_kb;  // dx_kb: k blocks of a split
  int p_kb, r_kb;                 // k blocks of the piece's vocabulary and of its rows
  int v0, r0;
  int dx_add, dw_add;             // add to what the piece before left (fp32)
  int dx_f32, dw_f32;
  float out_scale;                // of results in bf16
  int dx_rows;                    // rows of a split's partial dh
  int dx_first;                   // dh's tiles take longer than dw's: they come first
  // logits of the next piece: pair q takes tiles prob_first[q] up to prob_first[q + 1] behind the others
  int pv0, pr0, prow_tiles;
  uint16_t prob_first[kMaxPairs + 1];
  const float4 *rec;       // [rows, padded]: lse (log2 units), factor, subtracted at the target, target
  int *err;
  long long timeout_ns;
  int debug_flags;
};

template <int N>
struct Threads {
  static constexpr int value = N;
};

struct Job {
  int kind, m0, n0;  // first row and column (of the pair's tile)
  int k0, k1;        // k blocks
  int split;
};

// Tile i of a pair. Forward: dealt in turns. Backward: the products' tiles in alternating turns (the longer
// kind first), then the pair's share of the next piece's logits, which evens out what the turns left.
template <int MODE>
__device__ __forceinline__ bool job_at(const HeadParams &p, int pair, int i, Job &o) {
  o.split = 0;
  o.k0 = 0;
  if (MODE != kBackward) {
    const int j = pair + i * p.pairs;
    if (j >= p.row_tiles * p.col_tiles) return false;
    const int per = p.row_group * p.col_tiles, g = j / per, rest = j - g * per;
    const int cnt = min(p.row_group, p.row_tiles - g * p.row_group);
    const int v = rest / cnt;
    o.kind = kLogits;
    o.m0 = (g * p.row_group + rest - v * cnt) * kTile;
    o.n0 = v * p.bn;
    o.k1 = (p.dim + 63) >> 6;
    return true;
  }
  const int longs = p.n_dw + p.n_dx, full = longs / p.pairs;
  int j = i * p.pairs + ((i & 1) ? p.pairs - 1 - pair : pair);
  const int mine = full + (full * p.pairs + ((full & 1) ? p.pairs - 1 - pair : pair) < longs ? 1 : 0);
  if (i >= mine) {
    j = p.prob_first[pair] + i - mine;
    if (j >= p.prob_first[pair + 1]) return false;
    const int v = j / p.prow_tiles;
    o.kind = kProb;
    o.m0 = (j - v * p.prow_tiles) * kTile;
    o.n0 = v * kTile;
    o.k1 = (p.dim + 63) >> 6;
    return true;
  }
  bool dx = p.dx_first;
  const int first = dx ? p.n_dx : p.n_dw;
  if (j >= first) {
    j -= first;
    dx = !dx;
  }
  // (a pair's turns meet all channel tiles alike: the last one is cheaper)
  const int rest = j / p.d_tiles, d = (j + rest) % p.d_tiles;
  o.n0 = d * kTile;
  if (dx) {
    o.kind = kDx;
    o.split = rest % p.dx_splits;
    o.m0 = rest / p.dx_splits * kTile;
    o.k0 = o.split * p.dx_kb;
    o.k1 = min(o.k0 + p.dx_kb, p.p_kb);
  } else {
    o.kind = kDw;
    o.m0 = rest * kTile;  // within the piece
    o.k1 = p.r_kb;
  }
  return true;
}
// Columns of a tile of dh or dw: 256, of the last one 128 where they do.
__device__ __forceinline__ int d_cols(const HeadParams &p, int n0) {
  return p.dim - n0 <= 128 ? 128 : 256;
}

// ---- what the pair needs beyond sm103_ptx.cuh -----------------------------------------------------
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// shared-memory address of the pair's first CTA
__device__ __forceinline__ uint32_t in_first(const void *p) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity, uint32_t hint_ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(hint_ns)
      : "memory");
  return ok != 0;
}
// mbar_wait for barriers that the other CTA of the pair arrives on too
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, const Watchdog &wd) {
  if (try_wait_cluster(bar, parity, 20000u)) return true;
  const uint64_t t0 = global_timer_ns();
  uint32_t spins = 0;
  while (true) {
    if (try_wait_cluster(bar, parity, 20000u)) return true;
    if ((++spins & 63u) == 0) {
      if (*wd.abort_flag) return false;
      if ((long long)(global_timer_ns() - t0) > wd.timeout_ns) {
        *wd.abort_flag = 1;
        atomicOr(wd.err_word, wd.err_bit);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool warp_wait_cluster(uint64_t *bar, uint32_t parity,
                                                  const Watchdog &wd) {
  return __all_sync(0xffffffffu, wait_cluster(bar, parity, wd));
}
// a box into this CTA's shared memory, counted on a barrier of the pair's first CTA
__device__ __forceinline__ void load_pair(const CUtensorMap *map, uint32_t bar, uint32_t dst, int x,
                                          int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap *map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void add_box(const CUtensorMap *map, uint32_t src, int x, int y) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(src)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrive on the barrier at this place in both CTAs (ctas: a bit each) when the products so far are complete
__device__ __forceinline__ void commit_pair(uint64_t *bar, uint16_t ctas = 3) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
      ::"r"(smem_u32(bar)),
      "h"(ctas)
      : "memory");
}

__device__ __forceinline__ void keep_below(uint32_t (&x)[32], int lim, float v) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i >= lim) x[i] = __float_as_uint(v);
}

// A warp's 32 rows x 128 bytes to global memory through its staging buffer.
struct Staged {
  uint32_t buf;
  int lane;
  __device__ void wait() {  // the copy before has read the buffer
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
  }
  __device__ void put(int chunk, uint32_t x, uint32_t y, uint32_t z, uint32_t w) const {
    st_shared_v4(buf + lane * 128 + ((chunk ^ (lane & 7)) << 4), x, y, z, w);
  }
  __device__ void send(const CUtensorMap *map, bool add, int x, int y) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (add)
        add_box(map, buf, x, y);
      else
        store_box(map, buf, x, y);
      bulk_commit_group();
    }
  }
};

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fat_head_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_p,      // dz of this piece, read
                    const __grid_constant__ CUtensorMap tm_pnext,  // dz of the next, written
                    const __grid_constant__ CUtensorMap tm_dx,
                    const __grid_constant__ CUtensorMap tm_dw,
                    const __grid_constant__ HeadParams p) {
  using C = HeadCfg<MODE>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cta_rank(), pair = blockIdx.x >> 1;
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR);  // of the first CTA
  uint64_t *empty = full + C::STAGES;                              // of each CTA
  uint64_t *acc_full = empty + C::STAGES;                          // [2] of each CTA
  uint64_t *acc_empty = acc_full + 2;                              // [2] of the first CTA
  uint64_t *done = acc_empty + 2;                                  // of the first CTA
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int stages = MODE == kFew ? p.stages : C::STAGES;
  const int stage_bytes = MODE == kFew ? p.stage_bytes : 2 * kHalf;
  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full + a, 1);
      mbar_init(acc_empty + a, 2 * kEpiWarps);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpProd && lane == 0) {
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w);
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Watchdog wd{abort_flag, p.err, MODE == kBackward ? FAT_DEVERR_TIMEOUT_BWD : FAT_DEVERR_TIMEOUT_FWD,
                    p.timeout_ns};
  grid_dep_wait();

  if (warp == kWarpProd) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      int slot = 0;
      uint32_t phase = 1;
      bool ok = !(p.debug_flags & 1);  // test hook: no copies, the waits run out
      Job job;
      for (int i = 0; ok && job_at<MODE>(p, pair, i, job); ++i) {
        const int kind = job.kind;
        // rows of this CTA's half of the second operand
        const int bhalf = MODE != kBackward ? p.bn >> 1 : kind == kProb ? 128 : d_cols(p, job.n0) >> 1;
        for (int k = job.k0; k < job.k1; ++k) {
          if (!(ok = mbar_wait(empty + slot, phase, wd))) break;
          const uint32_t a = smem_u32(sm) + slot * stage_bytes, b = a + kHalf;
          const uint32_t bar = in_first(full + slot);
          if (rank == 0) mbar_arrive_expect_tx(full + slot, 2 * (kHalf + bhalf * 128));
          const int m = job.m0 + rank * 128, n = job.n0 + rank * bhalf;
          if (MODE == kForward || MODE == kLong) {
            load_pair(&tm_x, bar, a, k * 64, m);  // boxes of 128 and of bn / 2 rows
            load_pair(&tm_w, bar, b, k * 64, n);
          } else if (MODE == kFew) {
            load_pair(&tm_w, bar, a, k * 64, m);
            load_pair(&tm_x, bar, b, k * 64, n);
          } else if (kind == kProb) {
            load_pair(&tm_x, bar, a, k * 64, p.pr0 + m);
            load_pair(&tm_x, bar, a + 8192, k * 64, p.pr0 + m + 64);
            load_pair(&tm_w, bar, b, k * 64, p.pv0 + n);
            load_pair(&tm_w, bar, b + 8192, k * 64, p.pv0 + n + 64);
          } else if (kind == kDx) {
            load_pair(&tm_p, bar, a, k * 64, m);
            load_pair(&tm_p, bar, a + 8192, k * 64, m + 64);
            load_pair(&tm_w, bar, b, n, p.v0 + k * 64);
            if (bhalf == 128) load_pair(&tm_w, bar, b + 8192, n + 64, p.v0 + k * 64);
          } else {
            load_pair(&tm_p, bar, a, m, k * 64);
            load_pair(&tm_p, bar, a + 8192, m + 64, k * 64);
            load_pair(&tm_x, bar, b, n, p.r0 + k * 64);
            if (bhalf == 128) load_pair(&tm_x, bar, b + 8192, n + 64, p.r0 + k * 64);
          }
          if (++slot == stages) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      // every stage's last use has been released: nothing arrives here after this CTA has ended
      for (int i = 0; ok && i < stages; ++i) {
        ok = mbar_wait(empty + slot, phase, wd);
        if (++slot == stages) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (*abort_flag) {  // copies may still be on their way: give them time to land
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) __nanosleep(1000);
      }
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------------ products
    if (rank == 0 && lane == 0) {
      int slot = 0;
      uint32_t phase = 0, n = 0;
      bool ok = true;
      Job job;
      for (int i = 0; ok && job_at<MODE>(p, pair, i, job); ++i) {
        const bool a_mn = MODE == kBackward && job.kind == kDw, b_mn = MODE == kBackward && job.kind >= kDx;
        const int cols = MODE != kBackward ? p.bn : b_mn ? d_cols(p, job.n0) : 256;
        const uint32_t idesc = idesc_bf16_f32(256, cols, a_mn ? 1 : 0, b_mn ? 1 : 0);
        const uint32_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
        for (int k0 = job.k0; ok && k0 < job.k1; ++n) {  // an accumulator's share of the reduction
          const int k1 = MODE == kFew || MODE == kLong ? min(k0 + kChunk, job.k1) : job.k1;
          const uint32_t d = tmem + 256 * (n & 1);
          if (n >= 2 && !(ok = wait_cluster(acc_empty + (n & 1), (n / 2 - 1) & 1, wd))) break;
          tc_fence_after();
          for (int k = k0; k < k1; ++k) {
            if (!(ok = wait_cluster(full + slot, phase, wd))) break;
            tc_fence_after();
            const uint32_t a = smem_u32(sm) + slot * stage_bytes;
            const uint64_t da = sw128_desc(a, a_mn ? 8192 : 16, 1024);
            const uint64_t db = sw128_desc(a + kHalf, b_mn ? 8192 : 16, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_pair(d, da + kk * a_step, db + kk * b_step, idesc, k > k0 || kk > 0);
            commit_pair(empty + slot);
            if (++slot == stages) {
              slot = 0;
              phase ^= 1;
            }
          }
          commit_pair(acc_full + (n & 1));
          k0 = k1;
        }
      }
      commit_pair(done, 1);
      mbar_wait_teardown(done, 0, kTeardownNs);
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int half = warp >> 2;  // of the columns
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const int row_in = rank * 128 + (warp & 3) * 32;  // the warp's first row of the pair's tile
    Staged st{smem_u32(sm + C::OFF_BUF + warp * kBuf), lane};
    int *target_s = reinterpret_cast<int *>(sm + C::OFF_BUF);
    float *rows_s = reinterpret_cast<float *>(sm + C::OFF_ROWS) + half * 32 * C::LD;
    if (MODE == kFew) {
      const int t = tid & 127;  // each warpgroup its own rows' targets
      if (t < kFewHeadRows / 2) {
        const int r = half * (p.bn >> 1) + t;
        target_s[half * (kFewHeadRows / 2) + t] = t < p.bn >> 1 && r < p.rows ? __ldg(p.target + r) : -1;
      }
      target_s += half * (kFewHeadRows / 2);
      named_bar_sync(1 + half, 128);
    }
    uint32_t n = 0;  // accumulators so far
    bool ok = true;
    Job job;
    for (int i = 0; ok && job_at<MODE>(p, pair, i, job); ++i, ++n) {
      uint32_t d = tmem + lane_off + 256 * (n & 1);
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(in_first(acc_empty + (n & 1)));
      };
      if constexpr (MODE == kForward) {
        const int row = job.m0 + row_in + lane;
        const int t = row < p.rows ? __ldg(p.target + row) : -1;
        // this warpgroup's columns
        const int c0 = 128 * half, lim = min(min(p.bn, p.vocab - job.n0), c0 + 128);
        if (!(ok = warp_wait_cluster(acc_full + (n & 1), (n / 2) & 1, wd))) break;
        tc_fence_after();
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        for (int c = c0; c < lim; c += 32) {
          uint32_t x[32];
          tmem_ld32(d + c, x);
          if (c + 32 > lim) keep_below(x, lim - c, -INFINITY);
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            mx[(i >> 1) & 3] =
                fmax3(mx[(i >> 1) & 3], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
        }
        const float m = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * p.sl2;
        const float m_use = m == -INFINITY ? 0.f : m;
        const uint64_t sl = f2_pack(p.sl2, p.sl2), neg = f2_pack(-m_use, -m_use);
        uint64_t sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
        for (int c = c0; c < lim; c += 32) {
          uint32_t x[32];
          tmem_ld32(d + c, x);
          const int at = t - job.n0 - c;
          if (__any_sync(0xffffffffu, at >= 0 && at < 32)) {
            float zt = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i == at) zt = __uint_as_float(x[i]);
            if (at >= 0 && at < 32 && at < lim - c) p.zt[row] = zt * p.scale;
          }
          if (c + 32 > lim) keep_below(x, lim - c, -INFINITY);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float a, b;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), sl, neg), a, b);
            sum[(i >> 1) & 1] = f2_add(sum[(i >> 1) & 1], f2_pack(ex2(a), ex2(b)));
          }
        }
        release();
        float s0, s1;
        f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
        if (row < p.rows)
          p.part[(size_t)(2 * (job.n0 / p.bn) + half) * p.rows + row] = make_float2(m, s0 + s1);
      } else if constexpr (MODE == kLong) {
        // the same with the logits in registers, summed over the accumulators
        const int row = job.m0 + row_in + lane;
        const int t = row < p.rows ? __ldg(p.target + row) : -1;
        const int c0 = 128 * half, lim = min(p.bn, p.vocab - job.n0) - c0;
        uint64_t z[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) z[c] = 0;
        for (int k = job.k0;;) {
          if (!(ok = warp_wait_cluster(acc_full + (n & 1), (n / 2) & 1, wd))) break;
          tc_fence_after();
          d = tmem + lane_off + 256 * (n & 1) + c0;
#pragma unroll
          for (int c = 0; c < 128; c += 16) {
            if (c >= lim) break;
            uint32_t x[16];
            tmem_ld16(d + c, x);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              z[c / 2 + i] = f2_add(z[c / 2 + i],
                                    f2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])));
          }
          release();
          k += kChunk;
          if (k >= job.k1) break;
          ++n;
        }
        if (!ok) break;
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
          float a, b;
          f2_unpack(z[c / 2], a, b);
          if (c + 2 > lim) {
            a = c < lim ? a : -INFINITY;
            b = -INFINITY;
            z[c / 2] = f2_pack(a, b);
          }
          mx = fmax3(mx, a, b);
        }
        const float m = mx * p.sl2, m_use = m == -INFINITY ? 0.f : m;
        const uint64_t sl = f2_pack(p.sl2, p.sl2), neg = f2_pack(-m_use, -m_use);
        const int at = t - job.n0 - c0;
        if (__any_sync(0xffffffffu, at >= 0 && at < 128 && at < lim)) {
          float zt = 0.f;
#pragma unroll
          for (int c = 0; c < 128; c += 2) {
            float a, b;
            f2_unpack(z[c / 2], a, b);
            if (at == c) zt = a;
            if (at == c + 1) zt = b;
          }
          if (at >= 0 && at < 128 && at < lim) p.zt[row] = zt * p.scale;
        }
        uint64_t sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          float a, b;
          f2_unpack(f2_fma(z[c], sl, neg), a, b);
          sum[c & 1] = f2_add(sum[c & 1], f2_pack(ex2(a), ex2(b)));
        }
        float s0, s1;
        f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
        if (row < p.rows)
          p.part[(size_t)(2 * (job.n0 / p.bn) + half) * p.rows + row] = make_float2(m, s0 + s1);
      } else if constexpr (MODE == kFew) {
        // A thread holds a vocabulary entry's logits of this warpgroup's rows, and passes them on through
        // shared memory to the threads that share a row: its statistics over the CTA's 128 entries.
        const int r0 = half * (p.bn >> 1), nr = min(p.rows - r0, p.bn >> 1);
        const int t = tid & 127, v0 = job.m0 + rank * 128;
        const bool in = v0 + t < p.vocab;
        float x[2][32];
        for (int k = job.k0;;) {
          if (ok) ok = warp_wait_cluster(acc_full + (n & 1), (n / 2) & 1, wd);
          tc_fence_after();
          d = tmem + lane_off + 256 * (n & 1) + r0;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (32 * c >= nr) break;
            uint32_t y[32];
            tmem_ld32(d + 32 * c, y);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              x[c][i] = k > job.k0 ? x[c][i] + __uint_as_float(y[i]) : __uint_as_float(y[i]);
          }
          release();
          k += kChunk;
          if (k >= job.k1) break;
          ++n;
        }
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          if (c >= nr) break;
          const int cnt = min(nr - c, 32);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < cnt) rows_s[i * C::LD + t] = in ? x[c / 32][i] : -INFINITY;
          named_bar_sync(1 + half, 128);
          auto row_stats = [&](auto threads) {  // `threads` of them a row
            constexpr int TR = decltype(threads)::value, N = 128 / TR;
            const int r = t / TR, part = t % TR;
            float y[N], mx = -INFINITY, e = 0.f;
#pragma unroll
            for (int k = 0; k < N / 4; ++k) {
              const float4 q = *reinterpret_cast<const float4 *>(rows_s + r * C::LD + 4 * (part + TR * k));
              y[4 * k] = q.x;
              y[4 * k + 1] = q.y;
              y[4 * k + 2] = q.z;
              y[4 * k + 3] = q.w;
            }
#pragma unroll
            for (int k = 0; k < N; ++k) mx = fmaxf(mx, y[k]);
#pragma unroll
            for (int o = 1; o < TR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float m = mx * p.sl2, use = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int k = 0; k < N; ++k) e += ex2(fmaf(y[k], p.sl2, -use));
#pragma unroll
            for (int o = 1; o < TR; o <<= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
            if (part == 0 && r < cnt) {
              const int row = r0 + c + r, at = target_s[c + r] - v0;
              p.part[(size_t)(2 * (job.m0 / kTile) + rank) * p.rows + row] = make_float2(m, e);
              if (at >= 0 && at < 128 && v0 + at < p.vocab) p.zt[row] = rows_s[r * C::LD + at] * p.scale;
            }
          };
          if (cnt <= 8)
            row_stats(Threads<16>{});
          else
            row_stats(Threads<4>{});
          named_bar_sync(1 + half, 128);
        }
        // (the warps meet at barriers: after a wait that ran out they leave together)
        ok = !named_bar_any(1 + half, 128, !ok);
      } else {
        float4 rec = make_float4(0.f, 0.f, 0.f, 0.f);
        if (job.kind == kProb) rec = __ldg(p.rec + p.pr0 + job.m0 + row_in + lane);
        if (!(ok = warp_wait_cluster(acc_full + (n & 1), (n / 2) & 1, wd))) break;
        tc_fence_after();
        const int c0 = 128 * half;
        if (job.kind == kProb) {
          const int lim = p.vocab - (p.pv0 + job.n0);
          const int t = __float_as_int(rec.w) - (p.pv0 + job.n0);
          const uint64_t sl = f2_pack(p.sl2, p.sl2), neg = f2_pack(-rec.x, -rec.x);
          const uint64_t f = f2_pack(rec.y, rec.y);
#pragma unroll 1
          for (int c = c0; c < c0 + 128; c += 64) {
            uint32_t x[2][32];
            tmem_ld32_issue(d + c, x[0]);
            tmem_ld32_issue(d + c + 32, x[1]);
            tmem_ld32_fence(x[0]);
            tmem_ld32_fence(x[1]);
            st.wait();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float y[32];
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                float u, v;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(x[h][i]), __uint_as_float(x[h][i + 1])), sl,
                                 neg), u, v);
                f2_unpack(f2_mul(f2_pack(ex2(u), ex2(v)), f), y[i], y[i + 1]);
              }
              const int at = t - c - 32 * h;
              if (__any_sync(0xffffffffu, at >= 0 && at < 32)) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (i == at) y[i] -= rec.z;
              }
              if (c + 32 * h + 32 > lim) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (c + 32 * h + i >= lim) y[i] = 0.f;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
                st.put(4 * h + i, pack_bf16x2(y[8 * i], y[8 * i + 1]),
                       pack_bf16x2(y[8 * i + 2], y[8 * i + 3]), pack_bf16x2(y[8 * i + 4], y[8 * i + 5]),
                       pack_bf16x2(y[8 * i + 6], y[8 * i + 7]));
            }
            st.send(&tm_pnext, false, job.n0 + c, job.m0 + row_in);
          }
        } else {
          const bool dx = job.kind == kDx;
          const CUtensorMap *map = dx ? &tm_dx : &tm_dw;
          const bool f32 = dx ? p.dx_f32 : p.dw_f32, add = dx ? p.dx_add : p.dw_add;
          // rows: of dh (its split's partial), or the vocabulary's entries
          const int y = (dx ? job.split * p.dx_rows + (p.dx_f32 ? 0 : p.r0) : p.v0) + job.m0 + row_in;
          const int cols = min(c0 + 128, p.dim - job.n0);
          const int step = f32 ? 32 : 64;
#pragma unroll 1
          for (int c = c0; c < cols; c += step) {
            st.wait();
            uint32_t x[32];
            if (f32) {
              tmem_ld32(d + c, x);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                st.put(i, x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                tmem_ld32(d + c + 32 * h, x);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  uint32_t w[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    w[k] = pack_bf16x2(__uint_as_float(x[8 * i + 2 * k]) * p.out_scale,
                                       __uint_as_float(x[8 * i + 2 * k + 1]) * p.out_scale);
                  st.put(4 * h + i, w[0], w[1], w[2], w[3]);
                }
              }
            }
            st.send(map, add, job.n0 + c, y);
          }
        }
        release();
      }
    }
    if (MODE == kBackward && lane == 0) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  grid_dep_launch();
  cluster_sync();
  if (warp == kWarpMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ---- statistics of the tiles to lse and loss --------------------------------------------------------
// RB rows a block, 256 / RB threads a row, each a share of the halves of tiles.
template <int RB>
__global__ void __launch_bounds__(256) fat_head_merge_kernel(const float2 *part, const float *zt,
                                                             const int32_t *target, int rows,
                                                             int tiles, int vocab, float zc,
                                                             float *loss, float *lse_out, int *err) {
  constexpr int TL = 256 / RB;
  __shared__ float2 red[8][RB];
  grid_dep_launch();
  grid_dep_wait();
  const int r = threadIdx.x % RB, y = threadIdx.x / RB;
  const int row = blockIdx.x * RB + r;
  float m = -INFINITY, s = 0.f;
  auto add = [&](float2 v) {
    const float mn = fmaxf(m, v.x), ref = mn == -INFINITY ? 0.f : mn;
    s = s * ex2(m - ref) + v.y * ex2(v.x - ref);
    m = mn;
  };
  if (row < rows) {
    constexpr int U = 8;  // loads in flight
    for (int t0 = y; t0 < tiles; t0 += U * TL) {
      float2 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * TL;
        v[u] = t < tiles ? __ldg(part + (size_t)t * rows + row) : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) add(v[u]);
    }
  }
#pragma unroll
  for (int o = RB; o < 32; o <<= 1)  // over the lanes of the row, then over the warps
    add(make_float2(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o)));
  if ((threadIdx.x & 31) < RB) red[threadIdx.x >> 5][r] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x >= RB || row >= rows) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) add(red[i][r]);
  const float lse = m * kLn2 + logf(s);
  const int t = __ldg(target + row);
  if (t >= vocab) atomicOr(err, FAT_DEVERR_INDEX);
  if (lse_out != nullptr) lse_out[row] = lse;
  if (loss != nullptr) loss[row] = t >= 0 && t < vocab ? lse - zt[row] + zc * lse * lse : 0.f;
}

// ---- backward: the rows' records, hidden rows without the ignored ones' values ------------------------
// A warp per row. Ignored rows (and those that pad the last tile) count nothing, whatever they hold: their
// values are 0 in the copy, for 0 * NaN would reach dw.
__global__ void __launch_bounds__(256)
    fat_head_rows_kernel(const uint4 *hidden, long long stride16, const int32_t *target,
                         const float *lse, const float *dloss, float zc, int rows, int padded,
                         int vocab, int chunks, int pitch16, uint4 *copy,
                         float4 *rec, int *err) {
  grid_dep_launch();
  grid_dep_wait();
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= padded) return;
  const int t = row < rows ? __ldg(target + row) : -1;
  const bool counts = t >= 0 && t < vocab;
  if (lane == 0) {
    float4 r = make_float4(INFINITY, 0.f, 0.f, __int_as_float(-1));
    if (t >= vocab) atomicOr(err, FAT_DEVERR_INDEX);
    if (counts) {
      const float l = __ldg(lse + row);
      const float g = dloss ? __ldg(dloss + row) : 1.f;
      r = make_float4(l * kLog2e, g * (1.f + 2.f * zc * l), g, __int_as_float(t));
    }
    rec[row] = r;
  }
  if (row >= rows) return;
  for (int c = lane; c < chunks; c += 32)
    copy[(size_t)row * pitch16 + c] =
        counts ? __ldg(hidden + row * stride16 + c) : make_uint4(0u, 0u, 0u, 0u);
}

// rows of `chunks` 16-byte pieces, source_pitch and pitch of them apart
__global__ void __launch_bounds__(256) fat_head_copy_kernel(const uint4 *src, long long source_pitch,
                                                            long long n, int chunks, int pitch, uint4 *dst) {
  grid_dep_launch();
  grid_dep_wait();
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
    const long long row = i / chunks;
    const int c = (int)(i - row * chunks);
    dst[row * pitch + c] = __ldg(src + row * source_pitch + c);
  }
}

// dst = bf16(scale * sum of the parts), eight values a thread
__global__ void __launch_bounds__(256) fat_head_sum_kernel(const float4 *part, long long n8, int parts,
                                                           long long part_stride4, float scale, uint4 *dst) {
  grid_dep_launch();
  grid_dep_wait();
  const long long i = blockIdx.x * 256ll + threadIdx.x;
  if (i >= n8) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
  for (int q = 0; q < parts; ++q) {
    const float4 x = __ldg(part + q * part_stride4 + 2 * i), y = __ldg(part + q * part_stride4 + 2 * i + 1);
    a.x += x.x;
    a.y += x.y;
    a.z += x.z;
    a.w += x.w;
    b.x += y.x;
    b.y += y.y;
    b.z += y.z;
    b.w += y.w;
  }
  dst[i] = make_uint4(pack_bf16x2(a.x * scale, a.y * scale), pack_bf16x2(a.z * scale, a.w * scale),
                      pack_bf16x2(b.x * scale, b.y * scale), pack_bf16x2(b.z * scale, b.w * scale));
}

// ---- host -----------------------------------------------------------------------------------------------
bool odd(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }
size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }
int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

int check(const fat_linear_ce_shape_t *s) {
  if (!s) return FAT_EINVAL_NULL;
  if (s->rows < 0 || s->vocab <= 0 || s->dim <= 0 || s->dim % 8 || s->hidden_stride % 8 ||
      s->weight_stride % 8 || s->hidden_stride < s->dim || s->weight_stride < s->dim ||
      s->hidden_stride >= (1LL << 38) || s->weight_stride >= (1LL << 38))
    return FAT_EINVAL_SHAPE;
  if (!(s->logit_scale > 0.f) || !(s->logit_scale < INFINITY) || !(s->z_loss >= 0.f) ||
      !(s->z_loss < INFINITY))
    return FAT_EINVAL_SHAPE;
  if (s->dim > 65536 || s->vocab > (1 << 28) || s->rows > (1 << 28) ||
      (long long)ceil_div(s->rows, kTile) * ceil_div(s->vocab, 16) > (1 << 30))
    return FAT_EUNSUPPORTED;
  return FAT_OK;
}

template <int MODE>
bool head_ready() {
  return prepare_kernel((const void *)fat_head_kernel<MODE>, HeadCfg<MODE>::SMEM, kThreads, 0) == 0;
}
// Pairs of CTAs that run at once (0: no device)
int head_pairs() {
  if (!head_ready<kForward>() || !head_ready<kBackward>() || !head_ready<kFew>() || !head_ready<kLong>())
    return 0;
  return std::min(kMaxPairs, max_pair_ctas((const void *)fat_head_kernel<kBackward>,
                                           HeadCfg<kBackward>::SMEM, kThreads) / 2);
}

// Forward: tiles of 256 rows x 256 entries, or as many fewer entries as leave the same number of rounds over
// the pairs; up to 128 rows tiles of 256 entries x the rows (widths are multiples of kColStep). Entries
// as the tall side against rows, us: one row, 32768 entries of 512 channels 11.6 / 17.8; 17 rows of 1024
// channels 20.5 / 25.9; 64 20.4 / 20.8.
// Boxes whose rows begin between two 32-byte sectors (rows of an odd number of 16 bytes) are loaded at about
// half the rate: forward calls of many rows copy such hidden rows and weights to rows padded to kCopyPad
// channels (776 channels, 2077 rows and 50021 entries 159 us without, 135 with; 1024 rows and 32768
// entries 54 and 58). The backward's copy of the hidden rows is padded anyway; copying the weights too gained
// and lost up to 6% there.
constexpr int kCopyPad = 64, kCopyRows = 1536;
bool copies_rows(const fat_linear_ce_shape_t *s) { return s->dim % 16 && s->rows >= kCopyRows; }
int copy_pitch(const fat_linear_ce_shape_t *s) { return ceil_div(s->dim, kCopyPad) * kCopyPad; }

struct FwdPlan {
  bool few;
  int bn, row_tiles, col_tiles, parts;
  size_t zt, hidden, weight, bytes;  // hidden, weight: their copies, of calls that make them
};
FwdPlan forward_plan(const fat_linear_ce_shape_t *s, int pairs) {
  FwdPlan f{};
  f.few = s->rows <= kFewHeadRows;
  if (f.few) {
    f.bn = ceil_div(s->rows, kColStep) * kColStep;
    f.row_tiles = ceil_div(s->vocab, kTile);
    f.col_tiles = 1;
  } else {
    const long long rt = f.row_tiles = ceil_div(s->rows, kTile);
    const long long rounds = ceil_div(rt * ceil_div(s->vocab, kTile), pairs);
    f.bn = kTile;
    while (f.bn > kColStep && rt * ceil_div(s->vocab, f.bn - kColStep) <= rounds * pairs)
      f.bn -= kColStep;
    f.col_tiles = ceil_div(s->vocab, f.bn);
  }
  f.parts = 2 * f.row_tiles * f.col_tiles / (f.few ? 1 : f.row_tiles);
  f.zt = round256((size_t)f.parts * s->rows * 8);
  f.bytes = f.hidden = f.weight = f.zt + round256((size_t)s->rows * 4);
  if (copies_rows(s)) {
    f.weight = f.hidden + round256((size_t)s->rows * copy_pitch(s) * 2);
    f.bytes = f.weight + (size_t)s->vocab * copy_pitch(s) * 2;
  }
  return f;
}

// Pieces of the backward: blocks of at most kMaxBlock rows, in each as many vocabulary entries at a time
// as make up kPiece values of dz (two such buffers: one is read while the next is written).
constexpr int kMaxBlock = 16384;
constexpr long long kPiece = 64ll << 20;
struct BwdPlan {
  int block, blocks;     // rows of a block (a multiple of 256) and their number
  int piece, pieces;     // vocabulary entries of a piece (a multiple of 256), pieces of a block
  int splits, split_kb;  // of the vocabulary in dh
  int pitch;             // channels from row to row of the copy of the hidden rows
  bool dx_parts;         // dh goes through fp32 partials
  bool dw_parts;         // and dw
  size_t rec, copy, p[2], dx, dw, bytes;
};
BwdPlan backward_plan(const fat_linear_ce_shape_t *s, int pairs) {
  BwdPlan b{};
  const int padded = ceil_div(s->rows, kTile) * kTile;
  b.blocks = std::max(1, ceil_div(padded, kMaxBlock));
  b.block = ceil_div(ceil_div(padded, b.blocks), kTile) * kTile;
  const int vpad = ceil_div(s->vocab, kTile) * kTile;
  const long long most = std::max<long long>(kTile, kPiece / std::max(b.block, kTile) / kTile * kTile);
  b.pieces = ceil_div(vpad, most);
  b.piece = ceil_div(ceil_div(vpad, b.pieces), kTile) * kTile;
  b.pieces = ceil_div(vpad, b.piece);
  const int d_tiles = ceil_div(s->dim, kTile), kb = ceil_div(std::min(b.piece, s->vocab), 64);
  // dh: tiles with the whole piece as their reduction, cut while the pairs would wait for them
  const long long dx_tiles = (long long)(b.block / kTile) * d_tiles;
  const long long dw_units = (long long)(b.piece / kTile) * d_tiles * (b.block / 64);
  const long long share = (dx_tiles * kb + dw_units) / pairs;
  const int longest = (int)std::max<long long>(16, share / 2);
  b.splits = std::max(1, ceil_div(kb, longest));
  // no more of them than fill their rounds over the pairs
  const long long rounds = std::max<long long>(1, (2 * dx_tiles * b.splits + pairs) / (2 * pairs));
  if (b.splits > 1)
    b.splits = (int)std::max<long long>(1, std::min<long long>(b.splits, rounds * pairs / dx_tiles));
  b.split_kb = ceil_div(kb, b.splits);
  b.splits = ceil_div(kb, b.split_kb);
  b.dx_parts = b.splits > 1 || b.pieces > 1;
  b.dw_parts = b.blocks > 1;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return here;
  };
  b.rec = take((size_t)b.block * b.blocks * 16);
  b.pitch = copy_pitch(s);
  b.copy = take((size_t)s->rows * b.pitch * 2);
  const int buffers = b.pieces * b.blocks > 1 ? 2 : 1;
  for (int i = 0; i < 2; ++i) b.p[i] = i < buffers ? take((size_t)b.block * b.piece * 2) : b.p[0];
  if (b.dx_parts) b.dx = take((size_t)b.splits * b.block * s->dim * 4);
  if (b.dw_parts) b.dw = take((size_t)s->vocab * s->dim * 4);
  b.bytes = at;
  return b;
}

// What every call of at most s->rows rows takes: plans of fewer rows may cut the vocabulary into more
// tiles, pieces or splits than those of more, so each part is counted by a bound that grows with the rows.
size_t forward_bytes(const fat_linear_ce_shape_t *s, int pairs) {
  // statistics: two of 8 bytes a row for each tile; tiles are narrowed within the same rounds over the pairs
  const size_t tiles = (size_t)ceil_div(s->rows, kTile) * ceil_div(s->vocab, kTile) + pairs;
  size_t bytes = round256(tiles * 2 * kTile * 8) + round256((size_t)s->rows * 4);
  if (copies_rows(s))
    bytes += round256((size_t)s->rows * copy_pitch(s) * 2) +
             round256((size_t)s->vocab * copy_pitch(s) * 2);
  return bytes;
}
size_t backward_bytes(const fat_linear_ce_shape_t *s, int pairs) {
  const int d_tiles = ceil_div(s->dim, kTile);
  const long long tiles = ceil_div(s->rows, kTile), blocks = std::max(1, ceil_div(tiles * kTile, kMaxBlock));
  const long long block = std::min<long long>(tiles, kMaxBlock / kTile);
  const long long vpad = ceil_div(s->vocab, kTile) * (long long)kTile;
  // records (a block's last tiles may hold no row) and the copy of the hidden rows
  size_t bytes = round256((size_t)(tiles + blocks - 1) * kTile * 16) +
                 round256((size_t)s->rows * copy_pitch(s) * 2);
  // dz: all of it (of two blocks, as many rows each), or two pieces of up to kPiece values
  const bool one = tiles * kTile * vpad <= kPiece;
  bytes += one ? (size_t)(tiles + (blocks > 1)) * kTile * vpad * 2 : (size_t)kPiece * 4;
  // dh's partials: its tiles, and splits that fill two rounds and a bit over the pairs, of 16 k blocks at least
  const long long most = (long long)block * ceil_div(ceil_div(s->vocab, 64), 16);
  const long long parts = std::min(most, block + 3 * ceil_div(pairs, d_tiles));
  if (!one || parts > block) bytes += round256((size_t)std::max(parts, block) * kTile * s->dim * 4);
  if (blocks > 1) bytes += round256((size_t)s->vocab * s->dim * 4);
  return bytes;
}

// The pairs of a launch and their shares of the next piece's logits: what each one's turns at the products'
// tiles cost is filled up to one level.
void share_tiles(HeadParams &p, int pairs) {
  const int longs = p.n_dw + p.n_dx;
  p.pairs = std::max(1, std::min(pairs, longs + p.n_prob));
  p.dx_first = p.dx_kb > p.r_kb;
  const int per = (p.dim + 63) / 64;  // k blocks of a logits tile
  int load[kMaxPairs] = {0}, most = 0;
  const int first = p.dx_first ? p.n_dx : p.n_dw;
  for (int i = 0, j = 0; j < longs; ++i)
    for (int at = 0; at < p.pairs && j < longs; ++at, ++j) {
      const int cost = (j < first) == (p.dx_first != 0) ? p.dx_kb : p.r_kb;
      int &l = load[i & 1 ? p.pairs - 1 - at : at];
      l += cost;
      most = std::max(most, l);
    }
  auto room = [&](int level, int q) { return level > load[q] ? (level - load[q]) / per : 0; };
  auto total = [&](int level) {
    int n = 0;
    for (int q = 0; q < p.pairs; ++q) n += room(level, q);
    return n;
  };
  // the lowest level up to which all tiles fit; what is too many is left out of pairs that reach it exactly
  int lo = 0, hi = most + per * (p.n_prob / p.pairs + 1);
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (total(mid) >= p.n_prob)
      hi = mid;
    else
      lo = mid + 1;
  }
  int over = total(lo) - p.n_prob, at = 0;
  for (int q = 0; q < p.pairs; ++q) {
    p.prob_first[q] = (uint16_t)at;
    int n = room(lo, q);
    if (over > 0 && n > room(lo - 1, q)) {
      --n;
      --over;
    }
    at += n;
  }
  p.prob_first[p.pairs] = (uint16_t)p.n_prob;
}

// Rows of an odd number of 16 bytes to the workspace, and where they are from there on.
int copy_rows(const fat_linear_ce_shape_t *s, const void **rows, long long *stride, long long n, void *to,
              cudaStream_t stream) {
  if (*stride % 16 == 0) return FAT_OK;
  const int pitch = copy_pitch(s);
  const long long all = n * (s->dim / 8);
  const int blocks = (int)std::min<long long>((all + 255) / 256, 16ll * std::max(sm_count(), 1));
  const int rc = launch_dependent("linear cross-entropy copy launch", fat_head_copy_kernel,
                                  dim3((unsigned)blocks), 256, 0, stream,
                                  static_cast<const uint4 *>(*rows), *stride / 8, all, s->dim / 8, pitch / 8,
                                  static_cast<uint4 *>(to));
  *rows = to;
  *stride = pitch;
  return rc;
}

struct Span {
  const char *lo, *hi;
  Span(const void *p, size_t bytes)
      : lo(static_cast<const char *>(p)), hi(p ? lo + bytes : lo) {}
  bool meets(const Span &o) const { return lo < o.hi && o.lo < hi; }
};
Span rows_span(const void *p, long long rows, long long stride, int dim, int size) {
  return Span(p, rows > 0 ? (size_t)((rows - 1) * stride + dim) * size : 0);
}

}  // namespace
}  // namespace fat

using namespace fat;

extern "C" {

size_t fat_linear_cross_entropy_workspace_size(const fat_linear_ce_shape_t *s, int backward) {
  if (check(s)) return 0;
  const int pairs = head_pairs();
  if (pairs == 0 || s->rows == 0) return 0;
  return backward ? backward_bytes(s, pairs) : forward_bytes(s, pairs);
}

size_t fat_attn_debug_head_workspace(const fat_linear_ce_shape_t *s, int pairs, int backward, size_t *used) {
  if (used) *used = 0;
  if (check(s) || s->rows == 0 || pairs < 1) return 0;
  if (used) *used = backward ? backward_plan(s, pairs).bytes : forward_plan(s, pairs).bytes;
  return backward ? backward_bytes(s, pairs) : forward_bytes(s, pairs);
}

int fat_attn_debug_head_columns(const fat_linear_ce_shape_t *s, int pairs) {
  return check(s) || s->rows == 0 || pairs < 1 ? 0 : forward_plan(s, pairs).bn;
}

int fat_linear_cross_entropy_fwd(const fat_linear_ce_shape_t *s, const void *hidden,
                                 const void *weight, const int32_t *target, void *workspace,
                                 size_t workspace_bytes, float *loss, float *lse) {
  int rc = check(s);
  if (rc) return rc;
  if (s->rows == 0) return FAT_OK;
  if (!hidden || !weight || !target || !workspace) return FAT_EINVAL_NULL;
  if (odd(hidden, 16) || odd(weight, 16) || odd(target, 4) || odd(workspace, 256) || odd(loss, 4) ||
      odd(lse, 4))
    return FAT_EINVAL_SHAPE;
  const int pairs = head_pairs();
  if (pairs == 0) return FAT_ECUDA;
  const FwdPlan f = forward_plan(s, pairs);
  if (workspace_bytes < forward_bytes(s, pairs)) return FAT_EINVAL_SHAPE;
  const Span out[3] = {Span(loss, (size_t)s->rows * 4), Span(lse, (size_t)s->rows * 4),
                       Span(workspace, f.bytes)};
  const Span in[3] = {rows_span(hidden, s->rows, s->hidden_stride, s->dim, 2),
                      rows_span(weight, s->vocab, s->weight_stride, s->dim, 2),
                      Span(target, (size_t)s->rows * 4)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 3; ++j)
      if (out[i].meets(in[j])) return FAT_EINVAL_SHAPE;
    for (int j = i + 1; j < 3; ++j)
      if (out[i].meets(out[j])) return FAT_EINVAL_SHAPE;
  }
  HeadParams p{};
  rc = device_error_address(&p.err);
  if (rc) return rc;
  runtime_knobs(&p.timeout_ns, &p.debug_flags);
  p.rows = s->rows;
  p.vocab = s->vocab;
  p.dim = s->dim;
  p.scale = s->logit_scale;
  p.sl2 = s->logit_scale * kLog2e;
  p.bn = f.bn;
  p.row_tiles = f.row_tiles;
  p.col_tiles = f.col_tiles;
  // row tiles that walk the vocabulary together: their hidden rows stay in L2 (32 MB)
  p.row_group = f.few ? f.row_tiles
                      : std::max(1, std::min<int>(p.row_tiles, (int)((32ll << 20) / (512ll * s->dim))));
  p.pairs = std::min(pairs, p.row_tiles * p.col_tiles);
  p.part = static_cast<float2 *>(workspace);
  p.zt = reinterpret_cast<float *>(static_cast<char *>(workspace) + f.zt);
  p.target = target;
  p.stage_bytes = kHalf + (f.bn / 2 * 128 + 1023) / 1024 * 1024;
  p.stages = std::min<int>(HeadCfg<kFew>::STAGES, HeadCfg<kFew>::OFF_BUF / p.stage_bytes);
  const int half = f.bn / 2;
  const cudaStream_t stream = static_cast<cudaStream_t>(s->stream);
  long long hidden_stride = s->hidden_stride, weight_stride = s->weight_stride;
  if (copies_rows(s)) {
    char *ws = static_cast<char *>(workspace);
    rc = copy_rows(s, &hidden, &hidden_stride, s->rows, ws + f.hidden, stream);
    if (!rc) rc = copy_rows(s, &weight, &weight_stride, s->vocab, ws + f.weight, stream);
    if (rc) return rc;
  }
  CUtensorMap mx, mw;
  if (make_tmap_matrix(&mx, hidden, s->rows, s->dim, hidden_stride, f.few ? half : 128, false) ||
      make_tmap_matrix(&mw, weight, s->vocab, s->dim, weight_stride, f.few ? 128 : half, false))
    return FAT_ECUDA;
  const dim3 grid((unsigned)(2 * p.pairs));
  const bool more = s->dim > kChunk * 64;
  const auto kernel = f.few ? fat_head_kernel<kFew> : more ? fat_head_kernel<kLong> : fat_head_kernel<kForward>;
  rc = launch_dependent("linear cross-entropy launch", kernel, grid, kThreads,
                        f.few ? HeadCfg<kFew>::SMEM : HeadCfg<kForward>::SMEM, stream, mx, mw, mx, mx, mx,
                        mx, p);
  if (rc) return rc;
  // a row's statistics over as many threads as keep the SMs busy
  const auto merge = s->rows < 1024   ? fat_head_merge_kernel<4>
                     : s->rows < 8192 ? fat_head_merge_kernel<8>
                                      : fat_head_merge_kernel<32>;
  const int rb = s->rows < 1024 ? 4 : s->rows < 8192 ? 8 : 32;
  return launch_dependent("linear cross-entropy merge launch", merge, dim3((unsigned)ceil_div(s->rows, rb)),
                          256, 0, stream, p.part, p.zt, target, p.rows, f.parts, p.vocab, s->z_loss, loss,
                          lse, p.err);
}

int fat_linear_cross_entropy_bwd(const fat_linear_ce_shape_t *s, const void *hidden,
                                 const void *weight, const int32_t *target, const float *lse,
                                 const float *dloss, float grad_scale, void *workspace,
                                 size_t workspace_bytes, void *dhidden, void *dweight) {
  int rc = check(s);
  if (rc) return rc;
  const cudaStream_t stream = static_cast<cudaStream_t>(s->stream);
  if (!dhidden && !dweight) return FAT_OK;
  if (odd(dhidden, 16) || odd(dweight, 16)) return FAT_EINVAL_SHAPE;
  if (s->rows == 0) {
    if (dweight) {
      const cudaError_t e = cudaMemsetAsync(dweight, 0, (size_t)s->vocab * s->dim * 2, stream);
      if (e != cudaSuccess) {
        set_last_error("cudaMemsetAsync(dweight)", (int)e, cudaGetErrorString(e));
        return FAT_ECUDA;
      }
    }
    return FAT_OK;
  }
  if (!hidden || !weight || !target || !lse || !workspace) return FAT_EINVAL_NULL;
  if (odd(hidden, 16) || odd(weight, 16) || odd(target, 4) || odd(lse, 4) || odd(dloss, 4) ||
      odd(workspace, 256))
    return FAT_EINVAL_SHAPE;
  const int pairs = head_pairs();
  if (pairs == 0) return FAT_ECUDA;
  const BwdPlan b = backward_plan(s, pairs);
  if (workspace_bytes < backward_bytes(s, pairs)) return FAT_EINVAL_SHAPE;
  const size_t n4 = (size_t)s->rows * 4;
  const Span out[3] = {Span(dhidden, (size_t)s->rows * s->dim * 2),
                       Span(dweight, (size_t)s->vocab * s->dim * 2), Span(workspace, b.bytes)};
  const Span in[5] = {rows_span(hidden, s->rows, s->hidden_stride, s->dim, 2),
                      rows_span(weight, s->vocab, s->weight_stride, s->dim, 2), Span(target, n4),
                      Span(lse, n4), Span(dloss, n4)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 5; ++j)
      if (out[i].meets(in[j])) return FAT_EINVAL_SHAPE;
    for (int j = i + 1; j < 3; ++j)
      if (out[i].meets(out[j])) return FAT_EINVAL_SHAPE;
  }
  HeadParams p{};
  rc = device_error_address(&p.err);
  if (rc) return rc;
  runtime_knobs(&p.timeout_ns, &p.debug_flags);
  char *ws = static_cast<char *>(workspace);
  float4 *rec = reinterpret_cast<float4 *>(ws + b.rec);
  void *copy = ws + b.copy;
  const int padded = b.block * b.blocks;
  rc = launch_dependent("linear cross-entropy rows launch", fat_head_rows_kernel,
                        dim3((unsigned)(padded / 8)), 256, 0, stream,
                        static_cast<const uint4 *>(hidden), (long long)(s->hidden_stride / 8), target,
                        lse, dloss, s->z_loss, s->rows, padded, s->vocab,
                        s->dim / 8, b.pitch / 8, static_cast<uint4 *>(copy), rec, p.err);
  if (rc) return rc;
  p.rows = s->rows;
  p.vocab = s->vocab;
  p.dim = s->dim;
  p.sl2 = s->logit_scale * kLog2e;
  p.rec = rec;
  p.out_scale = grad_scale * s->logit_scale;
  p.d_tiles = ceil_div(s->dim, kTile);
  CUtensorMap mx, mw, mp[2], mps[2], mdx{}, mdw{};
  if (make_tmap_matrix(&mx, copy, s->rows, s->dim, b.pitch, 64, false) ||
      make_tmap_matrix(&mw, weight, s->vocab, s->dim, s->weight_stride, 64, false))
    return FAT_ECUDA;
  for (int i = 0; i < 2; ++i)
    if (make_tmap_matrix(&mp[i], ws + b.p[i], b.block, b.piece, b.piece, 64, false) ||
        make_tmap_matrix(&mps[i], ws + b.p[i], b.block, b.piece, b.piece, 32, false))
      return FAT_ECUDA;
  float *dx_part = reinterpret_cast<float *>(ws + b.dx), *dw_part = reinterpret_cast<float *>(ws + b.dw);
  if (dhidden && (b.dx_parts ? make_tmap_matrix(&mdx, dx_part, (long long)b.splits * b.block, s->dim,
                                                s->dim, 32, true)
                             : make_tmap_matrix(&mdx, dhidden, s->rows, s->dim, s->dim, 32, false)))
    return FAT_ECUDA;
  if (dweight &&
      (b.dw_parts ? make_tmap_matrix(&mdw, dw_part, s->vocab, s->dim, s->dim, 32, true)
                  : make_tmap_matrix(&mdw, dweight, s->vocab, s->dim, s->dim, 32, false)))
    return FAT_ECUDA;
  if (!dhidden) mdx = mx;
  if (!dweight) mdw = mx;
  auto block_rows = [&](int i) { return std::min(b.block, s->rows - i * b.block); };
  auto piece_vocab = [&](int i) { return std::min(b.piece, s->vocab - i * b.piece); };
  const int total = b.blocks * b.pieces;
  for (int q = -1; q < total; ++q) {  // products of piece q, logits of piece q + 1
    const int i = q / b.pieces, c = q % b.pieces;
    p.n_dw = p.n_dx = p.n_prob = 0;
    if (q >= 0) {
      const int rows = block_rows(i), entries = piece_vocab(c);
      p.v0 = c * b.piece;
      p.r0 = i * b.block;
      p.p_kb = ceil_div(entries, 64);
      p.r_kb = ceil_div(rows, 64);
      if (dweight) p.n_dw = ceil_div(entries, kTile) * p.d_tiles;
      p.dx_splits = ceil_div(p.p_kb, b.split_kb);
      p.dx_kb = b.split_kb;
      if (dhidden) p.n_dx = ceil_div(rows, kTile) * p.d_tiles * p.dx_splits;
      p.dx_rows = b.block;
      p.dx_f32 = b.dx_parts;
      p.dw_f32 = b.dw_parts;
      p.dx_add = c > 0;
      p.dw_add = i > 0;
    }
    if (q + 1 < total) {
      const int ni = (q + 1) / b.pieces, nc = (q + 1) % b.pieces;
      p.pv0 = nc * b.piece;
      p.pr0 = ni * b.block;
      p.prow_tiles = ceil_div(block_rows(ni), kTile);
      p.n_prob = p.prow_tiles * ceil_div(piece_vocab(nc), kTile);
    }
    share_tiles(p, pairs);
    rc = launch_dependent("linear cross-entropy backward launch", fat_head_kernel<kBackward>,
                          dim3((unsigned)(2 * p.pairs)), kThreads, HeadCfg<kBackward>::SMEM, stream, mx, mw,
                          mp[q & 1], mps[(q + 1) & 1], mdx, mdw, p);
    if (rc) return rc;
    if (q >= 0 && c == b.pieces - 1 && dhidden && b.dx_parts) {
      const long long n8 = (long long)block_rows(i) * s->dim / 8;
      // every split has been written by the first piece, whose vocabulary is the longest
      rc = launch_dependent("linear cross-entropy sum launch", fat_head_sum_kernel,
                            dim3((unsigned)ceil_div(n8, 256)), 256, 0, stream,
                            reinterpret_cast<const float4 *>(dx_part), n8, b.splits,
                            (long long)b.block * s->dim / 4, p.out_scale,
                            reinterpret_cast<uint4 *>(dhidden) + (long long)i * b.block * s->dim / 8);
      if (rc) return rc;
    }
  }
  if (dweight && b.dw_parts) {
    const long long n8 = (long long)s->vocab * s->dim / 8;
    rc = launch_dependent("linear cross-entropy sum launch", fat_head_sum_kernel,
                          dim3((unsigned)ceil_div(n8, 256)), 256, 0, stream,
                          reinterpret_cast<const float4 *>(dw_part), n8, 1, 0ll, p.out_scale,
                          static_cast<uint4 *>(dweight));
    if (rc) return rc;
  }
  return FAT_OK;
}

}  // extern "C"
