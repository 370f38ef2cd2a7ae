// Tree-masked attention over the 4-bit paged cache for many query rows, on the
// 5th-generation tensor cores (tcgen05).  The few-row kernel, the format and
// the precision choices are described in attention_q4.cu and q4.cuh.
//
// One block = 128 or 256 query rows of one kv head x a run of key-range segments (a
// part of the plan, attention_q4.cuh), each walked in 128-key tiles (8 pages).
// Decoding costs a fixed number of instructions per key, so the more rows share a
// decoded tile the better.
//   warps 0, 3   block ids, and the copies of K's and of V's pages into rings of packed
//                half tiles
//   warp 1       owns TMEM; lane 0 issues every MMA
//   warp 2       with two row tiles tells it when the decoded tiles are there (with one
//                the decoders do)
//   warps 4-7    decode packed tiles to fp16 K and V tiles (128-byte swizzle)
//   warps 8-15   softmax of chain 0, warps 16-23 of chain 1: one TMEM lane (=
//                one query row) per thread, two threads a row (64 keys each)
// Measured (device time): 4 trees of 127 nodes behind 32768 keys, 64 query and 8 kv heads of
// 128: 436 us, 1260 TFLOP/s (67% of the measured bf16 rate; 2900 cycles for the 32 MMAs
// of a tile, 80 each, and their two commits); 16 trees of 16 to 31 nodes behind 512 to 8192
// keys, 32 / 8 heads: 66 us.  There a tile has 16 MMAs and takes 2600 cycles: the
// chain from a tile's S through the release of its stage, the decoding of the tile
// two further (some 2000 cycles for a pair of warps), its hand-over and its MMAs. Four
// warps for K and four for V (896 threads, smaller register shares) took as long,
// decoding a half tile ahead in registers 73 us, the hand-over warp between them and the
// issuing thread 68.
// A chain is a row tile of 128 rows with its S (128 columns of TMEM, P over
// the first 64) and O.  With more than 128 rows the two chains are two row
// tiles that share every key tile; with fewer, chain c takes the key tiles j =
// c mod 2 of the same rows and the two are joined at the end.  Per tile:
//   S = Q K^T         M = 128, N = 128, fp16 in, fp32 accumulate
//   P = exp2(S c - m) fp16, over the first half of S
//   O += P V          A from TMEM, V MN-major
// The MMAs of a chain execute in issue order, S_{j+1} right behind P_j V_j, so
// the softmax that sees S_j complete may rescale O and overwrite S_j.  A chain
// is a loop of S, softmax, P V: for the tensor cores to stay busy the softmax has
// to take no longer than the other chain's MMAs (about 1280 cycles a tile), hence
// two threads a row.  They use one reference m, which moves before 64 keys' P can
// sum above 60000, i.e. before one of them can pass fp16's range; each row
// decides on its own scores alone.  Every tile ends in one barrier of the chain's
// softmax threads, after which P may go over S, and which says whether some row
// needs more than the plain path (no reference yet, or one to move).
// Pages of a tile that lie past the sequence are not fetched: whatever their
// bytes are, they decode to finite values and their P is 0.
// Every wait is bounded; on expiry the block flags TSD_STATUS_TIMEOUT, drains
// what it issued, frees its tensor memory and returns.

#include <cuda_bf16.h>

#include "attention_q4.cuh"
#include "sm100_ptx.cuh"

namespace tsd {
namespace {

constexpr int kTcThreads = 768;
constexpr int kBM = 128;            // rows of a chain's MMA
constexpr int kBN = 128;            // keys of a tile
constexpr int kTilePages = kBN / kPage;
constexpr int kItemPages = 4;       // pages of a packed item: half a tile
constexpr int kPackSlots = 3;       // packed items of K, and of V, in flight with two row tiles
constexpr int kPackMost = 6;        // with one: the second Q tile's memory holds the others
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemChain = 256, kTmemO = 128;
constexpr float kTcOffset = 8.f;    // P of the reference score is 2^8 .. 2^9
constexpr float kTcMaxSum = 60000.f;
constexpr float kTcLargeRef = 65536.f;  // a product there is off by 2^-8 at most
constexpr float kTcLn2 = 0.6931471805599453f;
constexpr uint64_t kTcDrainNs = 100000000ull;

template <int D>
struct TcLayout {
  static constexpr uint32_t kHalf = kBM * 128;         // one 64-column half of a tile
  static constexpr uint32_t kTile = kBM * D * 2;       // an fp16 Q, K or V tile
  static constexpr uint32_t kPack = kItemPages * Q4Page<D>::kBytes;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = 2 * kTile;
  static constexpr uint32_t kV = kK + 2 * kTile;
  static constexpr uint32_t kP = kV + 2 * kTile;       // packed rings
  static constexpr uint32_t kBytes = kP + 2 * kPackSlots * kPack;
  static constexpr uint32_t kAlloc = kBytes + 1024;    // alignment slack
  static_assert(kAlloc <= 227 * 1024, "shared memory");
  static_assert(2 * (kPackMost - kPackSlots) * kPack <= kTile, "packed items in place of a Q tile");
  // slot of the ring of K (v = 0) or V (v = 1)
  static __device__ __forceinline__ uint32_t pack(int v, int slot) {
    return slot < kPackSlots ? kP + (v * kPackSlots + slot) * kPack
                             : kQ + kTile + (v * (kPackMost - kPackSlots) + slot - kPackSlots) * kPack;
  }
};

constexpr int kTcBarriers = 4 * kPackMost + 17;

struct TcSeg {
  Q4Seg s;
  int n;     // its key tiles
  bool two;  // two row tiles (each with every key tile), or one row tile whose key
             // tiles alternate between the chains
  bool more;
};

struct TcShared {
  uint64_t pk_full[2][kPackMost], pk_empty[2][kPackMost];  // K, V
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_final[2], q_full, drain;
  uint64_t never;  // (kTcBarriers in all, in the order tc_segment counts on)
  float2 ml[kBM];           // chain 1's (reference, sum) when it shares chain 0's rows
  float half[2][2][kBM];    // by chain, thread of the row, row: exchange between the two
  uint8_t asks[2][2][kBM];  // likewise
  int stop[2][2];           // by chain and tile parity: a wait ran out
  uint32_t tmem_base;
  int abort, bad;
  int g;       // units of the block's part that were taken (q4_next)
  TcSeg seg;   // the segment in work; here, not in registers, which the roles lack
  Q4Plan plan;
};

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  // fp16 A and B (format 0), fp32 accumulator
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// mbar_wait with its polling loop kept a loop: unrolled at every wait, it made two
// thirds of the kernel's code, and instruction fetch bound the blocks.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  using namespace sm100;
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  for (int i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 0 && global_timer_ns() - t0 > limit_ns) return false;
  }
}
// The same, and it gives up when another wait of the block ran out.
__device__ __forceinline__ bool tc_wait(uint64_t &bar, uint32_t parity, uint64_t limit, volatile int *abort) {
  using namespace sm100;
  if (mbar_try_wait(smem_addr(&bar), parity)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  for (int i = 1;; ++i) {
    if (mbar_try_wait(smem_addr(&bar), parity)) return true;
    if ((i & 63) != 0) continue;
    if (*abort) return false;
    if (global_timer_ns() - t0 > limit) {
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Waits for this thread's TMEM loads; the registers are operands, so that no
// use of them can be scheduled before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Register split of the six warpgroups (80 a thread at launch, 480 in all).
template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegs));
}
constexpr int kRegsLaunch = 80, kRegsIssue = 56, kRegsDecode = 72, kRegsSoftmax = 88;
static_assert(kRegsIssue + kRegsDecode + 4 * kRegsSoftmax <= 6 * kRegsLaunch, "what the block was launched with");

// Barrier of a chain's 256 softmax threads; returns whether any passed true.
__device__ __forceinline__ bool chain_any(int c, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 256, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(2 + c)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void chain_sync(int c) {
  asm volatile("barrier.cta.sync %0, 256;\n" ::"r"(2 + c) : "memory");
}

// Visibility of the 32 keys from tail index j0 on.  Out of line, once: tiles that
// reach the tree are few.
__device__ __noinline__ uint32_t visible32(const Q4Attn &p, int b, int row, int j0, int nb) {
  if (row >= nb * p.g) return 0u;
  const int node = row / p.g;
  return q4_visible(p, b, node, j0, nb) | (q4_visible(p, b, node, j0 + 16, nb) << 16);
}

// The reference for a row whose largest score is m: 8 below, or m where 8 is less
// than its ulp.
__device__ __forceinline__ float reference(float m) {
  const float to = m - kTcOffset;
  return m - to <= kTcOffset + 1.f ? to : m;
}

// What the row may not see becomes -inf.
__device__ __forceinline__ void mask_scores(uint32_t vis, uint32_t (&s)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (!((vis >> i) & 1u)) s[i] = 0xFF800000u;
}

__device__ __forceinline__ void mbar_inval(uint32_t bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

// The block's next segment, and its barriers; every thread of the block calls it,
// after everything of the segment before has completed.  `fresh`: there was none.
__device__ __forceinline__ bool tc_segment(const Q4Attn &p, TcShared &sh, bool fresh, int tid) {
  using namespace sm100;
  tc_fence_before();
  __syncthreads();
  if (tid < 32) {
    int g = sh.g;
    TcSeg sg;
    sg.more = q4_next(p, sh.plan, g, sg.s);
    if (sg.more) {
      sg.n = (sg.s.last - sg.s.first + kTilePages - 1) / kTilePages;
      sg.two = sg.s.rb * p.rows_per_block + kBM < sg.s.nb * p.g && p.rows_per_block > kBM;
      // the barriers lie one after the other, from pk_full to never
      for (int i = tid; i < kTcBarriers; i += 32) {
        const uint32_t bar = smem_addr(&sh.pk_full[0][0] + i);
        const int k = i - 4 * kPackMost;  // the barriers behind the rings'
        int count = 1;
        if (i >= 2 * kPackMost && k < 0) count = 2;               // pk_empty: a pair of decoders
        if (k == 0 || k == 1 || k == 4 || k == 5) count = 2;      // k_full, v_full: likewise
        // p_full: the softmax warps, and the hand-over or both pairs of decoders
        if (k == 10 || k == 11) count = !sg.two ? 12 : k == 10 ? 9 : 8;
        if (k == 14) count = 16;                                  // q_full: softmax warps
        if (!fresh) mbar_inval(bar);
        mbar_init(bar, count);
      }
      fence_mbar_init();
    }
    __syncwarp();
    if (tid == 0) {
      if (!fresh && sh.bad && p.status) atomicOr(p.status, TSD_STATUS_BAD_PAGE);
      sh.bad = 0;
      sh.g = g;
      sh.seg = sg;
    }
  }
  __syncthreads();
  tc_fence_after();
  return sh.seg.more;
}

// A block a part of the plan, or grid (splits * row blocks * Hkv, B); blocks of
// 256 rows, or of 128 where a kv head has no more.
template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) tree_attn_q4_tc_kernel(const Q4Attn p) {
  using namespace sm100;
  using L = TcLayout<D>;
  using Page = Q4Page<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ TcShared sh;
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *gbase = smem_raw + (base - raw);
  volatile int *abort = &sh.abort;
  const uint64_t lim = p.wait_limit_ns;

  pdl_wait();
  if (p.planned && warp == 0) q4_plan(p, sh.plan);
  if (tid == 0) {
    sh.abort = 0;
    sh.bad = 0;
    for (int i = 0; i < 4; ++i) sh.stop[i >> 1][i & 1] = 0;
  }
  __syncthreads();
  {  // a block without work leaves before the set-up
    Q4Seg seg;
    int g = p.planned ? blockIdx.x * sh.plan.part : 0;
    if (tid == 0) sh.g = g;
    if (!q4_next(p, sh.plan, g, seg)) return;
    if (!p.planned) {
      const bool work = seg.rb * p.rows_per_block < seg.nb * p.g && seg.first < seg.last;
      // rows that no chain computes, when they go straight to the output (planned:
      // the join writes them)
      if (seg.direct) {
        const int row0 = seg.rb * p.rows_per_block, end = min(p.rows, row0 + p.rows_per_block);
        for (int x = tid; x < (end - row0) * (D / 8); x += kTcThreads) {
          const int r = row0 + x / (D / 8);
          if (work && r < seg.nb * p.g) continue;
          const size_t orow = q4_out_row(p, seg.b, seg.h, r);
          reinterpret_cast<uint4 *>(p.out + orow * D)[x % (D / 8)] = make_uint4(0u, 0u, 0u, 0u);
          if (x % (D / 8) == 0 && p.lse) p.lse[orow] = -INFINITY;
        }
      }
      if (!work) return;
    }
  }
  if (warp == 1) tmem_alloc(smem_addr(&sh.tmem_base), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  // The roles; each takes the block's segments in turn, all of them the same ones.
  // What follows the roles is compiled for all of them, so it has to fit the
  // smallest share of registers: nothing but the teardown.
  const volatile TcSeg &sg = sh.seg;
  if (warp < 4) {
    regs_down<kRegsIssue>();
    for (bool fresh = true; tc_segment(p, sh, fresh, tid); fresh = false) {
    const int b = sg.s.b, h = sg.s.h, first = sg.s.first, last = sg.s.last, n = sg.n;
    const bool two = sg.two;
    const int chains = two || n > 1 ? 2 : 1, ring = two ? kPackSlots : kPackMost;
    if (warp == 0 || warp == 3) {
      // ---- loaders: warp 0 K, warp 3 V, half a tile at a time; lane l < 4 copies the
      // item's page l.  (A warp needs some 60 ns to issue a copy: one warp for K and V
      // bound the blocks of one row tile.)  K and V have rings of their own, so that
      // each slot has one loader and one pair of decoders, which take its items in
      // order.  Block ids come 32 (eight items) at a time and a batch ahead: read for
      // each item, their latency was on every item's path. ----
      const int v = warp == 3 ? 1 : 0;
      const uint8_t *pool = v ? p.v : p.k;
      const int32_t *trow = p.table + (size_t)b * p.max_blocks;
      auto read_ids = [&](int batch) {
        const int pg = first + batch * 32 + lane;
        return pg < last ? __ldg(trow + pg) : 0;
      };
      int ids = read_ids(0), ahead = read_ids(1);
      bool ok = true;
      int issued = 0;
      // (slot and phase are counted: a division by the ring's size takes as long as
      // a wait)
      uint32_t phase = 1;
      for (int m = 0, slot = 0; m < 2 * n; ++m) {
        if (m > 0 && (m & 7) == 0) {
          ids = ahead;
          ahead = read_ids((m >> 3) + 1);
        }
        const int id = __shfl_sync(0xffffffffu, ids, (m & 7) * kItemPages + (lane & (kItemPages - 1)));
        const bool mine = lane < kItemPages && first + m * kItemPages + lane < last;
        const bool bad = mine && (id < 0 || id >= p.num_blocks);
        if (bad) sh.bad = 1;
        if (m >= ring)
          ok = __all_sync(0xffffffffu, tc_wait(sh.pk_empty[v][slot], phase, lim, abort));
        if (!ok) break;
        const bool copy = mine && !bad;
        const int copies = __popc(__ballot_sync(0xffffffffu, copy));
        const uint32_t bar = smem_addr(&sh.pk_full[v][slot]);
        if (lane == 0) mbar_arrive_expect_tx(bar, copies * Page::kBytes);
        __syncwarp();
        if (copy)
          bulk_load(base + L::pack(v, slot) + lane * Page::kBytes,
                    pool + ((size_t)id * p.Hkv + h) * Page::kBytes, Page::kBytes, bar);
        issued = m + 1;
        if (++slot == ring) {
          slot = 0;
          phase ^= 1;
        }
      }
      // no copy is in flight when the block exits
      for (int m = max(0, issued - ring); m < issued; ++m)
        wait_phase(smem_addr(&sh.pk_full[v][m % ring]), (m / ring) & 1, kTcDrainNs);
    } else if (warp == 1) {
      // ---- MMA issue ----
      if (lane == 0) {
        constexpr uint32_t idS = idesc_f16_f32(kBM, kBN, false);
        constexpr uint32_t idPV = idesc_f16_f32(kBM, D, true);
        auto issue_s = [&](int c, int qt, int st) {
          const uint64_t qd = smem_desc_sw128(base + L::kQ + qt * L::kTile, 16, 1024);
          const uint64_t kd = smem_desc_sw128(base + L::kK + st * L::kTile, 16, 1024);
          tc_fence_after();
  #pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16(tmem + c * kTmemChain, desc_add(qd, (kk >> 2) * L::kHalf + (kk & 3) * 32),
                      desc_add(kd, (kk >> 2) * L::kHalf + (kk & 3) * 32), idS, kk > 0);
          umma_commit(smem_addr(&sh.s_full[c]));
        };
        auto issue_pv = [&](int c, int st, bool accum, bool final) {
          const uint64_t vd = smem_desc_sw128(base + L::kV + st * L::kTile, L::kHalf, 1024);
          uint64_t v8[8];
  #pragma unroll
          for (int kk = 0; kk < 8; ++kk) v8[kk] = desc_add(vd, kk * 16 * 128);
          tc_fence_after();
          umma8_ts(tmem + c * kTmemChain + kTmemO, tmem + c * kTmemChain, v8, idPV, accum ? 1u : 0u);
          if (final) umma_commit(smem_addr(&sh.o_final[c]));
        };
        // This thread paces the tensor cores, so its only wait in the loop is the
        // one for P: warp 2 adds to that barrier once V_j and the next K are there.
        // (With waits of its own for them it lost 200 to 500 cycles each, behind
        // the shared-memory traffic of the other warps.)
        bool ok = !p.test_stall || tc_wait(sh.never, 0, lim, abort);
        ok = ok && tc_wait(sh.q_full, 0, lim, abort);
        ok = ok && tc_wait(sh.k_full[0], 0, lim, abort);
        if (ok) issue_s(0, 0, 0);
        if (chains == 2) {
          if (!two) ok = ok && tc_wait(sh.k_full[1], 0, lim, abort);
          if (ok) issue_s(1, two ? 1 : 0, two ? 0 : 1);
        }
        if (two) {
          for (int j = 0; ok && j < n; ++j) {
            const int st = j & 1;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              ok = ok && wait_phase(smem_addr(&sh.p_full[c]), j & 1, lim);
              if (!ok) break;
              issue_pv(c, st, j > 0, j == n - 1);
              if (j + 1 < n) issue_s(c, c, st ^ 1);
            }
          }
        } else {
          for (int j = 0; ok && j < n; ++j) {
            const int c = j & 1;
            ok = wait_phase(smem_addr(&sh.p_full[c]), (j >> 1) & 1, lim);
            if (!ok) break;
            issue_pv(c, c, j > 1, j + 2 >= n);
            if (j + 2 < n) issue_s(c, 0, c);
          }
        }
        if (!ok) *abort = 1;
        umma_commit(smem_addr(&sh.drain));
        wait_phase(smem_addr(&sh.drain), 0, kTcDrainNs);
      }
      __syncwarp();
    } else if (warp == 2 && two) {
      // ---- hand-over: phase j of p_full also means that V_j and the K tile of the
      // S behind P_j V_j are in shared memory.  (An arrival counts toward the phase
      // that is open: the one before has to be complete.  With one row tile the
      // decoders arrive there themselves, see there.) ----
      if (lane == 0) {
        // Each barrier's phases are waited for one after the other (a wait for a
        // phase whose predecessor is still open returns at once): the first K tile
        // too, which the issuing thread waits for itself.
        tc_wait(sh.k_full[0], 0, lim, abort);
        for (int j = 0; j < n; ++j) {
          const int k = j + 1;
          bool ok = k >= n || tc_wait(sh.k_full[k & 1], (k >> 1) & 1, lim, abort);
          if (ok) ok = tc_wait(sh.v_full[j & 1], (j >> 1) & 1, lim, abort);
          if (ok && j > 0) ok = tc_wait(sh.p_full[0], (j - 1) & 1, lim, abort);
          if (!ok) break;
          mbar_arrive(smem_addr(&sh.p_full[0]));
        }
      }
      __syncwarp();
    }
    }
  } else if (warp < 8) {
    regs_down<kRegsDecode>();
    for (bool fresh = true; tc_segment(p, sh, fresh, tid); fresh = false) {
    const int n = sg.n, ring = sg.two ? kPackSlots : kPackMost;
    const bool two = sg.two;
    // ---- decode: warps 4 and 5 K tiles, 6 and 7 V tiles (two tiles at a time hide
    // each other's waits and fences: 128-row blocks were bound by four warps on
    // one tile); a lane takes one group (16 columns) of a key at a time ----
    constexpr int kGroups = D / kQ4Group;        // lanes across one key
    constexpr int kKeys = 32 / kGroups;          // keys per warp step
    constexpr int kSteps = kItemPages * kPage / (2 * kKeys);  // steps of a warp
    const int v = warp >= 6 ? 1 : 0;
    const int dw = warp & 1;
    const int grp = lane % kGroups, kl = lane / kGroups;
    // the two halves of a key are stored in opposite order, so that the eight
    // lanes of a store's quarter touch different banks
    const int flip = D == 128 ? grp >> 2 : 0;
    const int c0 = (grp & 3) * 2;
    // Where a decoded tile is reported.  With one row tile straight to the barrier that
    // the issuing thread waits for, which saves a hop of some 450 cycles: its phase of
    // tile j wants V_j and K_{j+2}, both decoded only after S_j was seen (the first two V
    // at once), so after the phase before was complete.
    const uint32_t full_first = smem_addr(v == 0 ? sh.k_full : two ? sh.v_full : sh.p_full);
    const uint32_t full = two ? full_first : smem_addr(sh.p_full);
    uint32_t phase = 0;
    for (int m = 0, slot = 0; m < 2 * n; ++m) {  // half tiles
      const int tile = m >> 1, st = tile & 1;
      bool ok = tc_wait(sh.pk_full[v][slot], phase, lim, abort);
      if (ok && tile >= 2 && (m & 1) == 0)
        ok = tc_wait(v ? sh.v_empty[st] : sh.k_empty[st], ((tile >> 1) - 1) & 1, lim, abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint8_t *src = gbase + L::pack(v, slot);
      uint8_t *dst = gbase + (v ? L::kV : L::kK) + st * L::kTile + (D == 128 ? (grp >> 2) * L::kHalf : 0) +
                     (m & 1) * (kBN / 2) * 128;
      // every read comes before the first store: the compiler must assume that a
      // store changes what the next read sees, and would wait out each one's latency
      uint2 code[kSteps];
      uint32_t scale[kSteps];
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int key = (s * 2 + dw) * kKeys + kl;
        const uint8_t *page = src + (key / kPage) * Page::kBytes;
        const int r = key % kPage;
        code[s] = *reinterpret_cast<const uint2 *>(page + r * Page::kRow + grp * 8);
        scale[s] = page[Page::kScales + r * Page::kScaleRow + grp];
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int key = (s * 2 + dw) * kKeys + kl;
        const uint32_t sc = q4_scale2(scale[s]);
        uint32_t a[4], e[4];
        q4_decode8(flip ? code[s].y : code[s].x, a);
        q4_decode8(flip ? code[s].x : code[s].y, e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = q4_mul2(a[i], sc);
          e[i] = q4_mul2(e[i], sc);
        }
        *reinterpret_cast<uint4 *>(dst + sw128_offset(key, c0 + flip)) = make_uint4(a[0], a[1], a[2], a[3]);
        *reinterpret_cast<uint4 *>(dst + sw128_offset(key, c0 + 1 - flip)) = make_uint4(e[0], e[1], e[2], e[3]);
      }
      if (m & 1) fence_proxy_async_smem();  // the tensor core reads the tile through the async proxy
      __syncwarp();
      if (lane == 0) {
        if (m & 1) mbar_arrive((tile < 2 ? full_first : full) + st * 8);
        mbar_arrive(smem_addr(&sh.pk_empty[v][slot]));
      }
      if (++slot == ring) {
        slot = 0;
        phase ^= 1;
      }
    }
    // the last tiles' phases have no K_{j+2}
    for (int tile = max(n, 2); !two && v == 0 && tile < n + 2; ++tile) {
      if (!tc_wait(sh.k_empty[tile & 1], ((tile >> 1) - 1) & 1, lim, abort)) break;
      if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[tile & 1]));
    }
    }
  } else {
    regs_up<kRegsSoftmax>();
    for (bool fresh = true; tc_segment(p, sh, fresh, tid); fresh = false) {
    const int n = sg.n;
    const bool two = sg.two;
    const int chains = two || n > 1 ? 2 : 1;
    // (what the tile loop does not need is read again from the segment)
    auto row_of = [&](int rl, int rt) { return sg.s.rb * p.rows_per_block + rt * kBM + rl; };
    // ---- softmax ----
    const int c = (warp - 8) >> 3;             // chain
    const int half = ((warp - 8) >> 2) & 1;    // which 64 keys of a tile, and columns of O
    const int rt = two ? c : 0;                // its row tile
    const int quarter = warp & 3;
    const int rl = quarter * 32 + lane;        // row within the tile
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + c * kTmemChain + lane_off, tO = tS + kTmemO;

    // half a Q row -> fp16, scaled by a power of two (both chains know it)
    float mul;
    {
      const int row = row_of(rl, rt);
      const bool rvalid = row < sg.s.nb * p.g;
      const uint4 *src = reinterpret_cast<const uint4 *>(
          p.q + q4_out_row(p, sg.s.b, sg.s.h, rvalid ? row : 0) * D + half * (D / 2));
      uint4 x[D / 16];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) x[i] = rvalid ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
      uint32_t most = 0u;  // bf16 magnitudes order as integers (NaN above all)
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        most = __vmaxu2(__vmaxu2(most, x[i].x & 0x7FFF7FFFu), x[i].y & 0x7FFF7FFFu);
        most = __vmaxu2(__vmaxu2(most, x[i].z & 0x7FFF7FFFu), x[i].w & 0x7FFF7FFFu);
      }
      float amax = __uint_as_float(max(most << 16, most & 0xFFFF0000u));
      sh.half[c][half][rl] = amax;
      chain_sync(c);
      const float other = sh.half[c][half ^ 1][rl];
      amax = __uint_as_float(max(__float_as_uint(amax), __float_as_uint(other)));
      const int e = q4_exponent(amax);
      // the factor's sign goes into q, and it stays between the smallest and the
      // largest normal number, so that a masked score (-inf) stays one
      const float sign = p.scale_log2 < 0.f ? -1.f : p.scale_log2 > 0.f ? 1.f : 0.f;
      const float up1 = sign * q4_pow2(e / 2), up2 = q4_pow2(e - e / 2);
      mul = fabsf(p.scale_log2) * q4_pow2(-(e / 2)) * q4_pow2(-(e - e / 2));
      mul = fminf(fmaxf(mul, 1.1754944e-38f), 3.4028235e38f);
      if (two || c == 0) {
        uint8_t *dst = gbase + L::kQ + rt * L::kTile;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = pack_half2(__uint_as_float(w[k] << 16) * up1 * up2,
                              __uint_as_float(w[k] & 0xFFFF0000u) * up1 * up2);
          const int ch = half * (D / 16) + i;  // 16-byte chunk of the row
          *reinterpret_cast<uint4 *>(dst + (ch >> 3) * L::kHalf + sw128_offset(rl, ch & 7)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.q_full));
    }

    float ref = 0.f, l = 0.f;  // the row's reference, this thread's part of its sum
    bool unset = true, ok = c < chains;
    const unsigned long long mul2 = f2_pack(mul, mul);
    int u = 0;  // this chain's tiles
    // this thread's first key slot in tile j is 128 j + slot0; the tile reaches the
    // tree where it passes tree_from
    const int slot0 = sg.s.first * kPage + half * 64, tree_from = sg.s.P - 64 - slot0;
    auto visible = [&](int j, int k) {
      return visible32(p, sg.s.b, row_of(rl, rt), j * kBN + slot0 + k * 32 - sg.s.P, sg.s.nb);
    };
    for (int j = two ? 0 : c; ok && j < n; j += two ? 1 : 2, ++u) {
      // one warp looks at the barrier, the others wait for it without polling
      bool got = true;
      if (((warp - 8) & 7) == 0) {
        got = __all_sync(0xffffffffu, tc_wait(sh.s_full[c], u & 1, lim, abort));
        if (!got) sh.stop[c][u & 1] = 1;
      }
      chain_sync(c);
      tc_fence_after();
      if ((two ? c == 1 : true) && half == 0 && quarter == 0 && lane == 0) {
        // A commit follows every earlier MMA of its thread, so K_j and the V tile
        // that the P V in front of S_j read are free.  (Commits of their own for
        // that cost 0.3 us each on the tensor pipe.)
        mbar_arrive(smem_addr(&sh.k_empty[j & 1]));
        const int jv = two ? j - 1 : j - 2;
        if (jv >= 0) mbar_arrive(smem_addr(&sh.v_empty[jv & 1]));
      }
      const bool tail = j * kBN > tree_from;
      unsigned long long acc0 = 0ull, acc1 = 0ull;
      uint32_t pk[32], seen = 0u;
      {
        // both loads before the one wait: a load's latency is some 250 cycles
        uint32_t x[2][32];
        tmem_ld32(tS + half * 64, x[0]);
        tmem_ld32(tS + half * 64 + 32, x[1]);
        tmem_wait_ld(x[0]);
        tmem_wait_ld(x[1]);
        if (tail) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t vis = visible(j, k);
            seen |= vis;
            mask_scores(vis, x[k]);
          }
        }
        if (u == 0) {
          // the chain's first tile: the row's maximum over it is the reference
          float m = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; ++i) m = fmax3(m, __uint_as_float(x[0][i]), __uint_as_float(x[1][i]));
          sh.half[c][half][rl] = m;
          chain_sync(c);
          m = __fmul_rn(fmaxf(m, sh.half[c][half ^ 1][rl]), mul);
          if (m > -INFINITY) {
            ref = reference(m);
            unset = false;
          }
        }
        const unsigned long long ref2 = f2_pack(-ref, -ref);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 t = f2_unpack(f2_fma(
                f2_pack(__uint_as_float(x[k][2 * i]), __uint_as_float(x[k][2 * i + 1])), mul2, ref2));
            const float e0 = ex2_approx(t.x), e1 = ex2_approx(t.y);
            pk[k * 16 + i] = pack_half2(e0, e1);
            if (i & 1) acc1 = f2_add(acc1, f2_pack(e0, e1));
            else acc0 = f2_add(acc0, f2_pack(e0, e1));
          }
        }
      }
      const float2 acc = f2_unpack(f2_add(acc0, acc1));
      float sum = acc.x + acc.y;
      // Rows that need more than that: no reference yet, P out of fp16's range, or
      // a reference (itself a rounded product) so large that the exact product
      // above lies powers of two away from it; those round the product first.
      const bool mine = (unset && (!tail || seen != 0u)) || !(sum <= kTcMaxSum) || fabsf(ref) >= kTcLargeRef;
      tc_fence_before();
      const bool any = chain_any(c, mine || !got);
      tc_fence_after();
      if (__builtin_expect(any, 0)) {
        if (sh.stop[c][u & 1]) {  // the same for every warp of the chain
          ok = false;
          break;
        }
        float m = -INFINITY;
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          uint32_t s[32];
          tmem_ld32(tS + half * 64 + k * 32, s);
          tmem_wait_ld(s);
          if (tail) mask_scores(visible(j, k), s);
#pragma unroll
          for (int i = 0; i < 32; ++i) m = fmaxf(m, __fmul_rn(__uint_as_float(s[i]), mul));
        }
        // what the row's two threads know: its maximum, and whether either asked
        sh.half[c][half][rl] = m;
        sh.asks[c][half][rl] = mine;
        chain_sync(c);
        const bool row_asks = mine || sh.asks[c][half ^ 1][rl];
        m = fmaxf(m, sh.half[c][half ^ 1][rl]);
        float f = 1.f;
        if (row_asks && m > -INFINITY && (unset || !(m - ref <= kTcOffset + 2.f))) {
          const float to = reference(m);
          // (nothing was added yet to a row without a reference)
          if (!unset) f = ex2_approx(ref - to);
          ref = to;
          unset = false;
          l *= f;
        }
        if (__any_sync(0xffffffffu, row_asks)) {
          float again = 0.f;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t s[32];
            tmem_ld32(tS + half * 64 + k * 32, s);
            tmem_wait_ld(s);
            if (tail) mask_scores(visible(j, k), s);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float e0 = ex2_approx(__fsub_rn(__fmul_rn(__uint_as_float(s[2 * i]), mul), ref));
              const float e1 = ex2_approx(__fsub_rn(__fmul_rn(__uint_as_float(s[2 * i + 1]), mul), ref));
              again += e0 + e1;
              pk[k * 16 + i] = row_asks ? pack_half2(e0, e1) : pk[k * 16 + i];
            }
          }
          if (row_asks) sum = again;
        }
        if (u > 0 && __any_sync(0xffffffffu, f != 1.f)) {  // this thread's half of O
#pragma unroll 1
          for (int q = 0; q < D / 64; ++q) {
            uint32_t o[32];
            const uint32_t at = tO + half * (D / 2) + q * 32;
            tmem_ld32(at, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st32(at, o);
          }
        }
        tc_fence_before();
        chain_sync(c);  // S has been read again
        tc_fence_after();
      }
      l += sum;
      tmem_st32(tS + half * 32, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[c]));
    }

    // ---- epilogue: O of this chain is complete ----
    const bool joined = !two && chains == 2;
    if (ok) ok = __all_sync(0xffffffffu, tc_wait(sh.o_final[c], 0, lim, abort));
    // (the rows go over the K and V tiles, which the other chain's last MMAs may
    // still read)
    if (ok && chains == 2) ok = __all_sync(0xffffffffu, tc_wait(sh.o_final[c ^ 1], 0, lim, abort));
    tc_fence_after();
    sh.half[c][half][rl] = l;
    chain_sync(c);
    l += sh.half[c][half ^ 1][rl];
    float M = unset ? -INFINITY : ref;
    if (unset && l != l) M = 0.f;  // only NaN scores so far
    // K and V tiles are done with: chain 1's O when it shares chain 0's rows
    // (column-major, so that lanes do not collide), then the finished rows
    float *stage = reinterpret_cast<float *>(gbase + L::kK);
    const uint32_t rows_at = (two && c == 0 ? L::kK : L::kV);
    uint8_t *rows_out = gbase + rows_at;
    const int q0 = half * (D / 64);  // this thread's 32-column parts of O
    if (joined && c == 1) {
#pragma unroll 1
      for (int q = q0; ok && q < q0 + D / 64; ++q) {
        uint32_t o[32];
        tmem_ld32(tO + q * 32, o);
        tmem_wait_ld(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) stage[(q * 32 + i) * kBM + rl] = __uint_as_float(o[i]);
      }
      if (half == 0) sh.ml[rl] = make_float2(M, l);
    }
    if (joined) asm volatile("barrier.cta.sync 1, 512;\n" ::: "memory");
    if (c < (two ? 2 : 1)) {
      float f0 = 1.f, f1 = 0.f;
      if (joined) {
        const float2 other = sh.ml[rl];
        const float top = fmaxf(M, other.x);
        f0 = M == -INFINITY ? 0.f : ex2_approx(M - top);
        f1 = other.x == -INFINITY ? 0.f : ex2_approx(other.x - top);
        l = f0 * l + f1 * other.y;
        M = top;
      }
      const bool bad = sh.bad != 0, direct = sg.s.direct;
      const bool empty = direct && (bad || l == 0.f);
      // O times this; a row that is left out becomes 0 whatever its sums are
      if (direct) {
        const float inv = empty ? 0.f : 1.f / l;
        f0 *= inv;
        f1 *= inv;
      }
#pragma unroll 1
      for (int q = q0; ok && q < q0 + D / 64; ++q) {
        uint32_t o[32];
        tmem_ld32(tO + q * 32, o);
        tmem_wait_ld(o);
        if (empty) {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f0);
        if (joined && f1 != 0.f) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            o[i] = __float_as_uint(fmaf(f1, stage[(q * 32 + i) * kBM + rl], __uint_as_float(o[i])));
        }
        const float *v = reinterpret_cast<const float *>(o);
        // whole rows in shared memory, their 16-byte chunks swizzled by row
        if (direct) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4 *>(rows_out + rl * (D * 2) + (((q * 4 + i) ^ (rl & 7)) << 4)) =
                make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                           pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4 *>(rows_out + rl * (D * 4) + (((q * 8 + i) ^ (rl & 7)) << 4)) =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
      const int row = row_of(rl, rt);
      if (half == 0 && row < sg.s.nb * p.g) {
        if (!direct)
          p.part_ml[sg.s.part + rt * kBM + rl] = make_float2(M, bad ? -1.f : l);
        else if (p.lse)
          p.lse[q4_out_row(p, sg.s.b, sg.s.h, row)] = empty ? -INFINITY : (M + log2f(l)) * kTcLn2;
      }
      if (!direct) fence_proxy_async_smem();
      chain_sync(c);
      const int w = (warp - 8) & 7;
      if (direct) {
        constexpr int kLanes = D / 8;  // of a row
#pragma unroll 1
        for (int r0 = w * (32 / kLanes); ok && r0 < kBM; r0 += 8 * (32 / kLanes)) {
          const int r = r0 + lane / kLanes, ch = lane % kLanes, orow = row_of(r, rt);
          if (orow < sg.s.nb * p.g)
            reinterpret_cast<uint4 *>(p.out + q4_out_row(p, sg.s.b, sg.s.h, orow) * D)[ch] =
                *reinterpret_cast<const uint4 *>(rows_out + r * (D * 2) + ((ch ^ (r & 7)) << 4));
        }
      } else if (lane == 0 && ok) {  // 16 partial rows a warp, in one piece and as they lie
        const int rows = min(kBM / 8, sg.s.nb * p.g - row_of(w * (kBM / 8), rt));
        if (rows > 0) {
          bulk_store(p.part_o + (sg.s.part + rt * kBM + w * (kBM / 8)) * D,
                     base + rows_at + w * (kBM / 8) * (D * 4), rows * D * 4);
          bulk_wait_read();
        }
      }
    }
    }
    if (lane == 0) bulk_wait();  // (the last segments' partial rows are written)
  }
  // (the last tc_segment ended with a barrier)
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  if (tid == 0 && p.status && sh.abort) atomicOr(p.status, TSD_STATUS_TIMEOUT);
}

}  // namespace

namespace {
// The register split draws on what the block was launched with: a build that
// gives a thread fewer registers must not run (it would wait forever).
template <int D>
bool tc_ready() {
  static const bool enough = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, tree_attn_q4_tc_kernel<D>) == cudaSuccess && a.numRegs >= kRegsLaunch;
  }();
  return enough && set_smem((const void *)tree_attn_q4_tc_kernel<D>, TcLayout<D>::kAlloc);
}
}  // namespace

cudaError_t q4_tc_launch(const Q4Attn &p, int D, int blocks, cudaStream_t s) {
  const dim3 grid = p.planned ? dim3(blocks) : dim3((unsigned)p.splits * p.row_blocks * p.Hkv, p.B);
  if (D == 128) {
    if (!tc_ready<128>()) return cudaErrorUnknown;
    return launch(tree_attn_q4_tc_kernel<128>, grid, dim3(kTcThreads), TcLayout<128>::kAlloc, s, p);
  }
  if (!tc_ready<64>()) return cudaErrorUnknown;
  return launch(tree_attn_q4_tc_kernel<64>, grid, dim3(kTcThreads), TcLayout<64>::kAlloc, s, p);
}

}  // namespace tsd
