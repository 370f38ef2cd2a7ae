// Block tables and slot maps of the paged cache, built on the GPU from the
// requests' lengths, so that no length has to reach the host between steps.
//
// "Speculative Decoding Hierárquico: Medusa, EAGLE-2 e Multi-Token
// Prediction", section on vLLM PagedAttention: a sequence's cache is a table of
// fixed-size blocks taken from a pool, and the blocks of what was rejected go
// back to it.
//
// The pool's unused blocks are a stack, free_list[0 .. free_count).  With
// want_b = ceil((P_b + n_b) / 16) and need_b = max(0, want_b - held_b), the
// blocks taken are numbered by sequence, then by position in its table: the
// i-th is free_list[free_count - 1 - i].  A sequence is served when it needs no
// block or its whole need fits under an exclusive scan of the needs, so the
// result does not depend on the order in which threads run; giving blocks back
// numbers them the same way and undoes a take exactly.
//
// Nothing here is bound by bandwidth in a decoding step: the scan over the
// batch is one block's, and the map (4 bytes a token) is written by a second
// grid, or by the same block when it is small.

#include "sm100_ptx.cuh"
#include "tsd_common.cuh"

namespace tsd {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kFillTokens = 4 * kFillThreads;  // tokens one fill block maps
// Calls of at most this many sequences and tokens run in one block: one launch, and
// no workspace.  Measured on the device, one block / two kernels: 64 tokens 2.8 / 3.6
// us, 2048 3.0 / 3.6, 8192 4.4 / 3.6 (less than a launch and a workspace cost the
// host), 32768 9.9 / 3.6.
constexpr int kSmallSeqs = 64;
constexpr int kSmallTokens = 8192;

// What the scan leaves for the fill, per sequence: the number of its first
// block among those taken (or given back), -1 when it is not served, and the
// blocks it held before.
struct SlotWork {
  int64_t *start;  // [B]
  int32_t *held;   // [B]
  int32_t *count;  // [1]: free blocks before the call
  int32_t *after;  // [B + 1] or null: blocks held and free blocks after it, for whoever
                   // stores them; null: the scan does
};

__host__ __device__ inline size_t slot_ws_bytes(int B) {
  return (size_t)B * (sizeof(int64_t) + sizeof(int32_t)) + sizeof(int64_t);
}
__host__ __device__ inline SlotWork slot_ws(void *ws, int B) {
  SlotWork w;
  w.start = reinterpret_cast<int64_t *>(ws);
  w.held = reinterpret_cast<int32_t *>(w.start + B);
  w.count = w.held + B;
  w.after = nullptr;
  return w;
}

struct SlotArgs {
  const int32_t *prefix_len, *n_new;  // release: prefix_len holds the lengths to keep
  int B, N_max;
  int32_t *table;
  int max_blocks;
  int32_t *held;
  int32_t *free_list, *free_count;
  int num_blocks;
  int32_t *slots, *status;
};

__device__ __forceinline__ int new_tokens(const SlotArgs &a, int b) {
  return a.n_new ? a.n_new[b] : a.N_max;
}

// Exclusive scan over the block's threads; `total` gets the sum.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t &total, int64_t *warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int64_t s = lane < warps ? warp_sums[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const int64_t before = warp ? warp_sums[warp - 1] : 0;
  total = warp_sums[31];
  __syncthreads();
  return before + incl - x;
}

// Blocks sequence b has to take (take) or can give back; -1: its lengths are
// refused.
template <bool kTake>
__device__ __forceinline__ int64_t seq_blocks(const SlotArgs &a, int b, int held) {
  const int P = a.prefix_len[b];
  const int n = kTake ? new_tokens(a, b) : 0;
  if (P < 0 || held < 0 || held > a.max_blocks) return -1;
  if (kTake && (n < 0 || n > a.N_max || (int64_t)P + n > (int64_t)a.max_blocks * kPage)) return -1;
  const int64_t want = ((int64_t)P + n + kPage - 1) / kPage;
  const int64_t d = kTake ? want - held : held - want;
  return d > 0 ? d : 0;
}

// The scan, by one block: fills `w`, updates held and free_count.  `report`: this
// block tells the status.
template <bool kTake>
__device__ void scan_sequences(const SlotArgs &a, const SlotWork &w, bool report = true) {
  __shared__ int64_t warp_sums[32];
  __shared__ int s_served_end;  // blocks taken by the sequences that were served
  const int count = *a.free_count;
  const bool count_ok = count >= 0 && count <= a.num_blocks;
  if (threadIdx.x == 0) s_served_end = 0;
  int bad = count_ok ? 0 : TSD_STATUS_BAD_LEN;
  int64_t all = 0;
  if (!kTake) {  // what comes back has to fit the list as a whole
    for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
      const int b = b0 + threadIdx.x;
      const int64_t d = b < a.B ? seq_blocks<false>(a, b, a.held[b]) : 0;
      int64_t total;
      block_scan(d > 0 ? d : 0, total, warp_sums);
      all += total;
    }
    if (all > (int64_t)a.num_blocks - count) bad |= TSD_STATUS_BAD_LEN;
  }
  const bool move = count_ok && (kTake || all <= (int64_t)a.num_blocks - count);
  __syncthreads();
  int64_t carry = 0;
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int held = 0;
    int64_t d = 0;
    if (b < a.B) {
      held = a.held[b];
      d = seq_blocks<kTake>(a, b, held);
    }
    if (d < 0) bad |= TSD_STATUS_BAD_LEN;
    int64_t total;
    const int64_t start = carry + block_scan(d > 0 ? d : 0, total, warp_sums);
    carry += total;
    if (b < a.B) {
      bool served = d == 0;
      if (d > 0) {
        served = move && (!kTake || start + d <= count);
        if (served) {
          if (!w.after) a.held[b] = kTake ? held + (int)d : held - (int)d;
          if (kTake) atomicMax(&s_served_end, (int)(start + d));
        } else if (kTake && count_ok) {
          bad |= TSD_STATUS_NO_BLOCK;
        }
      }
      w.start[b] = served ? start : -1;
      w.held[b] = held;
      if (w.after) w.after[b] = !served ? held : kTake ? held + (int)d : held - (int)d;
    }
  }
  if (report && bad && a.status) atomicOr(a.status, bad);
  __syncthreads();
  if (threadIdx.x == 0) {
    *w.count = count;
    const int left = !move ? count : kTake ? count - s_served_end : count + (int)all;
    if (w.after)
      w.after[a.B] = left;
    else if (move)
      *a.free_count = left;
  }
}

// Block j of sequence b: taken in this call, or held before it.  -1 when the
// id does not name a block of the pool.
__device__ __forceinline__ int block_of(const SlotArgs &a, int b, int j, int held, int64_t top) {
  const int id = j >= held ? a.free_list[top - (j - held)] : a.table[(size_t)b * a.max_blocks + j];
  return id >= 0 && id < a.num_blocks ? id : -1;
}

// Slots of tokens [i0, i0 + 4) and, spread over the `workers` threads of the
// sequence's blocks, its new table entries.
__device__ __forceinline__ void fill_sequence(const SlotArgs &a, int b, int64_t start, int held,
                                              int count, int i_first, int i_step, int worker,
                                              int workers) {
  const int P = a.prefix_len[b];
  const int n = new_tokens(a, b);
  const int64_t top = (int64_t)count - 1 - start;  // free_list position of its first new block
  bool bad = false;
  if (start >= 0) {
    const int want = (int)(((int64_t)P + n + kPage - 1) / kPage);
    for (int j = held + worker; j < want; j += workers) {
      const int id = block_of(a, b, j, held, top);
      bad |= id < 0;
      a.table[(size_t)b * a.max_blocks + j] = id;
    }
  }
  const bool wide = (a.N_max & 3) == 0;
  for (int i = i_first; i < a.N_max; i += i_step) {
    int out[4] = {-1, -1, -1, -1};
    if (start >= 0 && i < n) {
      int last_j = -1, id = -1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (i + e >= n) break;
        const int t = P + i + e;
        if (t / kPage != last_j) {
          last_j = t / kPage;
          id = block_of(a, b, last_j, held, top);
          bad |= id < 0;
        }
        out[e] = id < 0 ? -1 : id * kPage + t % kPage;
      }
    }
    int32_t *dst = a.slots + (size_t)b * a.N_max + i;
    if (wide) {
      *reinterpret_cast<int4 *>(dst) = make_int4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < a.N_max) dst[e] = out[e];
    }
  }
  if (bad && a.status) atomicOr(a.status, TSD_STATUS_BAD_PAGE);
}

// Gives blocks [keep, held) of sequence b back and clears their entries; `after`: free
// blocks when the call is done.  An entry that names no block of the pool (the build
// left -1 for such an id) takes its place on the list as it stands, so that the
// numbering holds, and is reported.
__device__ __forceinline__ void release_sequence(const SlotArgs &a, int b, int64_t start, int keep,
                                                 int held, int worker, int workers, int after) {
  if (start < 0) return;
  // the call's last given-back block is number all - 1 and lands at the old count
  const int top = after - 1;
  bool bad = false;
  for (int j = keep + worker; j < held; j += workers) {
    int32_t *e = a.table + (size_t)b * a.max_blocks + j;
    const int id = *e;
    bad |= id < 0 || id >= a.num_blocks;
    a.free_list[top - (start + (j - keep))] = id;
    *e = -1;
  }
  if (bad && a.status) atomicOr(a.status, TSD_STATUS_BAD_PAGE);
}

// Taking, small calls: everything in one block.
__global__ void __launch_bounds__(kScanThreads) slots_take_kernel(const SlotArgs a) {
  __shared__ int64_t s_start[kSmallSeqs];
  __shared__ int32_t s_held[kSmallSeqs], s_count;
  pdl_wait();
  scan_sequences<true>(a, SlotWork{s_start, s_held, &s_count, nullptr});
  __syncthreads();
  // every thread takes four tokens of one sequence at a time
  const int q = max((a.N_max + 3) / 4, 1);  // quads of one sequence
  for (int x = threadIdx.x; x < a.B * q; x += blockDim.x) {
    const int b = x / q, i = (x % q) * 4;
    fill_sequence(a, b, s_start[b], s_held[b], s_count, i, max(a.N_max, 1), x % q, q);
  }
}

// Giving back, up to kSmallSeqs sequences: a cluster, whose blocks all make the scan.
// The first stores what it found once all have read what was there.  (How many
// blocks come back is known on the device only; with one block 32768 of them took 10
// us, with eight 3.)
__global__ void __launch_bounds__(kScanThreads) slots_release_kernel(const SlotArgs a) {
  using namespace sm100;
  __shared__ int64_t s_start[kSmallSeqs];
  __shared__ int32_t s_held[kSmallSeqs], s_count, s_after[kSmallSeqs + 1];
  pdl_wait();
  const int rank = cluster_ctarank(), ctas = cluster_nctarank();
  scan_sequences<false>(a, SlotWork{s_start, s_held, &s_count, s_after}, rank == 0);
  __syncthreads();
  if (ctas > 1) {
    cluster_arrive();
    cluster_wait();
  }
  if (rank == 0 && threadIdx.x < a.B && s_after[threadIdx.x] != s_held[threadIdx.x])
    a.held[threadIdx.x] = s_after[threadIdx.x];
  if (rank == 0 && threadIdx.x == 0 && s_after[a.B] != s_count) *a.free_count = s_after[a.B];
  // the warps are dealt out over the sequences
  const int warps = ctas * (kScanThreads / 32), each = max(warps / a.B, 1);
  for (int x = rank * (kScanThreads / 32) + (threadIdx.x >> 5); x < a.B * each; x += warps) {
    const int b = x / each;
    release_sequence(a, b, s_start[b], s_after[b], s_held[b], (x - b * each) * 32 + (threadIdx.x & 31), each * 32,
                     s_after[a.B]);
  }
}

template <bool kTake>
__global__ void __launch_bounds__(kScanThreads) slots_scan_kernel(const SlotArgs a, SlotWork w) {
  pdl_wait();
  scan_sequences<kTake>(a, w);
}

// Grid (token tiles, sequences).
template <bool kTake>
__global__ void __launch_bounds__(kFillThreads) slots_fill_kernel(const SlotArgs a, SlotWork w) {
  pdl_wait();
  const int worker = blockIdx.x * kFillThreads + threadIdx.x, workers = gridDim.x * kFillThreads;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    if (kTake)
      fill_sequence(a, b, w.start[b], w.held[b], *w.count, worker * 4, workers * 4, worker, workers);
    else
      // (the scan has stored what is held and free now)
      release_sequence(a, b, w.start[b], a.held[b], w.held[b], worker, workers, *a.free_count);
  }
}

template <bool kTake>
int slots_launch(const SlotArgs &a, void *workspace, size_t ws_bytes, tsd_stream_t stream) {
  const cudaStream_t s = as_cuda(stream);
  if (a.B <= kSmallSeqs && (int64_t)a.B * a.N_max <= kSmallTokens) {
    if (kTake)
      return launch(slots_take_kernel, dim3(1), dim3(kScanThreads), 0, s, a) == cudaSuccess ? TSD_OK : TSD_ERR_CUDA;
    // at most max_blocks a sequence come back; 256 a block of the cluster at least
    int ctas = 1;
    while (ctas < 8 && ctas * 256ll < (int64_t)a.B * a.max_blocks) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kScanThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, slots_release_kernel, a) == cudaSuccess ? TSD_OK : TSD_ERR_CUDA;
  }
  if (!workspace || ws_bytes < slot_ws_bytes(a.B)) return TSD_ERR_WORKSPACE;
  if (!aligned(workspace, 8)) return TSD_ERR_ARG;
  const SlotWork w = slot_ws(workspace, a.B);
  if (launch(slots_scan_kernel<kTake>, dim3(1), dim3(kScanThreads), 0, s, a, w) != cudaSuccess)
    return TSD_ERR_CUDA;
  const int tiles = kTake ? (a.N_max + kFillTokens - 1) / kFillTokens : 1;
  const dim3 grid(tiles > 0 ? tiles : 1, a.B);
  return launch(slots_fill_kernel<kTake>, grid, dim3(kFillThreads), 0, s, a, w) == cudaSuccess
             ? TSD_OK
             : TSD_ERR_CUDA;
}

int slots_check(int B, int N_max, int max_blocks, int num_blocks) {
  if (B < 0 || N_max < 0 || max_blocks < 1 || num_blocks < 1) return TSD_ERR_ARG;
  if (B > 65535 || N_max > 262144 || (int64_t)num_blocks * kPage > 0x7FFFFFFFll ||
      (int64_t)max_blocks * kPage > 0x7FFFFFFFll)
    return TSD_ERR_LIMIT;
  return TSD_OK;
}

}  // namespace
}  // namespace tsd

TSD_API size_t tsd_kv_slots_workspace_bytes(int B, int N_max) {
  using namespace tsd;
  if (B < 1 || N_max < 0 || B > 65535 || N_max > 262144) return 0;
  if (B <= kSmallSeqs && (int64_t)B * N_max <= kSmallTokens) return 0;
  return slot_ws_bytes(B);
}

TSD_API int tsd_kv_slots_build(const int32_t *prefix_len, const int32_t *n_new, int B, int N_max,
                               int32_t *block_table, int max_blocks, int32_t *held,
                               int32_t *free_list, int32_t *free_count, int num_blocks,
                               int32_t *slots, void *workspace, size_t ws_bytes, int32_t *status,
                               tsd_stream_t stream) {
  using namespace tsd;
  const int rc = slots_check(B, N_max, max_blocks, num_blocks);
  if (rc != TSD_OK || B == 0) return rc;
  if (!prefix_len || !block_table || !held || !free_list || !free_count || (!slots && N_max > 0))
    return TSD_ERR_ARG;
  if (N_max % 4 == 0 && !aligned(slots, 16)) return TSD_ERR_ARG;
  const SlotArgs a{prefix_len, n_new, B, N_max, block_table, max_blocks, held, free_list, free_count,
                   num_blocks, slots, status};
  return slots_launch<true>(a, workspace, ws_bytes, stream);
}

TSD_API int tsd_kv_blocks_release(const int32_t *keep_len, int B, int32_t *block_table,
                                  int max_blocks, int32_t *held, int32_t *free_list,
                                  int32_t *free_count, int num_blocks, void *workspace,
                                  size_t ws_bytes, int32_t *status, tsd_stream_t stream) {
  using namespace tsd;
  const int rc = slots_check(B, 0, max_blocks, num_blocks);
  if (rc != TSD_OK || B == 0) return rc;
  if (!keep_len || !block_table || !held || !free_list || !free_count) return TSD_ERR_ARG;
  const SlotArgs a{keep_len, nullptr, B, 0, block_table, max_blocks, held, free_list, free_count,
                   num_blocks, nullptr, status};
  return slots_launch<false>(a, workspace, ws_bytes, stream);
}
