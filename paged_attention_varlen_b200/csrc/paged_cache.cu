// paged_cache.cu -- the bookkeeping of a serving step on the device: block tables, slot map, positions and
// cumulative lengths from the requests' lengths (ala_paged_step), and the store of a step's new K / V rows
// into the cache by slot (ala_paged_write).
#include <algorithm>

#include "../../include/ala.h"
#include "paged.h"
#include "ptx.cuh"

namespace ala {

namespace {

// ---------------------------------------------------------------------------------------------- step
// With b the requests, n_b new tokens, c_b keys cached before (0 for a request that ended), s the block size:
//   kv_b = c_b + n_b,  taken_b = ceil(kv_b / s) - ceil(c_b / s),  given_b = ceil(old c_b / s) if it ended
// the blocks of ended requests go onto the stack in request order, new blocks come off its top in request
// order, and token t of request b at position c_b + t has slot table[b][pos / s] * s + pos % s.
//
// Three exclusive sums over the batch are all it takes, so every CTA computes them for itself (one thread a
// few rows) and keeps them in shared memory; the CTAs then share the rows and the tokens.  The one order
// between them, pushes before pops and reads of the inputs before writes of outputs that may be the same
// memory, is a cluster barrier, so a step is one launch.
//
// Launch and a chain of memory latencies bound it.  Measured: 56 requests, 48 of them with a token, one CTA: 6 us (2 of them
// the launch).  1000 requests, 90 of them ended, 79000 tokens: 13.6 us with 16 CTAs (the largest cluster), 17 with 8,
// 21 with one block move or token at a time.
constexpr int kStepThreads = 1024;
constexpr int kStepCluster = 16;

struct StepRow {
  int cu, taken, given, before;  // sums over earlier rows, and this row's keys cached before
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Both kernels are programmatic dependent launches, and wait (dependency_wait) before they touch memory.

// A warp moves n block numbers, eight loads in flight in each lane: a request of 12000 keys holds 750 blocks of 16.
template <class Load, class Store>
__device__ __forceinline__ void move_blocks(int n, int lane, Load load, Store store) {
  constexpr int U = 8;
  for (int i0 = lane; i0 < n; i0 += 32 * U) {
    int blk[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + 32 * u < n) blk[u] = load(i0 + 32 * u);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + 32 * u < n) store(i0 + 32 * u, blk[u]);
  }
}

__global__ void __launch_bounds__(kStepThreads, 1) paged_step_kernel(const PagedStepArgs a) {
  extern __shared__ StepRow rows[];  // [batch + 1]
  __shared__ int64_t warp_sum[3][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const int bs = a.block_size;
  const int64_t room = (int64_t)a.max_blocks * bs;
  const int per = (a.batch + threads - 1) / threads;
  const int first = min(tid * per, a.batch), last = min(first + per, a.batch);
  const bool wide = ((reinterpret_cast<uintptr_t>(a.slot_mapping) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0;
  dependency_wait();  // of what comes before on the stream; nothing was read until here
  const int count = *a.free_count;
  auto blocks_of = [&](int keys) { return (int)(((unsigned)keys + (unsigned)bs - 1) / (unsigned)bs); };  // keys <= 2^30

  // ---- this thread's rows: their sums, and whether a length is out of range
  int64_t sum[3] = {0, 0, 0};
  bool bad = false;
  for (int b = first; b < last; ++b) {
    const int n = a.seq_len[b], ctx = a.context_len[b];
    const bool ended = a.finished && a.finished[b] != 0;
    const int64_t kv = (int64_t)n + (ended ? 0 : ctx);
    if (n < 0 || ctx < 0 || ctx > room || kv > room) {
      bad = true;
      break;
    }
    sum[0] += n;
    sum[1] += blocks_of((int)kv) - (ended ? 0 : blocks_of(ctx));
    sum[2] += ended ? blocks_of(ctx) : 0;
  }
  int64_t x[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    x[i] = sum[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x[i], o);
      if (lane >= o) x[i] += y;
    }
    if (lane == 31) warp_sum[i][warp] = x[i];
  }
  bad = __syncthreads_or(bad);
  int64_t total[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int64_t mine = lane < threads / 32 ? warp_sum[i][lane] : 0;
    int64_t before = lane < warp ? mine : 0, all = mine;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      before += __shfl_xor_sync(0xffffffffu, before, o);
      all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    x[i] += before - sum[i];  // exclusive
    total[i] = all;
  }
  const int code = bad                                                ? ALA_STEP_BAD_LENGTH
                   : total[0] > a.n_tokens                            ? ALA_STEP_TOO_MANY_TOKENS
                   : count < 0 || (int64_t)count + total[2] > a.capacity ? ALA_STEP_BAD_FREE_COUNT
                   : total[1] > count + total[2]                      ? ALA_STEP_OUT_OF_BLOCKS
                                                                      : 0;
  if (code != 0) {  // the same for every CTA: the step changes nothing
    cluster_sync();  // every CTA has read its inputs
    const int t0 = blockIdx.x * threads + tid, stride = gridDim.x * threads;
    for (int b = t0; b < a.batch; b += stride)
      if (a.kv_seq_len != a.context_len) a.kv_seq_len[b] = a.context_len[b];
    for (int b = t0; b <= a.batch; b += stride) a.cu_seq_len[b] = 0;
    for (int t = t0; t < a.n_tokens; t += stride) {
      a.slot_mapping[t] = -1;
      a.positions[t] = 0;
    }
    if (t0 == 0) {
      *a.free_count_out = count;
      *a.status = code;
    }
    return;
  }
  {
    int64_t cu = x[0], taken = x[1], given = x[2];
    for (int b = first; b < last; ++b) {
      const int n = a.seq_len[b], ctx = a.context_len[b];
      const bool ended = a.finished && a.finished[b] != 0;
      const int before = ended ? 0 : ctx;
      rows[b] = StepRow{(int)cu, (int)taken, (int)given, before};
      cu += n;
      taken += blocks_of(before + n) - blocks_of(before);
      given += ended ? blocks_of(ctx) : 0;
    }
    if (tid == 0) rows[a.batch] = StepRow{(int)total[0], (int)total[1], (int)total[2], 0};
  }
  __syncthreads();

  // ---- blocks of ended requests onto the stack, one warp per row
  const int warps = gridDim.x * (threads / 32), w0 = blockIdx.x * (threads / 32) + warp;
  bool bad_block = false;
  if (total[2] > 0) {
    for (int b = w0; b < a.batch; b += warps) {
      const int at = count + rows[b].given, n = rows[b + 1].given - rows[b].given;
      const int32_t* row = a.block_tables + (int64_t)b * a.max_blocks;
      move_blocks(n, lane, [&](int i) { return row[i]; },
                  [&](int i, int blk) {
                    bad_block |= blk < 0 || blk >= a.capacity;
                    a.free_blocks[at + i] = blk;
                  });
    }
  }
  // one thread clears the status before any CTA may report into it
  if (blockIdx.x == 0 && tid == 0) *a.status = 0;
  cluster_sync();

  // ---- new blocks off its top; what other CTAs pushed is read past L1
  const int top = count + (int)total[2];
  for (int b = w0; b < a.batch; b += warps) {
    const StepRow r = rows[b];
    const int n = rows[b + 1].taken - r.taken, have = blocks_of(r.before);
    int32_t* row = a.block_tables + (int64_t)b * a.max_blocks;
    move_blocks(n, lane, [&](int i) { return __ldcg(a.free_blocks + (top - 1 - r.taken - i)); },
                [&](int i, int blk) {
                  bad_block |= blk < 0 || blk >= a.capacity;
                  row[have + i] = blk;
                });
    if (lane == 0) {
      a.kv_seq_len[b] = r.before + (rows[b + 1].cu - r.cu);
      a.cu_seq_len[b] = r.cu;
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.cu_seq_len[a.batch] = (int)total[0];
    *a.free_count_out = top - (int)total[1];
  }
  // ---- slot and position of every token, four at a time (one search, loads in flight together); a page that a row
  // already had is in its table, a new one is still on the stack's top (nothing is written over it here)
  for (int t0 = 4 * (blockIdx.x * threads + tid); t0 < a.n_tokens; t0 += 4 * gridDim.x * threads) {
    int slot[4], pos[4];
    int lo = 0, hi = a.batch;  // the last row with cu <= t0
    if (t0 < total[0])
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (rows[mid].cu <= t0) lo = mid;
        else hi = mid;
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + i;
      slot[i] = -1;
      pos[i] = 0;
      if (t < total[0]) {
        while (rows[lo + 1].cu <= t) ++lo;  // ends at the last row: rows[batch].cu is the total
        const StepRow r = rows[lo];
        pos[i] = r.before + t - r.cu;
        const int page = (unsigned)pos[i] / (unsigned)bs, have = blocks_of(r.before);
        const int blk = page < have ? a.block_tables[(int64_t)lo * a.max_blocks + page]
                                    : __ldcg(a.free_blocks + (top - 1 - r.taken - (page - have)));
        if (blk >= 0 && blk < a.capacity) slot[i] = blk * bs + pos[i] - page * bs;
        else bad_block = true;
      }
    }
    if (wide && t0 + 4 <= a.n_tokens) {
      *reinterpret_cast<int4*>(a.slot_mapping + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t0 + i >= a.n_tokens) break;
        a.slot_mapping[t0 + i] = slot[i];
        a.positions[t0 + i] = pos[i];
      }
    }
  }
  if (bad_block) *a.status = ALA_STEP_BAD_BLOCK;
}

// ---------------------------------------------------------------------------------------------- write
// Token t's K row goes to row slots[t] of the K cache and its V row to the same row of the V cache; slots
// outside the cache (-1: padding) are skipped.  Nothing is computed: bytes bound it, so every thread has kWriteLoads
// loads in flight before its first store.  The tokens' rows (K, then V) form one line of vectors, of which a block takes
// kWriteBlock, so that this holds whatever the rows' size.
// Measured: 40000 tokens of 8 heads of 128 in bf16: 50 to 51 us, 6.5 TB/s (a copy: 6.5); 120 tokens: 2 us, the launch.
// Against a group of threads for each token: 18939 tokens of 11 heads of 192 69 -> 55 us, 28237 of a latent cache's
// 512 + 64 in fp32 31 -> 25 us, sizes that fill such groups alike.
constexpr int kWriteLoads = 4, kWriteBlock = 256 * kWriteLoads;
template <typename V>
__global__ void __launch_bounds__(256) paged_write_kernel(const PagedWriteArgs a) {
  const unsigned nk = (unsigned)(a.key_row / sizeof(V)), n = nk + (unsigned)(a.value_row / sizeof(V));
  const int64_t first = (int64_t)blockIdx.x * kWriteBlock;
  const int64_t t0 = first / n;  // the block's first vector: its token, and its place in the row
  const unsigned j0 = (unsigned)(first - t0 * n);
  dependency_wait();
  V r[kWriteLoads];
  V* to[kWriteLoads];
#pragma unroll
  for (int u = 0; u < kWriteLoads; ++u) {
    const unsigned i = j0 + u * 256 + threadIdx.x, row = i / n, j = i - row * n;
    const int64_t t = t0 + row;
    to[u] = nullptr;
    if (t >= a.n_tokens) continue;
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.n_slots) continue;
    const bool key = j < nk;
    const uint8_t* from = key ? a.key + t * a.key_stride : a.value + t * a.value_stride;
    uint8_t* at = key ? a.key_cache + slot * a.key_row : a.value_cache + slot * a.value_row;
    const unsigned k = key ? j : j - nk;
    r[u] = reinterpret_cast<const V*>(from)[k];
    to[u] = reinterpret_cast<V*>(at) + k;
  }
#pragma unroll
  for (int u = 0; u < kWriteLoads; ++u)
    if (to[u]) *to[u] = r[u];
}

template <typename V>
cudaError_t write_as(const PagedWriteArgs& a, cudaStream_t stream) {
  const int64_t n = (a.key_row + a.value_row) / (int64_t)sizeof(V);
  // what the kernel counts in 32 bits; rows of 2 GB at least, or 2 TB in all
  if (n > INT32_MAX - kWriteBlock) return cudaErrorInvalidConfiguration;
  const int64_t blocks = (a.n_tokens * n + kWriteBlock - 1) / kWriteBlock;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_write_kernel<V>, a);
}

}  // namespace

cudaError_t launch_paged_step(const PagedStepArgs& a, cudaStream_t stream) {
  const int smem = (int)sizeof(StepRow) * (a.batch + 1);
  // One CTA of 256 threads where that has little to do, else the cluster, whose barrier and wider sums cost 1 us.  One CTA
  // against the cluster, 1000 keys each: 1 request 3.1 and 4.3 us, 56 5.6 and 6.1, 128 7.3 and 6.1, 256 10.2 and 6.2; 4 of
  // 256 tokens 4.5 and 5.6, 8 of 256 6.4 and 5.8.
  const bool small = a.n_tokens <= 1024 && a.batch <= 64;
  if (!small) {
    const cudaError_t e = cudaFuncSetAttribute(paged_step_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  if (smem > 40 * 1024) {  // above what a kernel may have without asking
    const cudaError_t e = cudaFuncSetAttribute(paged_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(StepRow) * (kPagedStepMaxBatch + 1));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  const int ctas = small ? 1 : kStepCluster;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(small ? 256 : kStepThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, paged_step_kernel, a);
}

cudaError_t launch_paged_write(const PagedWriteArgs& a, cudaStream_t stream) {
  if (a.n_tokens == 0 || a.n_slots == 0 || a.key_row + a.value_row == 0) return cudaSuccess;
  // the widest access that every address, stride and row allows: 16-byte rows are the rule, the others serve
  // odd row sizes and views
  const uint64_t all = reinterpret_cast<uint64_t>(a.key) | reinterpret_cast<uint64_t>(a.value) |
                       reinterpret_cast<uint64_t>(a.key_cache) | reinterpret_cast<uint64_t>(a.value_cache) |
                       (uint64_t)a.key_stride | (uint64_t)a.value_stride | (uint64_t)a.key_row | (uint64_t)a.value_row;
  if (all % 16 == 0) return write_as<uint4>(a, stream);
  if (all % 4 == 0) return write_as<uint32_t>(a, stream);
  return write_as<uint8_t>(a, stream);
}

}  // namespace ala
