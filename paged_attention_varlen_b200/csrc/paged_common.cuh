// paged_common.cuh -- what the kernels of ala_paged_attention share: their parameters, the line of key tiles that
// the CTAs split, and small helpers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "paged.h"
#include "ptx.cuh"

namespace ala {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: rescale O only when the max grows by > 2^8
constexpr float kNoKey = -3.0e38f;         // a running maximum before any key: below every score, and finite
constexpr int kGrid = 148;                 // one CTA per SM of a B200

// What a split item's first CTA leaves for the combine kernel.
struct PagedDesc {
  int32_t n_seg;    // CTAs that hold a segment of the item (0: this CTA starts no split item); head_stride apart
  int32_t token0;   // first token of the row tile
  int32_t tokens;   // its tokens
  int32_t kv_head;
  int32_t pos0;     // absolute position of token0
  int32_t two;      // rows in two blocks
};

struct PagedParams {
  const int32_t *seq_len, *kv_seq_len, *block_tables;
  const float *slopes, *lambda, *norm_weight;
  const void* q;
  void* out;
  float* lse;
  int* status;
  int* arrived;     // [kGrid]: segments of the item that starts in a CTA (few rows), 0 between executions
  PagedDesc* desc;  // [kGrid]
  float2* ml;       // [kGrid][2][128 NB]: running max (log2 units) and sum of each partial row
  float* part;      // [kGrid][2][128 NB][D]
  int64_t q_stride;
  int32_t n_tokens, batch, max_blocks, block_size, num_blocks, mask_type;
  int32_t heads, group, kv_heads;  // query heads, per kv head (both maps counted)
  int32_t tb1, tb;                 // tokens of one block of rows (128 / group), tokens per row tile
  int32_t dq, row;                 // query head size, elements of a K / V row
  int32_t box_rows;
  int32_t small;                   // few rows: at most 64 sequences whose lengths, whatever they are, make fewer than 2^24 tiles
  int32_t rows_min, rows_max;      // sequences with rows (per kv head) outside this range are another launch's
  int32_t head_stride;             // 1: the line holds all kv heads; kv_heads: a line for each, CTA c on that of head c % kv_heads
  float scale_log2, norm_eps, out_scale;

  __host__ __device__ int maps() const { return dq == row ? 1 : 2; }
};

// 1 / sqrt(mean square + eps) of a row whose squares add up to ss; 0 for a row of zeros without an epsilon (a row without
// a key is one), which then stays zeros.  A NaN row's values are NaN without it.
__device__ __forceinline__ float inv_rms(const PagedParams& p, float ss) {
  const float ms = ss / static_cast<float>(p.row) + p.norm_eps;
  return ms > 0.f ? rsqrtf(ms) : 0.f;
}

// Row of an item's partials that holds (token of the tile, head of the group without its map, map).
__device__ __forceinline__ int partial_row(const PagedParams& p, bool two, int token, int hh, int map) {
  const int maps = p.maps();
  if (!two) return token * p.group + hh * maps + map;
  if (maps == 2) return map * 128 + token * (p.group / 2) + hh;
  return token < p.tb1 ? token * p.group + hh : 128 + (token - p.tb1) * p.group + hh;
}

template <typename T>
struct ElemFmt;
template <>
struct ElemFmt<__half> {
  static constexpr uint32_t fmt = 0;
};
template <>
struct ElemFmt<__nv_bfloat16> {
  static constexpr uint32_t fmt = 1;
};

// 16 bytes of a query row.  attnOut may be the same memory, which the kernel writes, so this is no read-only load (__ldg);
// not volatile either, so that it is scheduled like one (a plain load, which stays behind the barriers before it, took
// four chunks of 40 tokens from 23.6 to 24.5 us).  Its address comes from the lengths, which keeps it behind the
// dependency wait.
__device__ __forceinline__ uint4 ld_query(const uint4* p) {
  uint4 v;
  asm("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* a) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a[0]), "r"(a[1]), "r"(a[2]),
               "r"(a[3]), "r"(a[4]), "r"(a[5]), "r"(a[6]), "r"(a[7])
               : "memory");
}
__device__ __forceinline__ void st_global_v4(void* p, const uint32_t* a) {
  asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]) : "memory");
}

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16*) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half*) {
  __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

template <typename T>
__device__ __forceinline__ T from_float(float x) {
  if constexpr (sizeof(T) == 2 && ElemFmt<T>::fmt == 1) return __float2bfloat16_rn(x);
  else return __float2half_rn(x);
}
__device__ __forceinline__ float2 unpack2(uint32_t v, __nv_bfloat16*) {
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&v));
}
__device__ __forceinline__ float2 unpack2(uint32_t v, __half*) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }

// Whether a wait has run out in this workspace since its status was cleared: the counters of cut items may then be left
// half way, so that later executions write nothing (until the workspace is bound again).  One thread of a CTA reads it,
// beside the lengths, and the CTA leaves by a vote: a CTA of the same launch may be failing meanwhile, so that two reads
// need not agree.
__device__ __forceinline__ int wait_failed(const PagedParams& p) {
  return threadIdx.x == 0 && *reinterpret_cast<const volatile int*>(p.status) != 0;
}

// ---------------------------------------------------------------------------------------------- the work line

// One sequence as the kernel takes it: lengths outside what the tensors hold are cut to it.  Keys stay below
// 2^30 (the plan checks it), so all but sums over sequences or row tiles is 32-bit arithmetic.
struct Seq {
  int seq, kv, tiles;  // new tokens, keys, row tiles (0: nothing here for this launch)
};

__device__ __forceinline__ int clamp_len(const PagedParams& p, int len) { return min(max(len, 0), p.n_tokens); }

__device__ __forceinline__ Seq make_seq(const PagedParams& p, int64_t cu, int raw, int kv) {
  Seq s;
  s.seq = (int)max((int64_t)0, min((int64_t)raw, p.n_tokens - cu));
  s.kv = min(max(kv, 0), p.max_blocks * p.block_size);
  const int64_t rows = (int64_t)s.seq * p.group;
  s.tiles = rows < p.rows_min || rows > p.rows_max ? 0 : s.seq <= p.tb ? s.seq > 0 : (int)((unsigned)(s.seq + p.tb - 1) / (unsigned)p.tb);
  return s;
}

// Key tiles of row tile `rt`: up to the last key its last token may see, and at least one, so that rows
// without keys are written too.
template <int TK>
__device__ __forceinline__ int key_tiles(const PagedParams& p, const Seq& s, int rt) {
  int keys = s.kv;
  if (p.mask_type != 0) keys = max(0, min((rt + 1) * p.tb, s.seq) + s.kv - s.seq);
  return max(1, (int)((unsigned)(keys + TK - 1) / TK));
}

// sum over i < n of floor((a i + b) / m), by Euclid's steps on (a, m)
__device__ __forceinline__ int64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint64_t b) {
  uint64_t s = 0;
  for (;;) {
    if (a >= m) {
      s += (uint64_t)n * (n - 1u) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      s += n * (b / m);
      b %= m;
    }
    const uint64_t y = (uint64_t)a * n + b;
    if (n == 0 || y < m) return (int64_t)s;
    n = (uint32_t)(y / m);
    b = y % m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
}

// Key tiles of the first r row tiles of one kv head.
template <int TK>
__device__ int64_t tiles_before(const PagedParams& p, const Seq& s, int r) {
  if (r == 0) return 0;
  if (p.mask_type == 0) return (int64_t)r * key_tiles<TK>(p, s, 0);
  int64_t last = 0;
  if (r == s.tiles) {  // the last row tile may be short
    last = key_tiles<TK>(p, s, r - 1);
    if (--r == 0) return last;
  }
  // full row tile i (from 1) sees off + i tb keys: one tile while that is at most TK, then ceil(. / TK)
  const int off = s.kv - s.seq;
  const int ones = off >= TK ? 0 : min((int)((unsigned)(TK - off) / (unsigned)p.tb), r);
  const int m = r - ones;
  return last + ones + (m > 0 ? floor_sum((uint32_t)m, TK, p.tb, (uint64_t)(off + (int64_t)(ones + 1) * p.tb + TK - 1)) : 0);
}

struct Start {
  int b, h, rt, t0, raw;
  Seq s;
  int64_t cu, left, line, total;  // line: this CTA's first tile on its line of `total` tiles
  int parts;                      // CTAs that share the line

  // The part q of a tile: the last with q * total / parts <= tile.
  __device__ __forceinline__ int part_of(int64_t tile) const {
    return total < (1 << 24) ? (int)(((unsigned)(tile + 1) * (unsigned)parts - 1) / (unsigned)total)
                             : (int)(((tile + 1) * parts - 1) / total);
  }
};

// A CTA's position on the work line: item (b, h, rt) and its tiles [t0, t1) of n.
template <int TK>
struct Walker {
  int b, h, rt, t0, t1, n;
  int raw, len_next, kv_next;  // the next sequence's lengths, as they lie in memory, are fetched ahead of their use
  int64_t cu, left;
  Seq s;

  __device__ __forceinline__ void fetch(const PagedParams& p) {
    if (b + 1 < p.batch) {
      len_next = __ldg(p.seq_len + b + 1);
      kv_next = __ldg(p.kv_seq_len + b + 1);
    }
  }
  __device__ __forceinline__ void begin(const PagedParams& p, const Start& st) {
    b = st.b;
    h = st.h;
    rt = st.rt;
    t0 = st.t0;
    raw = st.raw;
    cu = st.cu;
    left = st.left;
    s = st.s;
    fetch(p);
    enter(p);
  }
  __device__ __forceinline__ void enter(const PagedParams& p) {
    n = key_tiles<TK>(p, s, rt);
    t1 = (int)min((int64_t)n, t0 + left);
  }
  __device__ __forceinline__ bool next(const PagedParams& p) {
    left -= t1 - t0;
    if (left <= 0) return false;
    t0 = 0;
    if (++rt == s.tiles) {
      rt = 0;
      if (p.head_stride > 1 || ++h == p.kv_heads) {
        if (p.head_stride == 1) h = 0;
        do {
          cu += raw;
          if (++b >= p.batch) return false;
          raw = clamp_len(p, len_next);
          s = make_seq(p, cu, raw, kv_next);
          fetch(p);
        } while (s.tiles == 0);
      }
    }
    enter(p);
    return true;
  }
  __device__ __forceinline__ int tokens(const PagedParams& p) const { return min(p.tb, s.seq - rt * p.tb); }
};

// CTAs that share a line of `total` tiles: no more than give every one as many tiles as the busiest has anyway, so
// that a short line is not cut for nothing.
__device__ __forceinline__ int parts_of(const PagedParams& p, int64_t total) {
  const int most = gridDim.x / p.head_stride;
  if (total >= 64 * (int64_t)most) return most;
  const unsigned t = (unsigned)total;
  if (t == 0) return 0;
  const unsigned each = (t + most - 1) / most;
  return (int)((t + each - 1) / each);
}

// First tile of part q; 64-bit division only where the numbers need it.
__device__ __forceinline__ int64_t cut(int64_t total, int parts, int q) {
  return total < (1 << 24) ? (unsigned)total * (unsigned)q / (unsigned)parts : q * total / parts;
}

// The row tile that holds a tile of the head, by a whole warp, 32 candidates a round.
template <int TK>
__device__ __forceinline__ int find_row_tile(const PagedParams& p, const Seq& q, int64_t tile) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = q.tiles;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int c = lo + (lane + 1) * step;
    const bool below = c < hi && tiles_before<TK>(p, q, c) <= tile;
    const int k = __popc(__ballot_sync(0xffffffffu, below));
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The same as find_start where p.small, by every warp for itself: two sequences a lane, 32-bit numbers in registers,
// no meeting of the warps.  A single token of a single user spends 2 us less here.
template <int TK>
__device__ __forceinline__ void find_start_small(const PagedParams& p, Start& st) {
  const int lane = threadIdx.x & 31;
  int len[2], keys[2], raw[2], w[2], per_head[2];
  Seq s[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = 2 * lane + k;
    len[k] = b < p.batch ? __ldg(p.seq_len + b) : 0;
    keys[k] = b < p.batch ? __ldg(p.kv_seq_len + b) : 0;
    raw[k] = clamp_len(p, len[k]);
  }
  int x = raw[0] + raw[1];  // below 64 * 2^24
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  const int cu[2] = {x - raw[0] - raw[1], x - raw[1]};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    s[k] = make_seq(p, cu[k], raw[k], keys[k]);
    per_head[k] = s[k].tiles > 0 ? (int)tiles_before<TK>(p, s[k], s[k].tiles) : 0;
    w[k] = p.head_stride > 1 ? per_head[k] : per_head[k] * p.kv_heads;
    if (blockIdx.x == 0 && threadIdx.x < 32 && 2 * lane + k < p.batch && (s[k].seq != len[k] || s[k].kv != keys[k]))
      atomicCAS(p.status + 1, 0, kDevBadLength);
  }
  int z = w[0] + w[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, z, o);
    if (lane >= o) z += y;
  }
  const int total = __shfl_sync(0xffffffffu, z, 31);
  const int before[2] = {z - w[0] - w[1], z - w[1]};
  const int parts = parts_of(p, total), part = blockIdx.x / p.head_stride;
  st.total = total;
  st.parts = parts;
  st.b = -1;
  if (part >= parts) return;
  const int start = (int)((unsigned)total * (unsigned)part / (unsigned)parts);
  const int end = (int)((unsigned)total * (unsigned)(part + 1) / (unsigned)parts);
  const bool in1 = before[1] <= start && start < before[1] + w[1];
  const bool in0 = before[0] <= start && start < before[0] + w[0];
  const int src = __ffs(__ballot_sync(0xffffffffu, in0 || in1)) - 1;
  const int k = __shfl_sync(0xffffffffu, (int)in1, src);
  auto pick = [&](int a0, int a1) { return __shfl_sync(0xffffffffu, k ? a1 : a0, src); };
  st.b = 2 * src + k;
  st.raw = pick(raw[0], raw[1]);
  st.cu = pick(cu[0], cu[1]);
  st.s.seq = pick(s[0].seq, s[1].seq);
  st.s.kv = pick(s[0].kv, s[1].kv);
  st.s.tiles = pick(s[0].tiles, s[1].tiles);
  int tile = start - pick(before[0], before[1]);
  st.line = start;
  st.left = end - start;
  st.h = blockIdx.x % p.head_stride;
  if (p.head_stride == 1) {
    const int each = pick(per_head[0], per_head[1]);
    st.h = (unsigned)tile / (unsigned)each;
    tile -= st.h * each;
  }
  st.rt = 0;
  st.t0 = tile;
  if (st.s.tiles > 1) {
    st.rt = find_row_tile<TK>(p, st.s, tile);
    st.t0 = tile - (int)tiles_before<TK>(p, st.s, st.rt);
  }
}

// Every thread of the CTA scans the batch (kThreads sequences at a time); the results are in *st after the
// caller's __syncthreads.  `red` holds 2 * kThreads / 32 words.
template <int TK, int kThreads>
__device__ void find_start(const PagedParams& p, Start* st, int64_t* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = kThreads / 32;
  int cu0 = 0;         // tokens before this chunk; sums of tokens saturate (those past n_tokens are cut anyway)
  int64_t w0 = 0;      // tiles before this chunk
  int raw = 0, cu = 0;
  int64_t w_before = 0, w = 0, per_head = 0;
  Seq s{0, 0, 0};
  auto add = [](int x, int y) { return (int)min((unsigned)x + (unsigned)y, 0x7fffffffu); };
  // a chunk: each thread's sequence, the tokens before it and the tiles before it
  auto scan = [&](int b0) {
    const int b = b0 + threadIdx.x;
    const int len = b < p.batch ? __ldg(p.seq_len + b) : 0, keys = b < p.batch ? __ldg(p.kv_seq_len + b) : 0;
    raw = clamp_len(p, len);
    int x = raw;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = add(x, y);
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    int before = cu0, sum = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before = add(before, (int)red[i]);
      sum = add(sum, (int)red[i]);
    }
    cu = add(before, x - raw);
    cu0 = add(cu0, sum);
    s = make_seq(p, cu, raw, keys);
    per_head = b < p.batch && s.tiles > 0 ? tiles_before<TK>(p, s, s.tiles) : 0;
    w = p.head_stride > 1 ? per_head : per_head * p.kv_heads;
    if (blockIdx.x == 0 && b < p.batch && (s.seq != len || s.kv != keys)) atomicCAS(p.status + 1, 0, kDevBadLength);
    int64_t z = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, z, o);
      if (lane >= o) z += y;
    }
    if (lane == 31) red[kWarps + warp] = z;
    __syncthreads();
    int64_t all = 0;
    w_before = w0 + z - w;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) w_before += red[kWarps + i];
      all += red[kWarps + i];
    }
    w0 += all;
    if (p.batch > kThreads) __syncthreads();  // red is written again
  };
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) scan(b0);
  const int64_t total = w0;
  const int parts = parts_of(p, total);
  const int part = blockIdx.x / p.head_stride;
  if (threadIdx.x == 0) {
    st->total = total;
    st->parts = parts;
    st->b = -1;
  }
  if (part >= parts) return;
  const bool small = total < (1 << 24);
  const int64_t start = cut(total, parts, part), end = cut(total, parts, part + 1);
  __syncthreads();
  auto place = [&](int b0) {
    if (w > 0 && w_before <= start && start < w_before + w) {
      st->b = b0 + threadIdx.x;
      st->raw = raw;
      st->s = s;
      st->cu = cu;
      st->line = start;
      st->left = end - start;
      int h = 0;
      if (p.head_stride == 1) h = small ? (int)((unsigned)(start - w_before) / (unsigned)per_head) : (int)((start - w_before) / per_head);
      red[0] = start - w_before - h * per_head;  // tile within the head
      st->h = p.head_stride > 1 ? blockIdx.x % p.head_stride : h;
    }
  };
  if (p.batch <= kThreads) {
    place(0);
  } else {
    cu0 = 0;
    w0 = 0;
    for (int b0 = 0; b0 < p.batch && w0 <= start; b0 += kThreads) {
      scan(b0);
      place(b0);
    }
  }
  __syncthreads();
  if (warp == 0) {
    const Seq q = st->s;
    const int64_t tile = red[0];
    const int lo = find_row_tile<TK>(p, q, tile);
    if (lane == 0) {
      st->rt = lo;
      st->t0 = (int)(tile - tiles_before<TK>(p, q, lo));
    }
  }
}

// ---------------------------------------------------------------------------------------------- joining segments

template <int N>
__device__ __forceinline__ void load_f(const float* src, float (&v)[N]) {
  if constexpr (N == 2) {
    const float2 a = __ldcg(reinterpret_cast<const float2*>(src));
    v[0] = a.x;
    v[1] = a.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 a = __ldcg(reinterpret_cast<const float4*>(src) + i);
      v[4 * i] = a.x;
      v[4 * i + 1] = a.y;
      v[4 * i + 2] = a.z;
      v[4 * i + 3] = a.w;
    }
  }
}

// One output row (token of the tile, head of the group; both maps of a differential row) of an item that starts in
// CTA `first`, by one warp, its segments in order:
//   m = max_s m_s, O = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s.
// Other CTAs wrote them, so they are read past L1.  Latency is all it costs: the statistics and the first U segments'
// values are fetched together, and the maps too.
template <typename T, int D, int MAPS>
__device__ __forceinline__ void combine_row(const PagedParams& p, const PagedDesc& d, int first, int tok, int hh) {
  constexpr int NB = D == 256 ? 1 : 2;
  constexpr int N = D / 32;                   // columns per lane
  constexpr int U = D == 256 || MAPS == 2 ? 4 : 8;  // segments in flight
  const int lane = threadIdx.x & 31;
  const int gh = p.group / MAPS;
  const int col = lane * N;
  const int token = d.token0 + tok, head = (d.kv_head * gh + hh) * MAPS;
  // segment s lies in CTA first + s * head_stride: in its slot 1 where the item starts, in slot 0 after that
  int r[MAPS];
#pragma unroll
  for (int map = 0; map < MAPS; ++map) r[map] = partial_row(p, d.two, tok, hh, map);
  auto prow = [&](int map, int s) { return ((first + s * p.head_stride) * 2 + (s == 0 ? 1 : 0)) * (NB * 128) + r[map]; };
  // a lane's statistics: of segments lane, lane + 32, ...
  auto stat = [&](int map, int s) { return s < d.n_seg ? __ldcg(p.ml + prow(map, s)) : make_float2(-INFINITY, 0.f); };
  float2 own[MAPS];
#pragma unroll
  for (int map = 0; map < MAPS; ++map) own[map] = stat(map, lane);
  float v[MAPS][U][N];
  auto fetch = [&](int s0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int map = 0; map < MAPS; ++map)
        if (s0 + u < d.n_seg && col < p.row) load_f<N>(p.part + (int64_t)prow(map, s0 + u) * D + col, v[map][u]);
  };
  fetch(0);
  float top[MAPS], sum[MAPS], acc[MAPS][N];  // top is kNoKey at least, as every segment's maximum
#pragma unroll
  for (int map = 0; map < MAPS; ++map) {
    top[map] = own[map].x;
    for (int s = lane + 32; s < d.n_seg; s += 32) top[map] = fmaxf(top[map], stat(map, s).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) top[map] = fmaxf(top[map], __shfl_xor_sync(0xffffffffu, top[map], o));
    sum[map] = own[map].y * fast_exp2(own[map].x - top[map]);
    for (int s = lane + 32; s < d.n_seg; s += 32) {
      const float2 o = stat(map, s);
      sum[map] = fmaf(o.y, fast_exp2(o.x - top[map]), sum[map]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum[map] += __shfl_xor_sync(0xffffffffu, sum[map], o);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[map][i] = 0.f;
  }
  float wt[MAPS];
#pragma unroll 1
  for (int s0 = 0; s0 < d.n_seg; s0 += U) {
    if (s0 > 0) fetch(s0);
    if (s0 % 32 == 0) {
#pragma unroll
      for (int map = 0; map < MAPS; ++map) wt[map] = fast_exp2((s0 == 0 ? own[map] : stat(map, s0 + lane)).x - top[map]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int map = 0; map < MAPS; ++map) {
        const float f = __shfl_sync(0xffffffffu, wt[map], (s0 + u) & 31);
        if (s0 + u < d.n_seg && col < p.row) {
#pragma unroll
          for (int i = 0; i < N; ++i) acc[map][i] = fmaf(f, v[map][u][i], acc[map][i]);
        }
      }
  }
  float y[N];
  const float inv = sum[0] > 0.f ? 1.f / sum[0] : 0.f;  // a row without keys gets 0
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = acc[0][i] * inv;
  if constexpr (MAPS == 2) {
    const float f = sum[1] > 0.f ? -p.lambda[head >> 1] / sum[1] : 0.f;
    float post = p.out_scale, ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      y[i] = fmaf(f, acc[1][i], y[i]);
      ss = fmaf(y[i], y[i], ss);
    }
    if (p.norm_weight) {
#pragma unroll
      for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      post *= inv_rms(p, ss);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] *= post * (p.norm_weight && col + i < p.row ? __ldg(p.norm_weight + col + i) : 1.f);
  } else if (p.lse && lane == 0) {
    float lse = sum[0] != 0.f ? top[0] * kLn2 + logf(sum[0]) : -INFINITY;
    if (p.mask_type == 5) lse += p.slopes[head] * static_cast<float>(d.pos0 + tok);
    p.lse[(int64_t)token * p.heads + head] = lse;
  }
  if (col < p.row) {
    uint32_t o[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) o[i] = pack2(y[2 * i], y[2 * i + 1], (T*)nullptr);
    T* dst = static_cast<T*>(p.out) + ((int64_t)token * (p.heads / MAPS) + head / MAPS) * p.row + col;
    if constexpr (N == 2) *reinterpret_cast<uint32_t*>(dst) = o[0];
    else if constexpr (N == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <typename T, int D>
__device__ __forceinline__ void combine_row(const PagedParams& p, const PagedDesc& d, int first, int tok, int hh) {
  if (p.maps() == 1) combine_row<T, D, 1>(p, d, first, tok, hh);
  else combine_row<T, D, 2>(p, d, first, tok, hh);
}

// ---------------------------------------------------------------------------------------------- waits of a warp in step

__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* status, int code) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status, code));
}
// Two barriers at once: a wait that finds its phase over still costs some 150 cycles, and the issuing warp has six for
// every tile of a block.
__device__ __forceinline__ bool wait_warp2(uint64_t* bar0, uint32_t parity0, int code0, uint64_t* bar1, uint32_t parity1, int code1,
                                           int* status) {
  const bool first = mbar_test_wait(bar0, parity0), second = mbar_try_wait(bar1, parity1);
  if (__all_sync(0xffffffffu, first && second)) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar0, parity0, status, code0)) && __all_sync(0xffffffffu, mbar_wait(bar1, parity1, status, code1));
}

// ---------------------------------------------------------------------------------------------- launches

// Every kernel here is a programmatic dependent launch: it waits (dependency_wait) before it touches memory.
// Lets the next such kernel be scheduled from now on (it waits all the same).
__device__ __forceinline__ void dependency_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Rows of at most kFewRows queries per kv head (paged_few.cu).
constexpr int kFewRows = 32;
cudaError_t launch_paged_few(int32_t dtype, int D, const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedParams& p,
                             cudaStream_t stream);

}  // namespace ala
