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
  int32_t head_stride;             // 1: the line holds all kv heads; kv_heads: a line for each, CTA c on that of head c % kv_heads
  float scale_log2, norm_eps, out_scale;

  __host__ __device__ int maps() const { return dq == row ? 1 : 2; }
};

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

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* a) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a[0]), "r"(a[1]), "r"(a[2]),
               "r"(a[3]), "r"(a[4]), "r"(a[5]), "r"(a[6]), "r"(a[7])
               : "memory");
}
__device__ __forceinline__ void st_global_v4(void* p, const uint32_t* a) {
  asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]) : "memory");
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

// ---------------------------------------------------------------------------------------------- the work line

// One sequence as the kernel takes it: lengths outside what the tensors hold are cut to it.  Keys stay below
// 2^30 (the plan checks it), so all but sums over sequences or row tiles is 32-bit arithmetic.
struct Seq {
  int seq, kv, tiles;  // new tokens, keys, row tiles
};

__device__ __forceinline__ int raw_len(const PagedParams& p, int b) { return min(max(__ldg(p.seq_len + b), 0), p.n_tokens); }

__device__ __forceinline__ Seq make_seq(const PagedParams& p, int64_t cu, int raw, int kv) {
  Seq s;
  s.seq = (int)max((int64_t)0, min((int64_t)raw, p.n_tokens - cu));
  s.kv = min(max(kv, 0), p.max_blocks * p.block_size);
  s.tiles = (int)((unsigned)(s.seq + p.tb - 1) / (unsigned)p.tb);
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
    --r;
  }
  // full row tile i (from 1) sees off + i tb keys: one tile while that is at most TK, then ceil(. / TK)
  const int off = s.kv - s.seq;
  const int ones = off >= TK ? 0 : min((int)((unsigned)(TK - off) / (unsigned)p.tb), r);
  const int m = r - ones;
  return last + ones + (m > 0 ? floor_sum((uint32_t)m, TK, p.tb, (uint64_t)(off + (int64_t)(ones + 1) * p.tb + TK - 1)) : 0);
}

// A CTA's position on the work line: item (b, h, rt) and its tiles [t0, t1) of n.
template <int TK>
struct Walker {
  int b, h, rt, t0, t1, n;
  int raw, raw_next, kv_next;  // the next sequence's lengths are fetched ahead, so that no item waits for them
  int64_t cu, left;
  Seq s;

  __device__ __forceinline__ void fetch(const PagedParams& p) {
    if (b + 1 < p.batch) {
      raw_next = raw_len(p, b + 1);
      kv_next = __ldg(p.kv_seq_len + b + 1);
    }
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
          raw = raw_next;
          s = make_seq(p, cu, raw, kv_next);
          fetch(p);
        } while (s.seq == 0);
      }
    }
    enter(p);
    return true;
  }
  __device__ __forceinline__ int tokens(const PagedParams& p) const { return min(p.tb, s.seq - rt * p.tb); }
};

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
    raw = min(max(len, 0), p.n_tokens);
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
    per_head = b < p.batch && s.seq > 0 ? tiles_before<TK>(p, s, s.tiles) : 0;
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
  const int parts = (int)min((int64_t)(gridDim.x / p.head_stride), total);
  const int part = blockIdx.x / p.head_stride;
  if (threadIdx.x == 0) {
    st->total = total;
    st->parts = parts;
    st->b = -1;
  }
  if (part >= parts) return;
  // 64-bit division only where the numbers need it
  const bool small = total < (1 << 24);
  const int64_t start = small ? (unsigned)total * part / (unsigned)parts : part * total / parts;
  const int64_t end = small ? (unsigned)total * (part + 1) / (unsigned)parts : (part + 1) * total / parts;
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
    int lo = 0, hi = q.tiles;  // the row tile lies in [lo, hi): 32 candidates a round
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int c = lo + (lane + 1) * step;
      const bool below = c < hi && tiles_before<TK>(p, q, c) <= tile;
      const int k = __popc(__ballot_sync(0xffffffffu, below));
      lo += k * step;
      hi = min(hi, lo + step);
    }
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
// Other CTAs wrote them, so they are read past L1.
template <typename T, int D>
__device__ __forceinline__ void combine_row(const PagedParams& p, const PagedDesc& d, int first, int tok, int hh) {
  constexpr int NB = D == 256 ? 1 : 2;
  constexpr int N = D / 32;                   // columns per lane
  constexpr int NW = (kGrid + 31) / 32;       // segment weights per lane
  const int lane = threadIdx.x & 31;
  const int maps = p.maps(), gh = p.group / maps;
  const int col = lane * N;
  float y[N];
  float lse = 0.f;
  const int token = d.token0 + tok, head = (d.kv_head * gh + hh) * maps;
  for (int map = 0; map < maps; ++map) {
    const int r = partial_row(p, d.two, tok, hh, map);
    // segment s lies in CTA first + s * head_stride: in its slot 1 where the item starts, in slot 0 after that
    auto prow = [&](int s) { return ((int64_t)(first + s * p.head_stride) * 2 + (s == 0 ? 1 : 0)) * (NB * 128) + r; };
    float wt[NW], top = -INFINITY, sum = 0.f;
    float2 ml[NW];
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const int s = k * 32 + lane;
      ml[k] = s < d.n_seg ? __ldcg(p.ml + prow(s)) : make_float2(-INFINITY, 0.f);
      top = fmaxf(top, ml[k].x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      wt[k] = fast_exp2(ml[k].x - base);
      sum = fmaf(ml[k].y, wt[k], sum);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const int n = min(32, d.n_seg - k * 32);
#pragma unroll 8
      for (int s = 0; s < n; ++s) {
        const float f = __shfl_sync(0xffffffffu, wt[k], s);
        if (col < p.row) {
          float v[N];
          load_f<N>(p.part + prow(k * 32 + s) * D + col, v);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] = fmaf(f, v[i], acc[i]);
        }
      }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    if (map == 0) {
      lse = sum > 0.f ? top * kLn2 + logf(sum) : -INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = acc[i] * inv;
    } else {
      const float f = -p.lambda[head >> 1] * inv;
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = fmaf(f, acc[i], y[i]);
    }
  }
  if (maps == 2) {
    float post = p.out_scale;
    if (p.norm_weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
      for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      post *= rsqrtf(ss / static_cast<float>(p.row) + p.norm_eps);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] *= post * (p.norm_weight && col + i < p.row ? __ldg(p.norm_weight + col + i) : 1.f);
  } else if (p.lse && lane == 0) {
    if (p.mask_type == 5) lse += p.slopes[head] * static_cast<float>(d.pos0 + tok);
    p.lse[(int64_t)token * p.heads + head] = lse;
  }
  if (col < p.row) {
    uint32_t o[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) o[i] = pack2(y[2 * i], y[2 * i + 1], (T*)nullptr);
    T* dst = static_cast<T*>(p.out) + ((int64_t)token * (p.heads / maps) + head / maps) * p.row + col;
    if constexpr (N == 2) *reinterpret_cast<uint32_t*>(dst) = o[0];
    else if constexpr (N == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ---------------------------------------------------------------------------------------------- launches

// Every kernel here is a programmatic dependent launch: it is scheduled while the one before it on the stream ends,
// and waits here, before it touches memory, until that has completed.
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
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
