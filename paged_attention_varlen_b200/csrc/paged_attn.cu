// paged_attn.cu -- attention of each sequence's new tokens (one, a few, or a chunk) over its paged cache,
// with every length read on the device, and its differential form.
//
//   O[t, h] = sum_j softmax_j(qkScale q[t, h] . k_j + bias) v_j                       (ala_paged_attention)
//   O[t, h] = sum_j (softmax_j(s1) - lambda_h softmax_j(s2)) v_j, s_m = qkScale q[t, 2h + m] . k_(m),j
//             and then, optionally, O <- O * rsqrt(mean(O^2) + eps) * w               (ala_paged_diff_attention)
//
// Rows.  The queries of one kv head are packed (token, head of the group) into tiles of up to 128 rows, so a
// single token of a group of 8 heads is one tile of 8 rows and K / V are read once for the group.
//
// Differential attention is the same kernel over K rows [k1 | k2] of 2d elements, as they lie in the cache:
// the query row of map 1 is [q1 | 0], that of map 2 is [0 | q2], and the two maps of a head are neighbouring
// rows, so that their difference is one shuffle between neighbouring lanes.  Decoding reads the cache once
// and pays nothing for the zeros; a compute-bound chunk pays 8d instead of 6d products per pair.
//
// Work split.  All key tiles of all (sequence, kv head, row tile) items form one line; CTA c of G takes the
// tiles [c T / G, (c + 1) T / G).  A CTA finds its start by a scan over the batch and a search inside one
// sequence, so the schedule needs no host lengths and no planning launch, and every CTA gets the same number
// of tiles whatever the lengths are.  An item cut by a CTA boundary leaves unnormalised fp32 partials with
// the running max and sum of each row; paged_combine_kernel joins them in segment order.
//
// Pipeline of a CTA (one per SM):
//   warps 4, 5  TMA producers of the K and the V ring; lane i gathers box i of a tile through the block table
//   warp 6      tcgen05 issuer: S = Q K^T into one of two TMEM buffers, O += P V with P read from TMEM;
//               QK of tile j + 1 runs while the softmax works on tile j
//   warps 0..3  softmax, thread r owns row r (TMEM lane r).  With 32 rows or fewer, the rows are repeated in
//               the four lane quarters and quarter w takes a quarter of each tile's keys (P is zero on the
//               others), so that all four warps share the exponentials of a single token; the quarters are
//               joined through shared memory at the end of the item.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "internal.h"
#include "paged.h"
#include "ptx.cuh"

namespace ala {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: rescale O only when the max grows by > 2^8
constexpr int kGrid = 148;                 // one CTA per SM of a B200
constexpr int kThreads = 256;
constexpr int kCombineY = 4;               // blocks per segment list in the combine grid

// What a split item's first CTA leaves for the combine kernel.
struct PagedDesc {
  int32_t n_seg;    // CTAs that hold a segment of the item (0: this CTA starts no split item)
  int32_t token0;   // first token of the row tile
  int32_t rows;     // valid rows
  int32_t kv_head;
  int32_t pos0;     // absolute position of token0
};

struct PagedParams {
  const int32_t *seq_len, *kv_seq_len, *block_tables;
  const float *slopes, *lambda, *norm_weight;
  const void* q;
  void* out;
  float* lse;
  int* status;
  PagedDesc* desc;  // [kGrid]
  float2* ml;       // [kGrid][2][128]: running max (log2 units) and sum of each partial row
  float* part;      // [kGrid][2][128][D]
  int64_t q_stride;
  int32_t n_tokens, batch, max_blocks, block_size, num_blocks, mask_type;
  int32_t heads, group, kv_heads;  // query heads, per kv head (both maps counted)
  int32_t tb;                      // tokens per row tile: 128 / group
  int32_t dq, row;                 // query head size, elements of a K / V row
  int32_t box_rows;
  float scale_log2, norm_eps, out_scale;
};

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

// Two S buffers of TK columns and O of D columns fit tensor memory for D up to 256 with 64-key tiles.  The
// rings fill what shared memory leaves: a tile arrives a few thousand cycles after its load is issued, so
// depth is what keeps HBM busy.
template <typename T, int D_>
struct Cfg {
  static constexpr int D = D_;
  static constexpr int TK = D == 256 ? 64 : 128;  // keys per tile
  static constexpr int CB = D / 64;               // 128-byte column blocks of a row
  static constexpr int Q_BYTES = 128 * D * 2;
  static constexpr int KV_BYTES = TK * D * 2;
  static constexpr int NSK = D == 64 ? 6 : 3;
  static constexpr int NSV = D == 64 ? 6 : D == 128 ? 3 : 2;
  static constexpr int N_BARS = 1 + 2 * NSK + 2 * NSV + 2 + 2 + 1 + 1 + 1 + 1;
  static constexpr int SMEM = 1024 + Q_BYTES + (NSK + NSV) * KV_BYTES + 128 * 8 + N_BARS * 8 + 64;
  static constexpr uint32_t IDESC_QK = instr_desc(ElemFmt<T>::fmt, false, false, 128, TK);
  static constexpr uint32_t IDESC_PV = instr_desc(ElemFmt<T>::fmt, false, true, 128, D);
  static constexpr uint32_t O_COL = 2 * TK;  // S0 [0, TK) S1 [TK, 2 TK) O [2 TK, 2 TK + D)
  static constexpr uint32_t TMEM_COLS = 512;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(O_COL + D <= TMEM_COLS, "tensor memory budget");
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

// ---------------------------------------------------------------------------------------------- the work line

// One sequence as the kernel takes it: lengths outside what the tensors hold are cut to it.
struct Seq {
  int seq, kv, tiles;  // new tokens, keys, row tiles
};

__device__ __forceinline__ int raw_len(const PagedParams& p, int b) { return min(max(__ldg(p.seq_len + b), 0), p.n_tokens); }

__device__ __forceinline__ Seq load_seq(const PagedParams& p, int b, int64_t cu, int raw) {
  Seq s;
  s.seq = cu >= p.n_tokens ? 0 : (int)min((int64_t)raw, p.n_tokens - cu);
  const int64_t room = (int64_t)p.max_blocks * p.block_size;
  s.kv = (int)min((int64_t)max(__ldg(p.kv_seq_len + b), 0), room);
  s.tiles = (s.seq + p.tb - 1) / p.tb;
  return s;
}

// Key tiles of row tile `rt`: up to the last key its last token may see, and at least one, so that rows
// without keys are written too.
template <int TK>
__device__ __forceinline__ int key_tiles(const PagedParams& p, const Seq& s, int rt) {
  int64_t keys = s.kv;
  if (p.mask_type != 0) {
    const int64_t end = min((int64_t)(rt + 1) * p.tb, (int64_t)s.seq) + s.kv - s.seq;
    keys = max((int64_t)0, min(end, (int64_t)s.kv));
  }
  return max(1, (int)((keys + TK - 1) / TK));
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
  const int64_t off = (int64_t)s.kv - s.seq;
  int64_t ones = off >= TK ? 0 : (TK - off) / p.tb;
  ones = min(ones, (int64_t)r);
  const int64_t m = r - ones;
  return last + ones + (m > 0 ? floor_sum((uint32_t)m, TK, p.tb, (uint64_t)(off + (ones + 1) * p.tb + TK - 1)) : 0);
}

// A CTA's position on the work line: item (b, h, rt) and its tiles [t0, t1) of n.
template <int TK>
struct Walker {
  int b, h, rt, t0, t1, n;
  int raw;
  int64_t cu, left;
  Seq s;

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
      if (++h == p.kv_heads) {
        h = 0;
        do {
          cu += raw;
          if (++b >= p.batch) return false;
          raw = raw_len(p, b);
          s = load_seq(p, b, cu, raw);
        } while (s.seq == 0);
      }
    }
    enter(p);
    return true;
  }
  __device__ __forceinline__ int rows(const PagedParams& p) const { return min(p.tb, s.seq - rt * p.tb) * p.group; }
};

struct Start {
  int b, h, rt, t0, raw;
  int64_t cu, left, line, total;  // line: this CTA's first tile on the line of `total` tiles
  int ctas;                       // CTAs that take part
};

// Every thread of the CTA scans the batch (kThreads sequences at a time); the results are in *st after the
// caller's __syncthreads.  `red` holds 2 * kThreads / 32 + 2 words.
template <int TK>
__device__ void find_start(const PagedParams& p, Start* st, int64_t* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = kThreads / 32;
  int64_t cu0 = 0, w0 = 0;  // tokens and tiles before this chunk
  int64_t start = 0, end = 0;
  int raw = 0;
  int64_t cu = 0, w_before = 0, w = 0;
  Seq s{0, 0, 0};
  // a chunk: each thread's sequence, the tokens before it and the tiles before it
  auto scan = [&](int b0) {
    const int b = b0 + threadIdx.x;
    raw = b < p.batch ? raw_len(p, b) : 0;
    int64_t x = raw;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    int64_t before = cu0, sum = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += red[i];
      sum += red[i];
    }
    cu = before + x - raw;
    cu0 += sum;
    w = 0;
    if (b < p.batch) {
      s = load_seq(p, b, cu, raw);
      if (s.seq > 0) w = tiles_before<TK>(p, s, s.tiles) * p.kv_heads;
      if (blockIdx.x == 0 && (raw != __ldg(p.seq_len + b) || s.seq != raw || s.kv != __ldg(p.kv_seq_len + b)))
        atomicCAS(p.status + 1, 0, kDevBadLength);
    }
    x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) red[kWarps + warp] = x;
    __syncthreads();
    before = w0;
    sum = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += red[kWarps + i];
      sum += red[kWarps + i];
    }
    w_before = before + x - w;
    w0 += sum;
    __syncthreads();
  };
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) scan(b0);
  const int64_t total = w0;
  const int ctas = (int)min((int64_t)gridDim.x, total);
  if (threadIdx.x == 0) {
    st->total = total;
    st->ctas = ctas;
    st->b = -1;
  }
  if ((int)blockIdx.x >= ctas) return;
  start = blockIdx.x * total / ctas;
  end = (blockIdx.x + 1) * total / ctas;
  __syncthreads();
  auto place = [&](int b0) {
    if (w > 0 && w_before <= start && start < w_before + w) {
      st->b = b0 + threadIdx.x;
      st->raw = raw;
      st->cu = cu;
      st->line = start;
      st->left = end - start;
      const int64_t per_head = w / p.kv_heads;
      st->h = (int)((start - w_before) / per_head);
      red[0] = start - w_before - st->h * per_head;  // tile within the head
    }
  };
  if (p.batch <= kThreads) {
    place(0);
  } else {
    cu0 = w0 = 0;
    for (int b0 = 0; b0 < p.batch && w0 <= start; b0 += kThreads) {
      scan(b0);
      place(b0);
    }
  }
  __syncthreads();
  if (warp == 0) {
    const int b = st->b;
    const Seq q = load_seq(p, b, st->cu, st->raw);
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

// ---------------------------------------------------------------------------------------------- softmax

template <int NC>
__device__ __forceinline__ void load_cols(uint32_t col, float (&x)[NC]) {
  if constexpr (NC >= 32) {
    uint32_t r[NC / 32][32];
#pragma unroll
    for (int i = 0; i < NC / 32; ++i) tmem_ld32(col + i * 32, r[i]);
    tmem_ld_wait();  // one wait for all loads
#pragma unroll
    for (int c = 0; c < NC; ++c) x[c] = __uint_as_float(r[c >> 5][c & 31]);
  } else {
    uint32_t r[16];
    tmem_ld16(col, r);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < 16; ++c) x[c] = __uint_as_float(r[c]);
  }
}

// NC / 2 packed columns of P
template <int N>
__device__ __forceinline__ void store_p(uint32_t col, const uint32_t (&pk)[N]) {
  if constexpr (N >= 32) {
#pragma unroll
    for (int i = 0; i < N / 32; ++i) {
      uint32_t t[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) t[c] = pk[i * 32 + c];
      tmem_st32(col + i * 32, t);
    }
  } else if constexpr (N == 16) {
    tmem_st16(col, pk);
  } else {
    tmem_st8(col, pk);
  }
}

// What a row keeps over an item.
struct RowState {
  float m, l;        // running max (log2 units; the one P is computed against) and sum
  int last_key;      // keys j <= last_key are allowed (-1: none)
  int pos;           // absolute position of the row's token
  float slope_log2;
};

// One tile's softmax for the NC columns from `c0` of a row: P over S in TMEM, returns the factor that O must
// be rescaled by (1: none).
template <typename T, int NC>
__device__ __forceinline__ float softmax_cols(const PagedParams& p, RowState& rs, uint32_t s_col, int j0, int c0) {
  float x[NC];
  load_cols<NC>(s_col + c0, x);
  const int mt = p.mask_type;
  const float scale = p.scale_log2;
  const bool raw_max = (mt == 0 || mt == 9) && scale > 0.f;  // max of the raw scores, scale folded into the exponent
  const int first = j0 + c0;
  const int lim = rs.last_key - first;  // columns c <= lim are allowed
  if (mt == 3 || mt == 5) {
    // right- and left-aligned bias differ by a per-row constant; both use (j - pos)
    const float b0 = rs.slope_log2 * static_cast<float>(first - rs.pos);
#pragma unroll
    for (int c = 0; c < NC; ++c) x[c] = fmaf(x[c], scale, fmaf(rs.slope_log2, static_cast<float>(c), b0));
  } else if (mt == 4) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      x[c] = fmaf(x[c], scale, -rs.slope_log2 * sqrtf(fmaxf(static_cast<float>(rs.pos - first - c), 0.f)));
  } else if (!raw_max) {
#pragma unroll
    for (int c = 0; c < NC; ++c) x[c] *= scale;
  }
  if (lim < NC - 1) {
#pragma unroll
    for (int c = 0; c < NC; ++c) x[c] = (c > lim) ? -INFINITY : x[c];
  }
  float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
  for (int c = 0; c < NC; c += 8) {
    mx0 = max3(mx0, x[c], x[c + 1]);
    mx1 = max3(mx1, x[c + 2], x[c + 3]);
    mx2 = max3(mx2, x[c + 4], x[c + 5]);
    mx3 = max3(mx3, x[c + 6], x[c + 7]);
  }
  float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
  if (raw_max) mx *= scale;
  const float m_new = fmaxf(rs.m, mx);
  float alpha = 1.f;
  if (m_new - rs.m > kRescaleThreshold) {  // false while both are -inf
    alpha = fast_exp2(rs.m - m_new);
    rs.m = m_new;
  }
  const float m_base = (rs.m == -INFINITY) ? 0.f : rs.m;
  const uint64_t scale2 = f2pack(raw_max ? scale : 1.f, raw_max ? scale : 1.f);
  const uint64_t negm2 = f2pack(-m_base, -m_base);
  uint64_t acc[4] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f), f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
  // P is rounded to the operand type of the tensor core; the sum takes the unrounded values, so a row's
  // rounding errors (at most half a step of each weight) average out instead of biasing the normalisation
  uint32_t pk[NC / 2];
#pragma unroll
  for (int c = 0; c < NC; c += 2) {
    float e0, e1;
    f2unpack(fma_x2(f2pack(x[c], x[c + 1]), scale2, negm2), e0, e1);
    e0 = fast_exp2(e0);
    e1 = fast_exp2(e1);
    acc[(c >> 1) & 3] = add_x2(acc[(c >> 1) & 3], f2pack(e0, e1));
    pk[c / 2] = pack2(e0, e1, (T*)nullptr);
  }
  store_p<NC / 2>(s_col + c0 / 2, pk);
  float s0, s1;
  f2unpack(add_x2(add_x2(acc[0], acc[1]), add_x2(acc[2], acc[3])), s0, s1);
  rs.l = rs.l * alpha + (s0 + s1);
  return alpha;
}

// O rows in TMEM times alpha.
template <int D>
__device__ __forceinline__ void scale_rows(uint32_t o_col, float alpha) {
#pragma unroll 1
  for (int c32 = 0; c32 < D / 32; ++c32) {
    uint32_t regs[32];
    tmem_ld32(o_col + c32 * 32, regs);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < 32; ++c) regs[c] = __float_as_uint(__uint_as_float(regs[c]) * alpha);
    tmem_st32(o_col + c32 * 32, regs);
  }
  tmem_st_wait();
}

// ---------------------------------------------------------------------------------------------- kernel

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const PagedParams p) {
  using C = Cfg<T, D>;
  constexpr int TK = C::TK, NSK = C::NSK, NSV = C::NSV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                     // [Q_BYTES]; between items the scratch of the join of lane quarters
  uint8_t* sK = sQ + C::Q_BYTES;          // [NSK][KV_BYTES]
  uint8_t* sV = sK + NSK * C::KV_BYTES;   // [NSV][KV_BYTES]
  float2* sML = reinterpret_cast<float2*>(sV + NSV * C::KV_BYTES);  // [4][32]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sML + 128);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;
  uint64_t* k_empty = k_full + NSK;
  uint64_t* v_full = k_empty + NSK;
  uint64_t* v_empty = v_full + NSV;
  uint64_t* s_full = v_empty + NSV;  // [2] per S buffer
  uint64_t* p_full = s_full + 2;     // [2]
  uint64_t* pv_done = p_full + 2;
  uint64_t* o_done = pv_done + 1;  // the item's last product
  uint64_t* join = o_done + 1;     // meetings of the softmax warps, with the limit of every other wait
  uint64_t* fin = join + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BARS);
  __shared__ Start st;
  __shared__ int64_t red[2 * kThreads / 32 + 2];

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  int* status = p.status;

  find_start<TK>(p, &st, red);
  if (threadIdx.x == 0) {
    mbar_init(q_full, 128);
    for (int s = 0; s < NSK; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(k_empty + s, 1);
    }
    for (int s = 0; s < NSV; ++s) {
      mbar_init(v_full + s, 1);
      mbar_init(v_empty + s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full + s, 1);
      mbar_init(p_full + s, 128);
    }
    mbar_init(pv_done, 1);
    mbar_init(o_done, 1);
    mbar_init(join, 128);
    mbar_init(fin, 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (st.b < 0) {  // fewer tiles than CTAs
    if (threadIdx.x == 0) p.desc[blockIdx.x].n_seg = 0;
    return;
  }
  if (warp == 6) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  Walker<TK> w;
  w.b = st.b;
  w.h = st.h;
  w.rt = st.rt;
  w.t0 = st.t0;
  w.raw = st.raw;
  w.cu = st.cu;
  w.left = st.left;
  w.s = load_seq(p, w.b, w.cu, w.raw);
  w.enter(p);

  // Barrier phases run on across items: the rings and the S buffers by counters of all tiles (slot g % depth,
  // phase g / depth), q_full by the item.
  if (warp == 4 || warp == 5) {
    // -------------------------------------------------------------- producers: warp 4 K, warp 5 V
    const bool is_k = warp == 4;
    const int depth = is_k ? NSK : NSV;
    uint8_t* ring = is_k ? sK : sV;
    uint64_t* full_bar = is_k ? k_full : v_full;
    uint64_t* empty_bar = is_k ? k_empty : v_empty;
    const CUtensorMap* map = is_k ? &tmK : &tmV;
    const bool leader = elect_one();
    if (leader) tma_prefetch_desc(map);
    const int bs = p.block_size, box = p.box_rows;
    const bool has_box = lane * box < TK;  // lane i loads box i of each tile
    const int oob_row = p.num_blocks * bs;
    bool ok = true;
    uint32_t g = 0;  // tiles loaded so far
    do {
      const int32_t* bt = p.block_tables + (size_t)w.b * p.max_blocks;
      const int pages = (w.s.kv + bs - 1) / bs;
      // the table entry of a tile's box is fetched one tile ahead, so its latency is not in the loop
      int pg = (w.t0 * TK + lane * box) / bs;
      int blk = has_box && pg < pages ? __ldg(bt + pg) : -1;
      for (int j = w.t0; j < w.t1; ++j, ++g) {
        const int slot = g % depth;
        const int pos = j * TK + lane * box;
        int row = oob_row;  // past the last page: the load fills zeros
        if (has_box && pg < pages) {
          if (blk >= 0 && blk < p.num_blocks) row = blk * bs + (pos - pg * bs);
          else atomicCAS(status + 1, 0, kDevBadBlockIndex);
        }
        if (j + 1 < w.t1) {
          pg = (pos + TK) / bs;
          blk = has_box && pg < pages ? __ldg(bt + pg) : -1;
        }
        if (g >= (uint32_t)depth &&
            !__all_sync(0xffffffffu, mbar_wait(empty_bar + slot, ((g / depth) - 1) & 1, status,
                                               is_k ? kDevTimeoutKEmpty : kDevTimeoutVEmpty))) {
          ok = false;
          break;
        }
        if (leader) mbar_expect_tx(full_bar + slot, C::KV_BYTES);
        __syncwarp();
        if (has_box) {
          uint8_t* dst = ring + slot * C::KV_BYTES + lane * box * 128;
#pragma unroll
          for (int cb = 0; cb < C::CB; ++cb) tma_load_3d(dst + cb * TK * 128, map, full_bar + slot, cb * 64, w.h, row);
        }
      }
    } while (ok && w.next(p));
    // never leave the CTA while loads this warp issued are still landing in shared memory
    for (uint32_t i = g >= (uint32_t)depth ? g - depth : 0; i < g; ++i)
      mbar_wait(full_bar + (i % depth), (i / depth) & 1, status, is_k ? kDevTimeoutKFull : kDevTimeoutVFull);
  } else if (warp == 6) {
    // -------------------------------------------------------------- MMA issuer
    const bool leader = elect_one();
    const uint64_t dq = smem_desc_sw128(smem_addr(sQ), 16, 1024);
    const uint64_t dk = smem_desc_sw128(smem_addr(sK), 16, 1024);
    const uint64_t dv = smem_desc_sw128(smem_addr(sV), TK * 128, 1024);  // MN-major
    constexpr uint64_t kStep = C::KV_BYTES >> 4;
    auto wait_all = [&](uint64_t* bar, uint32_t parity, int code) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, status, code));
    };
    auto commit = [&](uint64_t* bar) {
      if (leader) mma_commit(bar);
    };
    auto issue_qk = [&](uint32_t g) -> bool {
      const int slot = g % NSK;
      if (!wait_all(k_full + slot, (g / NSK) & 1, kDevTimeoutKFull)) return false;
      tc_fence_after();
      if (leader) {
        const uint64_t b0 = dk + slot * kStep;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int ke = kk * 16;
          const uint64_t in = (uint64_t)(ke % 64) * 2;
          mma_ss(tmem + (g & 1) * TK, dq + (((ke / 64) * (128 * 128) + in) >> 4), b0 + (((ke / 64) * (TK * 128) + in) >> 4),
                 C::IDESC_QK, kk > 0, false);
        }
      }
      commit(s_full + (g & 1));
      commit(k_empty + slot);
      return true;
    };
    bool ok = true;
    uint32_t g0 = 0, item = 0;
    do {
      const int cnt = w.t1 - w.t0;
      // Q is written after the previous item's last P V, so both S buffers and O are free from here on
      ok = wait_all(q_full, item & 1, kDevTimeoutQ) && issue_qk(g0) && (cnt < 2 || issue_qk(g0 + 1));
      for (int i = 0; i < cnt && ok; ++i) {
        const uint32_t g = g0 + i;
        const int slot = g % NSV;
        if (!wait_all(v_full + slot, (g / NSV) & 1, kDevTimeoutVFull) ||
            !wait_all(p_full + (g & 1), (g >> 1) & 1, kDevTimeoutPFull)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (leader) {
          const uint64_t v0 = dv + slot * kStep;
#pragma unroll
          for (int kk = 0; kk < TK / 16; ++kk)
            mma_ts(tmem + C::O_COL, tmem + (g & 1) * TK + kk * 8, v0 + ((kk * 16 * 128) >> 4), C::IDESC_PV,
                   (i > 0 || kk > 0) ? 1u : 0u, false);
        }
        commit(v_empty + slot);
        commit(pv_done);
        if (i == cnt - 1) commit(o_done);
        if (i + 2 < cnt) ok = wait_all(pv_done, g & 1, kDevTimeoutODone) && issue_qk(g + 2);
      }
      g0 += cnt;
      ++item;
    } while (ok && w.next(p));
    // all tensor-core work this thread issued has finished before TMEM is released
    commit(fin);
    wait_all(fin, 0, kDevTimeoutFinal);
  } else if (warp < 4) {
    // -------------------------------------------------------------- softmax and epilogue
    const int r = threadIdx.x;  // TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t o_col = tmem + lane_base + C::O_COL;
    const int group = p.group;
    uint32_t g = 0, item = 0, meetings = 0;
    bool ok = true, owner = false;
    int64_t line = st.line;
    auto meet = [&]() {
      mbar_arrive(join);
      ok = ok && __all_sync(0xffffffffu, mbar_wait(join, meetings & 1, status, kDevTimeoutODone));
      ++meetings;
    };
    do {
      const int rows = w.rows(p);
      const bool quarters = rows <= 32;       // rows repeated in each lane quarter, which shares the keys
      const int rr = quarters ? lane : r;     // this thread's row of the tile
      const bool valid = rr < rows;
      const int tok = w.rt * p.tb + rr / group, head = w.h * group + rr % group;
      const int64_t token = w.cu + tok;
      const int off = w.s.kv - w.s.seq;
      RowState rs;
      rs.m = -INFINITY;
      rs.l = 0.f;
      rs.pos = tok + off;
      rs.last_key = !valid ? -1 : p.mask_type == 0 ? w.s.kv - 1 : min(rs.pos, w.s.kv - 1);
      rs.slope_log2 = (valid && p.slopes) ? p.slopes[head] * kLog2e : 0.f;
      // ---- Q row to shared memory, K-major with the 128-byte swizzle
      if (valid) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + token * p.q_stride + (int64_t)head * p.dq);
        const int lo = p.dq < p.row ? (head & 1) * (p.dq / 8) : 0, hi = lo + p.dq / 8;  // map 2 in the upper half
        const uint32_t dst = smem_addr(sQ) + r * 128;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (c >= lo && c < hi) v = __ldg(src + (c - lo));
          st_shared_v4(dst + (c >> 3) * (128 * 128) + (((c & 7) ^ (r & 7)) << 4), v);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();  // the previous item's loads of O come before the product that overwrites it
      mbar_arrive(q_full);
      // ---- key tiles
      const int cnt = w.t1 - w.t0;
      const bool warp_rows = quarters || warp * 32 < rows;
      for (int i = 0; i < cnt; ++i, ++g) {
        const int j0 = (w.t0 + i) * TK;
        const uint32_t s_col = tmem + lane_base + (g & 1) * TK;
        ok = __all_sync(0xffffffffu, mbar_wait(s_full + (g & 1), (g >> 1) & 1, status, kDevTimeoutSFull));
        if (!ok) break;
        tc_fence_after();
        float alpha = 1.f;
        if (quarters) {
          constexpr int NC = TK / 4;
          alpha = softmax_cols<T, NC>(p, rs, s_col, j0, warp * NC);
          const uint32_t zero[NC / 2] = {};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q != warp) store_p<NC / 2>(s_col + q * (NC / 2), zero);
        } else if (warp_rows) {  // the other warps' rows of P and O are read by nobody
          alpha = softmax_cols<T, TK>(p, rs, s_col, j0, 0);
        }
        if (j0 + TK > w.s.kv) {
          // slots past kvSeqLen may hold anything, NaN included, and 0 * NaN is not 0: clear their V rows
          const int slot = g % NSV;
          ok = __all_sync(0xffffffffu, mbar_wait(v_full + slot, (g / NSV) & 1, status, kDevTimeoutVFull));
          if (!ok) break;
          if (r < TK && j0 + r >= w.s.kv) {
            const uint32_t dst = smem_addr(sV + slot * C::KV_BYTES) + r * 128;
#pragma unroll
            for (int cb = 0; cb < C::CB; ++cb)
#pragma unroll
              for (int c = 0; c < 8; ++c) st_shared_v4(dst + cb * TK * 128 + c * 16, make_uint4(0, 0, 0, 0));
          }
          fence_proxy_async_smem();
        }
        if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          ok = __all_sync(0xffffffffu, mbar_wait(pv_done, (g - 1) & 1, status, kDevTimeoutODone));
          if (!ok) break;
          tc_fence_after();
          scale_rows<D>(o_col, alpha);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full + (g & 1));
      }
      if (!ok) break;
      // o_done has one phase per item and is waited for once in each, so no wait can meet the phase before or
      // after its own (pv_done may be two phases on, or one short, when a warp gets here)
      ok = __all_sync(0xffffffffu, mbar_wait(o_done, item & 1, status, kDevTimeoutODone));
      ++item;
      if (!ok) break;
      tc_fence_after();
      // ---- join the four lane quarters into the first: O' = sum_w 2^(m_w - M) O_w, l alike
      if (quarters) {
        sML[warp * 32 + lane] = make_float2(rs.m, rs.l);
        meet();
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) top = fmaxf(top, sML[q * 32 + lane].x);
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int q = 0; q < 4; ++q) sum += sML[q * 32 + lane].y * fast_exp2(sML[q * 32 + lane].x - base);
        const float f = fast_exp2(rs.m - base);
        rs.m = top;
        rs.l = sum;
        // half of the columns at a time: 3 quarters x 32 rows x D / 2 floats fit the Q buffer
        float4* scratch = reinterpret_cast<float4*>(sQ);
        constexpr int F4 = D / 8;  // float4 chunks of half a row
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll 1
          for (int c32 = 0; c32 < D / 64; ++c32) {
            if (warp > 0) {
              uint32_t regs[32];
              tmem_ld32(o_col + half * (D / 2) + c32 * 32, regs);
              tmem_ld_wait();
              if (valid) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  const float4 v = make_float4(__uint_as_float(regs[4 * c]) * f, __uint_as_float(regs[4 * c + 1]) * f,
                                               __uint_as_float(regs[4 * c + 2]) * f, __uint_as_float(regs[4 * c + 3]) * f);
                  scratch[((warp - 1) * 32 + lane) * F4 + ((c32 * 8 + c) ^ (lane & 7))] = v;
                }
              }
            }
          }
          meet();
          if (warp == 0) {
#pragma unroll 1
            for (int c32 = 0; c32 < D / 64; ++c32) {
              uint32_t regs[32];
              tmem_ld32(o_col + half * (D / 2) + c32 * 32, regs);
              tmem_ld_wait();
              if (valid) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  float4 a = make_float4(__uint_as_float(regs[4 * c]) * f, __uint_as_float(regs[4 * c + 1]) * f,
                                         __uint_as_float(regs[4 * c + 2]) * f, __uint_as_float(regs[4 * c + 3]) * f);
#pragma unroll
                  for (int q = 0; q < 3; ++q) {
                    const float4 b = scratch[(q * 32 + lane) * F4 + ((c32 * 8 + c) ^ (lane & 7))];
                    a.x += b.x;
                    a.y += b.y;
                    a.z += b.z;
                    a.w += b.w;
                  }
                  regs[4 * c] = __float_as_uint(a.x);
                  regs[4 * c + 1] = __float_as_uint(a.y);
                  regs[4 * c + 2] = __float_as_uint(a.z);
                  regs[4 * c + 3] = __float_as_uint(a.w);
                }
              }
              __syncwarp();
              tmem_st32(o_col + half * (D / 2) + c32 * 32, regs);
            }
            tmem_st_wait();
          }
          meet();
        }
      }
      if (!ok) break;
      // ---- epilogue
      const bool whole = w.t0 == 0 && w.t1 == w.n;
      const bool has_rows = warp_rows && (!quarters || warp == 0);
      if (!whole) {
        // a cut item: unnormalised O, max and sum; slot 1 when the item starts here, 0 when it began earlier
        const int64_t prow = ((int64_t)blockIdx.x * 2 + (w.t0 == 0 ? 1 : 0)) * 128 + rr;
        if (has_rows) {
          if (valid) p.ml[prow] = make_float2(rs.m, rs.l);
          float* dst = p.part + prow * D;
#pragma unroll 1
          for (int c32 = 0; c32 < D / 32; ++c32) {
            if (c32 * 32 >= p.row) break;
            uint32_t regs[32];
            tmem_ld32(o_col + c32 * 32, regs);
            tmem_ld_wait();
            if (valid) {
#pragma unroll
              for (int i = 0; i < 4; ++i) st_global_v8(dst + c32 * 32 + i * 8, regs + i * 8);
            }
          }
        }
        if (w.t0 == 0 && threadIdx.x == 0) {
          // the last CTA c with c * total / ctas <= last tile
          const int64_t last = line + w.n - 1;
          PagedDesc d;
          d.n_seg = (int)(((last + 1) * st.ctas - 1) / st.total) - (int)blockIdx.x + 1;
          d.token0 = (int)(w.cu + w.rt * p.tb);
          d.rows = rows;
          d.kv_head = w.h;
          d.pos0 = w.rt * p.tb + off;
          p.desc[blockIdx.x] = d;
          owner = true;
        }
      } else if (has_rows) {
        const float inv_l = rs.l > 0.f ? 1.f / rs.l : 0.f;  // a row without keys gets 0
        if (p.dq == p.row) {
          T* orow = static_cast<T*>(p.out) + (token * p.heads + head) * p.row;
          const bool wide = p.row % 16 == 0;
#pragma unroll 1
          for (int c32 = 0; c32 < D / 32; ++c32) {
            if (c32 * 32 >= p.row) break;
            uint32_t regs[32], o[16];
            tmem_ld32(o_col + c32 * 32, regs);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = pack2(__uint_as_float(regs[2 * i]) * inv_l, __uint_as_float(regs[2 * i + 1]) * inv_l, (T*)nullptr);
            if (valid) {
              if (wide) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (c32 * 32 + i * 16 < p.row) st_global_v8(orow + c32 * 32 + i * 16, o + i * 8);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (c32 * 32 + i * 8 < p.row) st_global_v4(orow + c32 * 32 + i * 8, o + i * 4);
              }
            }
          }
          if (valid && p.lse) {
            float lse = rs.l > 0.f ? rs.m * kLn2 + logf(rs.l) : -INFINITY;
            if (p.mask_type == 5) lse += p.slopes[head] * static_cast<float>(rs.pos);  // left-aligned = right-aligned + slope * pos
            p.lse[token * p.heads + head] = lse;
          }
        } else {
          // even lanes hold map 1, odd lanes map 2 of the same head: even lanes finish the first 16 columns of
          // each 32, odd lanes the others
          const bool odd = lane & 1;
          const int oh = head >> 1;
          const float f = odd ? (valid ? -p.lambda[oh] * inv_l : 0.f) : inv_l;
          float y[16];
          auto diff = [&](int c32) {
            uint32_t regs[32];
            tmem_ld32(o_col + c32 * 32, regs);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float a = __uint_as_float(regs[i]) * f, b = __uint_as_float(regs[16 + i]) * f;
              y[i] = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
            }
          };
          float post = p.out_scale;
          if (p.norm_weight) {
            float ss = 0.f;
#pragma unroll 1
            for (int c32 = 0; c32 < D / 32; ++c32) {
              diff(c32);
#pragma unroll
              for (int i = 0; i < 16; ++i) ss = fmaf(y[i], y[i], ss);
            }
            ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            post *= rsqrtf(ss / static_cast<float>(p.row) + p.norm_eps);
          }
          T* orow = static_cast<T*>(p.out) + (token * (p.heads / 2) + oh) * p.row;
#pragma unroll 1
          for (int c32 = 0; c32 < D / 32; ++c32) {
            const int col = c32 * 32 + (odd ? 16 : 0);
            diff(c32);
            if (valid && col < p.row) {
              uint32_t o[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float a = y[2 * i] * post, b = y[2 * i + 1] * post;
                if (p.norm_weight) {
                  a *= __ldg(p.norm_weight + col + 2 * i);
                  b *= __ldg(p.norm_weight + col + 2 * i + 1);
                }
                o[i] = pack2(a, b, (T*)nullptr);
              }
              st_global_v8(orow + col, o);
            }
          }
        }
      }
      line += cnt;
    } while (w.next(p));
    if (threadIdx.x == 0 && !owner) p.desc[blockIdx.x].n_seg = 0;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 6) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------------------------- combine

template <int N>
__device__ __forceinline__ void load_f(const float* src, float (&v)[N]) {
  if constexpr (N == 2) {
    const float2 a = *reinterpret_cast<const float2*>(src);
    v[0] = a.x;
    v[1] = a.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 a = reinterpret_cast<const float4*>(src)[i];
      v[4 * i] = a.x;
      v[4 * i + 1] = a.y;
      v[4 * i + 2] = a.z;
      v[4 * i + 3] = a.w;
    }
  }
}

// Joins the segments of the items that CTA boundaries cut, one warp per output row (both maps of a
// differential row), in segment order: m = max_s m_s, O = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PagedDesc d = p.desc[blockIdx.x];
  if (d.n_seg == 0) return;
  constexpr int N = D / 32;                   // columns per lane
  constexpr int NW = (kGrid + 31) / 32;       // segment weights per lane
  const int lane = threadIdx.x & 31;
  const int maps = p.dq == p.row ? 1 : 2;
  const int col = lane * N;
  for (int u = blockIdx.y * 8 + (threadIdx.x >> 5); u * maps < d.rows; u += kCombineY * 8) {
    float y[N];
    float lse = 0.f;
    const int r0 = u * maps;
    const int token = d.token0 + r0 / p.group, head = d.kv_head * p.group + r0 % p.group;
    for (int map = 0; map < maps; ++map) {
      const int r = r0 + map;
      // segment s lies in CTA blockIdx.x + s: in its slot 1 where the item starts, in slot 0 after that
      auto prow = [&](int s) { return ((int64_t)(blockIdx.x + s) * 2 + (s == 0 ? 1 : 0)) * 128 + r; };
      float wt[NW], top = -INFINITY, sum = 0.f;
      float2 ml[NW];
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const int s = k * 32 + lane;
        ml[k] = s < d.n_seg ? p.ml[prow(s)] : make_float2(-INFINITY, 0.f);
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
#pragma unroll 4
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
      if (p.mask_type == 5) lse += p.slopes[head] * static_cast<float>(d.pos0 + r0 / p.group);
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
}

template <typename T, int D>
cudaError_t launch(const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedParams& p, cudaStream_t stream) {
  using C = Cfg<T, D>;
  // at least 120 KB so a second CTA never shares the SM (each CTA allocates all 512 TMEM columns)
  constexpr int kSmem = C::SMEM > 120 * 1024 ? C::SMEM : 120 * 1024;
  cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  paged_attn_kernel<T, D><<<kGrid, kThreads, kSmem, stream>>>(tmK, tmV, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // a programmatic dependent launch: the combine grid is scheduled during the attention kernel's tail, and
  // griddepcontrol.wait holds it until that kernel has completed
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kGrid, kCombineY);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel<T, D>, p);
}

uint64_t align256(uint64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

int paged_kernel_d(int64_t row) {
  if (row <= 0 || row % 8 != 0 || row > 256) return 0;
  return row <= 64 ? 64 : row <= 128 ? 128 : 256;
}

void paged_layout(PagedPlan* plan) {
  const int D = paged_kernel_d(plan->row);
  plan->off_desc = kPagedStatusBytes;
  plan->off_ml = align256(plan->off_desc + sizeof(PagedDesc) * kGrid);
  plan->off_part = align256(plan->off_ml + sizeof(float2) * kGrid * 2 * 128);
  plan->ws_size = plan->off_part + (uint64_t)sizeof(float) * kGrid * 2 * 128 * D;
}

int paged_run(PagedPlan* plan, void* workspace, cudaStream_t stream, char* err, size_t errlen) {
  if (plan->n_tokens == 0 || plan->batch == 0) return ALA_OK;  // no rows to write
  const int D = paged_kernel_d(plan->row);
  const int box = kv_box_rows(plan->block_size, D == 256 ? 64 : 128);
  if (!plan->maps_ready) {
    const int64_t rows = (int64_t)plan->num_blocks * plan->block_size;
    if (!encode_rows_heads_d(&plan->tmK, plan->k, plan->dtype, rows, plan->kv_heads, plan->row, box, false) ||
        !encode_rows_heads_d(&plan->tmV, plan->v, plan->dtype, rows, plan->kv_heads, plan->row, box, true)) {
      snprintf(err, errlen, "cuTensorMapEncodeTiled failed");
      return ALA_CUDA_ERROR;
    }
    plan->maps_ready = true;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaError_t e = cudaSuccess;
  if (workspace != plan->bound_ws) e = cudaMemsetAsync(workspace, 0, kPagedStatusBytes, stream);
  if (e == cudaSuccess) {
    PagedParams p{};
    p.seq_len = plan->seq_len;
    p.kv_seq_len = plan->kv_seq_len;
    p.block_tables = plan->block_tables;
    p.slopes = plan->slopes;
    p.lambda = plan->lambda;
    p.norm_weight = plan->norm_weight;
    p.q = plan->q;
    p.out = plan->out;
    p.lse = plan->lse;
    p.status = reinterpret_cast<int*>(ws);
    p.desc = reinterpret_cast<PagedDesc*>(ws + plan->off_desc);
    p.ml = reinterpret_cast<float2*>(ws + plan->off_ml);
    p.part = reinterpret_cast<float*>(ws + plan->off_part);
    p.q_stride = plan->q_stride;
    p.n_tokens = (int32_t)plan->n_tokens;
    p.batch = plan->batch;
    p.max_blocks = plan->max_blocks;
    p.block_size = plan->block_size;
    p.num_blocks = plan->num_blocks;
    p.mask_type = plan->mask_type;
    p.heads = plan->heads;
    p.kv_heads = plan->kv_heads;
    p.group = plan->heads / plan->kv_heads;
    p.tb = 128 / p.group;
    p.dq = plan->d;
    p.row = plan->row;
    p.box_rows = box;
    p.scale_log2 = plan->qk_scale * kLog2e;
    p.norm_eps = plan->norm_eps;
    p.out_scale = plan->out_scale;
    const bool f16 = plan->dtype == ALA_F16;
    if (D == 64)
      e = f16 ? launch<__half, 64>(plan->tmK, plan->tmV, p, stream) : launch<__nv_bfloat16, 64>(plan->tmK, plan->tmV, p, stream);
    else if (D == 128)
      e = f16 ? launch<__half, 128>(plan->tmK, plan->tmV, p, stream) : launch<__nv_bfloat16, 128>(plan->tmK, plan->tmV, p, stream);
    else
      e = f16 ? launch<__half, 256>(plan->tmK, plan->tmV, p, stream) : launch<__nv_bfloat16, 256>(plan->tmK, plan->tmV, p, stream);
  }
  if (e != cudaSuccess) {
    snprintf(err, errlen, "kernel launch failed: %s", cudaGetErrorString(e));
    return ALA_CUDA_ERROR;
  }
  return ALA_OK;
}

}  // namespace ala
