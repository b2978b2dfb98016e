// paged_few.cu -- paged attention where a kv head has few query rows: one token, or a few, of each sequence.
//
// With R rows (8, 16 or 32 that hold the item's) the products are taken transposed, so that the keys, of which
// there are many, fill the 128 lanes of the tensor core, and the rows are its N:
//   S^T [128 keys x R]  = K_tile [128 x d] Q^T
//   O^T [d x N]        += V_tile^T [d x 128 keys] P^T
// A thread owns a key and half of the rows: it takes R / 2 scores, and its part of their sums stays in registers
// until the item ends, so a tile needs no reduction at all.  The running maxima are common to all threads and only
// move when some score is more than 2^8 above its row's (one vote of the threads a tile; under ALiBi too, since
// tiles run from the last key to the first, the largest scores first).  P goes to shared memory as the products'
// second operand.
// With R <= 16, and in the difference of two maps, the N columns are 2 R: the second R carry what rounding P to 16
// bits dropped, which makes P V exact to 2^-17 or so at no cost (N is at least 16, and the products are a tenth of
// the time).
//
// It is bound by the cache's bytes: some 500 cycles of tensor work and 1000 to 1700 of softmax a tile of 128 keys,
// against 2700 (d = 128) that the tile takes to arrive at a CTA's share of HBM.  What is left for speed is to keep
// loads in flight, so the rest of shared memory is one ring of K and V tiles in the order of their use (192 KB: 4.2 us
// of HBM at a CTA's share), which also covers the change from one item to the next.  With pages of 16 rows, or row
// tiles of 32 under ALiBi, issuing the boxes and the softmax take 1800 to 2000 cycles a tile.
// Measured: 124 tokens over 8300 keys on average, 32 / 8 heads, d 128: 611 to 623 us, 6.8 to 6.9 TB/s (a copy: 6.5 TB/s);
// one token over 213 keys: 9 us, the chain of its latencies.  5 tokens of 32 requests over 4700 keys, 40 / 8 heads, d 80,
// pages of 16, ALiBi: 106 us (the bytes 59); with pages of 128 94, without ALiBi too 90; one token each 86, and 76 with
// pages of 128 and no ALiBi.
//
// The line of tiles, its split over the CTAs and the partials of cut items are those of paged_attn.cu.
//   warps 0..7  softmax (threads r and r + 128: key r of the tile, TMEM lane r, the first and the second half of
//               the rows) and epilogue (column r of O)
//   warps 8, 9  TMA producers of K and of V;  warp 10  tcgen05 issuer
#include "paged_common.cuh"

namespace ala {

namespace {

template <typename T, int D_>
struct Few {
  static constexpr int D = D_, TK = 128, CB = D / 64;
  static constexpr int KV_BYTES = TK * D * 2;
  static constexpr int NS = 192 * 1024 / KV_BYTES;  // ring slots
  // 128-row tiles of O^T.  With D = 64 the lanes from 64 on multiply what lies behind a V tile, in shared memory still,
  // and are read by nobody.
  static constexpr int MT = D == 256 ? 2 : 1;
  static constexpr int QCB = kFewRows * 128;        // bytes of a 64-column block of Q
  static constexpr int Q_BYTES = CB * QCB;
  static constexpr int P_BYTES = 2 * QCB;           // [2 blocks of 64 keys][32 rows][128 B]
  static constexpr int N_BARS = 1 + 2 * NS + 6 + 2;
  static constexpr int THREADS = 352;
  static constexpr int SMEM = 1024 + NS * KV_BYTES + Q_BYTES + 2 * P_BYTES + N_BARS * 8 + 16;
  static constexpr uint32_t O_COL = 64, TMEM_COLS = 256;  // S^T [0, 32) and [32, 64), O^T from 64, 64 columns a tile
  static_assert(D != 64 || Q_BYTES + 2 * P_BYTES >= KV_BYTES, "behind the last V tile");
};

// What the threads share about an item's rows, and the scratch of their reductions.
struct RowTables {
  float4 bias[kFewRows / 2];   // of rows 2i and 2i + 1: slopes of their heads (log2 units), minus their tokens' places in the tile
  int pos[kFewRows];           // position of the row's token
  int last_key[kFewRows];      // keys up to this one are allowed (-1: none)
  float m[kFewRows];
  float red[4][kFewRows];      // per lane quarter
  Start start;                 // where this CTA starts, and the scratch of finding it
  int64_t scan[2 * 12];
  PagedDesc join[2];           // n_seg != 0: this CTA's segment was the last of a cut item to arrive (a CTA has two at most)
  int first[2];                // the CTA where that starts
};

__device__ __forceinline__ bool any_of_256(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 2, 256, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// N columns of 32-bit values from TMEM column `col` on (no wait)
template <int N>
__device__ __forceinline__ void ld_cols(uint32_t col, uint32_t (&r)[N]) {
  if constexpr (N == 4) tmem_ld4(col, r);
  else if constexpr (N == 8) tmem_ld8(col, r);
  else tmem_ld16(col, r);
}
template <int N>
__device__ __forceinline__ void st_cols(uint32_t col, const uint32_t (&r)[N]) {
  if constexpr (N == 4) tmem_st4(col, r);
  else if constexpr (N == 8) tmem_st8(col, r);
  else tmem_st16(col, r);
}

__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"((uint16_t)v) : "memory");
}

// Where the softmax warps are.
struct FewState {
  uint32_t g;     // steps so far (buffer g & 1, phase g / 2)
  uint32_t item;  // items so far
  bool ok;
};

// One item: its key tiles and its epilogue, R rows, RT of them this thread's.  After a failed wait a warp skips the waits that are left, but
// goes through every tile and item, so that the warps meet as often as ever.
template <typename T, int D, int R, int MAPS>
__device__ __forceinline__ void few_item(const PagedParams& p, const Walker<128>& w, FewState& f, RowTables& tab, uint8_t* sVring,
                                         uint32_t v_slot0, uint64_t* v_full0, uint32_t v_phase0, uint32_t sP, uint64_t* s_full,
                                         uint64_t* p_full, uint64_t* pv_done, uint64_t* o_done, uint32_t tmem, int64_t token0,
                                         int tokens) {
  using C = Few<T, D>;
  constexpr bool kCarry = R <= 16 || MAPS == 2;
  // 32 rows and what their rounding drops: P takes both buffers, [2 blocks of 64 keys][64 rows][128 B]
  constexpr bool kOneP = R == 32 && kCarry;
  constexpr int PCB = kOneP ? 2 * C::QCB : C::QCB;
  constexpr int RT = R / 2;
  const int r = threadIdx.x & 127, quarter = r >> 5, lane = r & 31;
  const int n0 = (threadIdx.x >> 7) * RT;  // this thread's rows: n0 .. n0 + RT - 1
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
  const int group = p.group, rows = tokens * group, mt = p.mask_type;
  const bool alibi = mt == 3 || mt == 4 || mt == 5;
  const float scale = p.scale_log2;
  int* status = p.status;
  const int first_last = tab.last_key[0];  // the earliest token sees fewest keys
  const int pos0 = tab.pos[0];
  // Maxima in log2 units (the ones P is computed against) and sums.  A row that has met no key has a maximum below
  // any score, and finite, so that it needs no case of its own.
  float m[RT], l[RT];
#pragma unroll
  for (int n = 0; n < RT; ++n) {
    m[n] = kNoKey;
    l[n] = 0.f;
  }
  // this key's place in a row of P: [block of 64 keys][row][128 B], 16-byte chunks swizzled by the row
  const uint32_t pk0 = (r >> 6) * PCB + (r & 7) * 2, pchunk = (r & 63) >> 3;
  const int cnt = w.t1 - w.t0;
  for (int u = 0; u < cnt; ++u, ++f.g) {
    const int j0 = (w.t1 - 1 - u) * 128, key = j0 + r;
    const int b = f.g & 1;
    if (f.ok) f.ok = __all_sync(0xffffffffu, mbar_wait(s_full + b, (f.g >> 1) & 1, status, kDevTimeoutSFull));
    tc_fence_after();
    uint32_t raw[RT];
    ld_cols<RT>(tmem + lanes + b * 32 + n0, raw);
    tmem_ld_wait();
    float t[RT];
#pragma unroll
    for (int n = 0; n < RT; ++n) t[n] = __uint_as_float(raw[n]) * scale;
    if (alibi) {
      // right- and left-aligned bias differ by a per-row constant; both use (key - pos), which is exact below 2^24 as a
      // difference of 32-bit floats too: one conversion a thread, pairs of rows in one instruction
      const float ahead0 = static_cast<float>(key - pos0);
#pragma unroll
      for (int n = 0; n < RT; n += 2) {
        const float4 sb = tab.bias[(n0 + n) / 2];
        const uint64_t ahead = add_x2(f2pack(ahead0, ahead0), f2pack(sb.z, sb.w));
        if (mt == 4) {
          float a0, a1;
          f2unpack(ahead, a0, a1);
          t[n] = fmaf(-sb.x, sqrt_approx(fmaxf(-a0, 0.f)), t[n]);
          t[n + 1] = fmaf(-sb.y, sqrt_approx(fmaxf(-a1, 0.f)), t[n + 1]);
        } else {
          f2unpack(fma_x2(f2pack(sb.x, sb.y), ahead, f2pack(t[n], t[n + 1])), t[n], t[n + 1]);
        }
      }
    }
    if (j0 + 127 > first_last) {
#pragma unroll
      for (int n = 0; n < RT; ++n) t[n] = key > tab.last_key[n0 + n] ? -INFINITY : t[n];
    }
    float over = -INFINITY;
#pragma unroll
    for (int n = 0; n < RT; n += 2) over = max3(over, t[n] - m[n], t[n + 1] - m[n + 1]);
    if (any_of_256(over > kRescaleThreshold)) {
      // some row's maximum moves: every row takes its tile's
#pragma unroll
      for (int n = 0; n < RT; ++n) {
        float v = t[n];
#pragma unroll
        for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (lane == 0) tab.red[quarter][n0 + n] = v;
      }
      named_barrier_sync(1, 256);
      float alpha[RT];
#pragma unroll
      for (int n = 0; n < RT; ++n) {
        const float top = fmaxf(fmaxf(tab.red[0][n0 + n], tab.red[1][n0 + n]), fmaxf(tab.red[2][n0 + n], tab.red[3][n0 + n]));
        const float m_new = fmaxf(m[n], top);
        alpha[n] = fast_exp2(m[n] - m_new);
        m[n] = m_new;
        l[n] *= alpha[n];
      }
      if (u > 0) {
        if (f.ok)
          f.ok = __all_sync(0xffffffffu, mbar_wait(pv_done + (b ^ 1), ((f.g - 1) >> 1) & 1, status, kDevTimeoutODone));
        tc_fence_after();
#pragma unroll
        for (int mi = 0; mi < C::MT; ++mi)
#pragma unroll
          for (int part = 0; part < (kCarry ? 2 : 1); ++part) {
            const uint32_t col = tmem + lanes + C::O_COL + mi * 64 + part * R + n0;
            uint32_t o[RT];
            ld_cols<RT>(col, o);
            tmem_ld_wait();
#pragma unroll
            for (int n = 0; n < RT; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * alpha[n]);
            st_cols<RT>(col, o);
          }
        tmem_st_wait();
      }
    }
    // P: rounded to the operands' 16 bits; the sums take the unrounded values, so a row's rounding errors average
    // out instead of biasing its normalisation
    uint32_t hi[RT / 2], lo[RT / 2];
#pragma unroll
    for (int n = 0; n < RT; n += 2) {
      const float e0 = fast_exp2(t[n] - m[n]), e1 = fast_exp2(t[n + 1] - m[n + 1]);
      l[n] += e0;
      l[n + 1] += e1;
      hi[n / 2] = pack2(e0, e1, (T*)nullptr);
      if constexpr (kCarry) {
        const float2 h = unpack2(hi[n / 2], (T*)nullptr);
        lo[n / 2] = pack2(e0 - h.x, e1 - h.y, (T*)nullptr);
      }
    }
    // The buffer's previous P has been multiplied: two tiles back that product was issued before this tile's scores,
    // and a commit waits for all products before it.
    if (kOneP && u > 0 && f.ok)
      f.ok = __all_sync(0xffffffffu, mbar_wait(pv_done + (b ^ 1), ((f.g - 1) >> 1) & 1, status, kDevTimeoutODone));
    const uint32_t prow = sP + (kOneP ? 0 : b * C::P_BYTES) + pk0 + n0 * 128;
#pragma unroll
    for (int n = 0; n < RT; ++n) {
      const uint32_t at = prow + n * 128 + ((pchunk ^ ((n0 + n) & 7)) << 4);
      st_shared_u16(at, (n & 1) ? hi[n / 2] >> 16 : hi[n / 2]);
      if constexpr (kCarry) st_shared_u16(at + R * 128, (n & 1) ? lo[n / 2] >> 16 : lo[n / 2]);  // R is a multiple of 8
    }
    if (u == 0 && j0 + 128 > w.s.kv) {
      // slots past kvSeqLen may hold anything, NaN included, and 0 * NaN is not 0: clear their V rows
      if (f.ok) f.ok = __all_sync(0xffffffffu, mbar_wait(v_full0, v_phase0, status, kDevTimeoutVFull));
      if (threadIdx.x < 128 && key >= w.s.kv && f.ok) {
        const uint32_t dst = smem_addr(sVring + v_slot0 * C::KV_BYTES) + r * 128;
#pragma unroll
        for (int cb = 0; cb < C::CB; ++cb)
#pragma unroll
          for (int c = 0; c < 8; ++c) st_shared_v4(dst + cb * (128 * 128) + c * 16, make_uint4(0, 0, 0, 0));
      }
      __syncwarp();
    }
    fence_proxy_async_smem();
    tc_fence_before();
    mbar_arrive(p_full + b);
  }
  // ---- the sums of all keys, and O
#pragma unroll
  for (int n = 0; n < RT; ++n) {
#pragma unroll
    for (int o = 16; o; o >>= 1) l[n] += __shfl_xor_sync(0xffffffffu, l[n], o);
  }
  if (f.ok) f.ok = __all_sync(0xffffffffu, mbar_wait(o_done, f.item & 1, status, kDevTimeoutODone));
  ++f.item;
  tc_fence_after();
  // every thread has left the last tile, so what it shared there has been read
#pragma unroll
  for (int n = 0; n < RT; ++n) {
    if (lane == 0) tab.red[quarter][n0 + n] = l[n];
    if (r == 0) tab.m[n0 + n] = m[n];
  }
  named_barrier_sync(1, 256);
  const bool whole = w.t0 == 0 && w.t1 == w.n;
  const int64_t prow0 = ((int64_t)blockIdx.x * 2 + (w.t0 == 0 ? 1 : 0)) * (D == 256 ? 128 : 256);
  auto total = [&](int n) { return (tab.red[0][n] + tab.red[1][n]) + (tab.red[2][n] + tab.red[3][n]); };
  if (threadIdx.x < rows && f.ok) {  // thread n: row n's statistics
    const int n = threadIdx.x;
    const float sum = total(n), top = tab.m[n];
    if (!whole) {
      p.ml[prow0 + n] = make_float2(top, sum);
    } else if (p.lse) {
      const int h = w.h * group + n % group;
      float lse = sum != 0.f ? top * kLn2 + logf(sum) : -INFINITY;
      if (mt == 5) lse += p.slopes[h] * static_cast<float>(tab.pos[n]);  // left-aligned = right-aligned + slope * position
      p.lse[(token0 + n / group) * p.heads + h] = lse;
    }
  }
  float o[C::MT][RT];  // column r (+ 128) of this thread's rows
#pragma unroll
  for (int mi = 0; mi < C::MT; ++mi) {
    uint32_t raw[RT], rest[RT];
    const uint32_t col = tmem + lanes + C::O_COL + mi * 64 + n0;
    ld_cols<RT>(col, raw);
    if constexpr (kCarry) ld_cols<RT>(col + R, rest);
    tmem_ld_wait();
#pragma unroll
    for (int n = 0; n < RT; ++n) {
      o[mi][n] = __uint_as_float(raw[n]);
      if constexpr (kCarry) o[mi][n] += __uint_as_float(rest[n]);
    }
  }
  if (!whole) {
#pragma unroll
    for (int mi = 0; mi < C::MT; ++mi) {
      const int col = mi * 128 + r;
      if (col >= p.row || !f.ok) continue;
      float* dst = p.part + (prow0 + n0) * D + col;
#pragma unroll
      for (int n = 0; n < RT; ++n)
        if (n0 + n < rows) dst[(int64_t)n * D] = o[mi][n];
    }
  } else if constexpr (MAPS == 1) {
    // the rows of one token follow each other; the next token's lie p.heads rows on
    int hh = n0 % group;
    T* dst = static_cast<T*>(p.out) + ((token0 + n0 / group) * p.heads + w.h * group + hh) * p.row + r;
#pragma unroll
    for (int n = 0; n < RT; ++n) {
      if (n0 + n < rows) {
        const float sum = total(n0 + n), inv = sum > 0.f ? 1.f / sum : 0.f;  // a row without keys gets 0
#pragma unroll
        for (int mi = 0; mi < C::MT; ++mi)
          if (mi * 128 + r < p.row && f.ok) dst[mi * 128] = from_float<T>(o[mi][n] * inv);
        dst += p.row;
        if (++hh == group) {
          hh = 0;
          dst += (int64_t)(p.heads - group) * p.row;
        }
      }
    }
  } else {
    // rows 2i and 2i + 1 are the two maps of a head
    const int gh = group / 2, i0 = n0 / 2, outs = rows / 2;
#pragma unroll
    for (int i = 0; i < RT / 2; ++i) {
      if (i0 + i < outs) {
        const float s1 = total(n0 + 2 * i), s2 = total(n0 + 2 * i + 1);
        const float w1 = s1 > 0.f ? 1.f / s1 : 0.f, w2 = s2 > 0.f ? -__ldg(p.lambda + w.h * gh + (i0 + i) % gh) / s2 : 0.f;
#pragma unroll
        for (int mi = 0; mi < C::MT; ++mi)
          o[mi][i] = mi * 128 + r < p.row ? fmaf(o[mi][2 * i], w1, o[mi][2 * i + 1] * w2) : 0.f;
      }
    }
    if (p.norm_weight) {
      named_barrier_sync(1, 256);  // the sums have been read
#pragma unroll
      for (int i = 0; i < RT / 2; ++i) {
        if (i0 + i < outs) {
          float ss = 0.f;
#pragma unroll
          for (int mi = 0; mi < C::MT; ++mi) ss = fmaf(o[mi][i], o[mi][i], ss);
#pragma unroll
          for (int x = 16; x; x >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
          if (lane == 0) tab.red[quarter][i0 + i] = ss;
        }
      }
      named_barrier_sync(1, 256);
    }
    int hh = i0 % gh;
    T* dst = static_cast<T*>(p.out) + ((token0 + i0 / gh) * (p.heads / 2) + w.h * gh + hh) * p.row + r;
#pragma unroll
    for (int i = 0; i < RT / 2; ++i) {
      if (i0 + i < outs) {
        float post = p.out_scale;
        if (p.norm_weight) post *= inv_rms(p, total(i0 + i));
#pragma unroll
        for (int mi = 0; mi < C::MT; ++mi) {
          const int col = mi * 128 + r;
          if (col < p.row && f.ok)
            dst[mi * 128] = from_float<T>(o[mi][i] * post * (p.norm_weight ? __ldg(p.norm_weight + col) : 1.f));
        }
        dst += p.row;
        if (++hh == gh) {
          hh = 0;
          dst += (int64_t)(p.heads / 2 - gh) * p.row;
        }
      }
    }
  }
}

template <typename T, int D, int MAPS>
__global__ void __launch_bounds__(Few<T, D>::THREADS, 1)
    paged_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ PagedParams p) {
  using C = Few<T, D>;
  constexpr int NS = C::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;                            // [NS][KV_BYTES]: K(0), K(1), V(0), K(2), V(1), ... of each item
  uint8_t* sQ = ring + NS * C::KV_BYTES;           // [CB][32 rows][128 B]
  uint8_t* sP = sQ + C::Q_BYTES;                   // [2][P_BYTES]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sP + 2 * C::P_BYTES);
  uint64_t* q_full = bars;
  uint64_t* full = bars + 1;
  uint64_t* empty = full + NS;
  uint64_t* s_full = empty + NS;    // [2]
  uint64_t* p_full = s_full + 2;    // [2]
  uint64_t* pv_done = p_full + 2;   // [2]
  uint64_t* o_done = pv_done + 2;
  uint64_t* fin = o_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BARS);
  __shared__ RowTables tab;
  static_assert(C::SMEM + sizeof(RowTables) <= 232448, "shared memory budget");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  int* status = p.status;
  constexpr int kWarpK = 8, kWarpV = 9, kWarpMma = 10;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 256);
    for (int s = 0; s < NS; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full + s, 1);
      mbar_init(p_full + s, 256);
      mbar_init(pv_done + s, 1);
    }
    mbar_init(o_done, 1);
    mbar_init(fin, 1);
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  dependency_wait();
  dependency_trigger();
  const int failed = wait_failed(p);
  tc_fence_before();
  Start st;
  bool stop;
  if (p.small) {
    find_start_small<128>(p, st);
    stop = __syncthreads_or(failed);
  } else {
    find_start<128, C::THREADS>(p, &tab.start, tab.scan);
    stop = __syncthreads_or(failed);
    st = tab.start;
  }
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (stop || st.b < 0) {  // fewer tiles than CTAs
    if (warp == kWarpMma) tmem_dealloc(tmem, C::TMEM_COLS);
    return;
  }
  Walker<128> w;
  w.begin(p, st);

  // Barrier phases run on across items: the ring by a slot and its phase, the S and P buffers by a counter of tiles
  // (buffer g & 1, phase g / 2), q_full and o_done by items.
  if (warp == kWarpK || warp == kWarpV) {
    // -------------------------------------------------------------- producers: lane i loads box i of each tile
    // Two warps, since the boxes of small pages are many and a warp issues one in about 80 cycles; the order of the
    // ring says which slots are whose.
    const bool is_k = warp == kWarpK;
    const CUtensorMap* map = is_k ? &tmK : &tmV;
    const bool leader = elect_one();
    if (leader) tma_prefetch_desc(map);
    const int bs = p.block_size, box = p.box_rows;
    const bool has_box = lane * box < 128;
    const int oob_row = p.num_blocks * bs;
    bool ok = true;
    uint32_t loads = 0, last = 0;  // ring loads of the items before; this warp's last load
    do {
      const int32_t* bt = p.block_tables + (size_t)w.b * p.max_blocks;
      const int pages = (w.s.kv + bs - 1) / bs;
      const int cnt = w.t1 - w.t0;
      // the table entry of a tile's box is fetched one tile ahead, so its latency is not in the loop
      int pg = ((w.t1 - 1) * 128 + lane * box) / bs;
      int blk = has_box && pg < pages ? __ldg(bt + pg) : -1;
      for (int i = 0; i < cnt && ok; ++i) {
        const int j = w.t1 - 1 - i;
        const int pos = j * 128 + lane * box;
        int row = oob_row;  // past the last page: the load fills zeros
        if (has_box && pg < pages) {
          if (blk >= 0 && blk < p.num_blocks) row = blk * bs + (pos - pg * bs);
          else atomicCAS(status + 1, 0, kDevBadBlockIndex);
        }
        if (j > w.t0) {
          pg = (pos - 128) / bs;
          blk = has_box && pg < pages ? __ldg(bt + pg) : -1;
        }
        // K(0), K(1), V(0), K(2), V(1), ..., V(cnt - 1)
        const uint32_t g = loads + (is_k ? (i == 0 ? 0 : 2 * i - 1) : (i == cnt - 1 ? 2 * i + 1 : 2 * i + 2));
        const uint32_t slot = g % NS;
        if (g >= (uint32_t)NS)
          ok = __all_sync(0xffffffffu, mbar_wait(empty + slot, ((g / NS) - 1) & 1, status, kDevTimeoutKEmpty));
        if (!ok) break;
        if (leader) mbar_expect_tx(full + slot, C::KV_BYTES);
        __syncwarp();
        if (has_box) {
          uint8_t* dst = ring + slot * C::KV_BYTES + lane * box * 128;
#pragma unroll
          for (int cb = 0; cb < C::CB; ++cb) tma_load_3d(dst + cb * (128 * 128), map, full + slot, cb * 64, w.h, row);
        }
        __syncwarp();
        last = g;
      }
      loads += 2 * cnt;
    } while (ok && w.next(p));
    // Never leave the CTA while loads are still landing in shared memory.  The CTA ends when the last tile has been
    // multiplied, so that can only be after a failure, when these waits return within milliseconds.
    if (!ok)
      for (int s = 0; s < NS; ++s) mbar_wait(full + s, (last / NS) & 1, status, is_k ? kDevTimeoutKFull : kDevTimeoutVFull);
    __syncwarp();
  } else if (warp == kWarpMma) {
    // -------------------------------------------------------------- MMA issuer: warp-uniform, one lane issues
    const uint32_t lead = elect_one();
    const uint64_t dq = smem_desc_sw128(smem_addr(sQ), 16, 1024);
    const uint64_t dk = smem_desc_sw128(smem_addr(ring), 16, 1024);
    const uint64_t dv = smem_desc_sw128(smem_addr(ring), 128 * 128, 1024);  // V^T: the columns run along M
    const uint64_t dp = smem_desc_sw128(smem_addr(sP), 16, 1024);
    constexpr uint64_t kStep = C::KV_BYTES >> 4, kPStep = C::P_BYTES >> 4;
    auto wait_all = [&](uint64_t* bar, uint32_t parity, int code) { return wait_warp(bar, parity, status, code); };
    uint32_t slot = 0, phase = 0;
    auto advance = [&]() {
      if (++slot == NS) {
        slot = 0;
        phase ^= 1;
      }
    };
    bool ok = true;
    uint32_t g = 0, item = 0;
    do {
      const int cnt = __shfl_sync(0xffffffffu, w.t1 - w.t0, 0);
      const int rows = __shfl_sync(0xffffffffu, w.tokens(p) * p.group, 0);
      const uint32_t idesc_qk = instr_desc(ElemFmt<T>::fmt, false, false, 128, rows <= 16 ? 16 : 32);
      const bool one_p = MAPS == 2 && rows > 16;  // few_item's kOneP
      const uint32_t idesc_pv = instr_desc(ElemFmt<T>::fmt, true, false, 128, rows <= 8 ? 16 : one_p ? 64 : 32);
      const uint32_t p_cb = (one_p ? 2 * C::QCB : C::QCB) >> 4;
      auto issue_qk = [&](uint32_t b) -> bool {
        if (!wait_all(full + slot, phase, kDevTimeoutKFull)) return false;
        tc_fence_after();
        const uint64_t a0 = dk + slot * kStep;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss_by(lead, tmem + b * 32, a0 + (kk / 4) * ((128 * 128) >> 4) + (kk % 4) * 2, dq + (kk / 4) * (C::QCB >> 4) + (kk % 4) * 2,
                    idesc_qk, kk > 0);
        mma_commit_by(lead, s_full + b);
        mma_commit_by(lead, empty + slot);
        advance();
        return true;
      };
      // Q is written after the previous item's last product, so the S buffers and O are free from here on
      ok = wait_all(q_full, item & 1, kDevTimeoutQ) && issue_qk(g & 1);
      for (int u = 0; u < cnt && ok; ++u, ++g) {
        const uint32_t b = g & 1;
        // S of the next tile goes over that of the last one, which has been read: its P has come
        if (u + 1 < cnt && !(ok = issue_qk(b ^ 1))) break;
        ok = wait_warp2(full + slot, phase, kDevTimeoutVFull, p_full + b, (g >> 1) & 1, kDevTimeoutPFull, status);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a0 = dv + slot * kStep, b0 = dp + (one_p ? 0 : b * kPStep);
#pragma unroll
        for (int mi = 0; mi < C::MT; ++mi)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss_by(lead, tmem + C::O_COL + mi * 64, a0 + mi * ((2 * 128 * 128) >> 4) + kk * ((16 * 128) >> 4),
                      b0 + (kk / 4) * p_cb + (kk % 4) * 2, idesc_pv, (u > 0 || kk > 0) ? 1u : 0u);
        mma_commit_by(lead, empty + slot);
        mma_commit_by(lead, pv_done + b);
        if (u == cnt - 1) mma_commit_by(lead, o_done);
        advance();
      }
      ++item;
    } while (ok && w.next(p));
    // all tensor-core work this warp issued has finished before TMEM is released
    mma_commit_by(lead, fin);
    wait_all(fin, 0, kDevTimeoutFinal);
  } else {
    // -------------------------------------------------------------- softmax and epilogue
    const int r = threadIdx.x;
    const int group = p.group;
    FewState f{0, 0, true};
    uint32_t loads = 0;  // ring slots used so far
    if (r == 0) tab.join[0].n_seg = tab.join[1].n_seg = 0;
    int64_t line = st.line;
    do {
      const int tokens = w.tokens(p), rows = tokens * group, cnt = w.t1 - w.t0;
      const int64_t token0 = w.cu + (int64_t)w.rt * p.tb;
      const int off = w.s.kv - w.s.seq;
      const int R = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
      named_barrier_sync(1, 256);  // the last item's tables have been read
      if (r < R) {
        const int pos = w.rt * p.tb + r / group + off;
        tab.pos[r] = pos;
        // rows that fill up R see every key, so that they never decide whether a tile needs masks
        tab.last_key[r] = p.mask_type == 0 || r >= rows ? w.s.kv - 1 : min(pos, w.s.kv - 1);
        float* bias = reinterpret_cast<float*>(&tab.bias[r / 2]) + (r & 1);
        bias[0] = p.slopes && r < rows ? p.slopes[w.h * group + r % group] * kLog2e : 0.f;
        bias[2] = -static_cast<float>(r / group);
      }
      // ---- Q, K-major with the 128-byte swizzle, zeros in the rows that fill up R and behind the row's columns
      for (int i = r; i < R * (D / 8); i += 256) {
        const int row = i / (D / 8), c = i % (D / 8);
        const int qh = w.h * group + row % group;
        const int lo = MAPS == 2 ? (qh & 1) * (p.dq / 8) : 0;  // map 2 in the upper half
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < rows && c >= lo && c < lo + p.dq / 8)
          v = ld_query(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + (token0 + row / group) * p.q_stride + (int64_t)qh * p.dq) + (c - lo));
        st_shared_v4(smem_addr(sQ) + (c >> 3) * C::QCB + row * 128 + (((c & 7) ^ (row & 7)) << 4), v);
      }
      __syncwarp();
      fence_proxy_async_smem();
      tc_fence_before();  // the previous item's loads of O come before the product that overwrites it
      mbar_arrive(q_full);
      named_barrier_sync(1, 256);  // the tables are written
      const uint32_t v0 = loads + (cnt > 1 ? 2 : 1);  // the first tile's V in the order of loads
      uint64_t* v_full0 = full + v0 % NS;
      const uint32_t v_phase0 = (v0 / NS) & 1;
      const uint32_t sp = smem_addr(sP);
      if (R == 8)
        few_item<T, D, 8, MAPS>(p, w, f, tab, ring, v0 % NS, v_full0, v_phase0, sp, s_full, p_full, pv_done, o_done, tmem, token0, tokens);
      else if (R == 16)
        few_item<T, D, 16, MAPS>(p, w, f, tab, ring, v0 % NS, v_full0, v_phase0, sp, s_full, p_full, pv_done, o_done, tmem, token0, tokens);
      else
        few_item<T, D, 32, MAPS>(p, w, f, tab, ring, v0 % NS, v_full0, v_phase0, sp, s_full, p_full, pv_done, o_done, tmem, token0, tokens);
      loads += 2 * cnt;
      if (w.t0 > 0 || w.t1 < w.n) {
        // ---- a cut item: whoever brings its last segment joins them, so nobody waits
        named_barrier_sync(1, 256);
        if (r == 0) {
          __threadfence();  // with the barrier: all threads' partials come before the count
          const int64_t tile0 = line - w.t0;
          const int q0 = st.part_of(tile0), n_seg = st.part_of(tile0 + w.n - 1) - q0 + 1;
          const int first = q0 * p.head_stride + (p.head_stride > 1 ? w.h : 0);
          const bool last = f.ok && atomicAdd(p.arrived + first, 1) == n_seg - 1;
          if (last) {
            p.arrived[first] = 0;  // for the next execution
            __threadfence();
          }
          const int k = w.t0 > 0 ? 0 : 1;
          tab.join[k] = PagedDesc{last ? n_seg : 0, (int)token0, tokens, w.h, w.rt * p.tb + off, 0};
          tab.first[k] = first;
        }
      }
      line += cnt;
    } while (w.next(p));
    // ---- the joins that fell to this CTA, both items' rows side by side (after the loop, so that what a join holds in
    // registers does not weigh on the tiles)
    named_barrier_sync(1, 256);
    const int n0 = tab.join[0].n_seg ? tab.join[0].tokens * group / MAPS : 0, n1 = tab.join[1].n_seg ? tab.join[1].tokens * group / MAPS : 0;
    for (int o = warp; o < n0 + n1; o += 8) {
      const int k = o < n0 ? 0 : 1, row = o - k * n0, gh = group / MAPS;
      combine_row<T, D, MAPS>(p, tab.join[k], tab.first[k], row / gh, row % gh);
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

template <typename T, int D, int MAPS>
cudaError_t launch_maps(const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedParams& p, cudaStream_t stream) {
  using C = Few<T, D>;
  const cudaError_t e = cudaFuncSetAttribute(paged_few_kernel<T, D, MAPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_few_kernel<T, D, MAPS>, dim3(kGrid), C::THREADS, C::SMEM, stream, tmK, tmV, p);
}

template <typename T, int D>
cudaError_t launch(const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedParams& p, cudaStream_t stream) {
  return p.maps() == 1 ? launch_maps<T, D, 1>(tmK, tmV, p, stream) : launch_maps<T, D, 2>(tmK, tmV, p, stream);
}

}  // namespace

cudaError_t launch_paged_few(int32_t dtype, int D, const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedParams& p,
                             cudaStream_t stream) {
  if (dtype == kF16)
    return D == 64 ? launch<__half, 64>(tmK, tmV, p, stream)
         : D == 128 ? launch<__half, 128>(tmK, tmV, p, stream) : launch<__half, 256>(tmK, tmV, p, stream);
  return D == 64 ? launch<__nv_bfloat16, 64>(tmK, tmV, p, stream)
       : D == 128 ? launch<__nv_bfloat16, 128>(tmK, tmV, p, stream) : launch<__nv_bfloat16, 256>(tmK, tmV, p, stream);
}

}  // namespace ala
