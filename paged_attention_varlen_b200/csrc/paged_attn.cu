// paged_attn.cu -- attention of each sequence's new tokens (one, a few, or a chunk) over its paged cache,
// with every length read on the device, and its differential form.
//
//   O[t, h] = sum_j softmax_j(qkScale q[t, h] . k_j + bias) v_j                       (ala_paged_attention)
//   O[t, h] = sum_j (softmax_j(s1) - lambda_h softmax_j(s2)) v_j, s_m = qkScale q[t, 2h + m] . k_(m),j
//             and then, optionally, O <- O * rsqrt(mean(O^2) + eps) * w               (ala_paged_diff_attention)
//
// This kernel is for many query rows of a kv head, paged_few.cu for up to 32 (paged_run says which runs when).
//
// Rows.  The queries of one kv head are packed (token, head of the group), so that K / V are read once for the
// group.  An item is the rows of up to two blocks of 128 (one at D = 256, whose O leaves no room in tensor
// memory for a second) against one kv head's keys, in tiles of 128 keys (64 at D = 256).
//   two blocks    more than 128 rows: every tile serves both blocks, and one block's products run while the
//                 other's softmax does
//   in turns      up to 128 rows: the blocks are the same rows, and take the tiles in turn; joined at the end
//
// Differential attention is the same kernel over K rows [k1 | k2] of 2d elements, as they lie in the cache:
// the query row of map 1 is [q1 | 0], that of map 2 is [0 | q2].  With two blocks a block is a map, and its
// score product runs over that map's half alone; otherwise the two maps of a head are neighbouring rows.
//
// Work split.  All key tiles of all (sequence, kv head, row tile) items form one line; CTA c of G takes the
// tiles [c T / G, (c + 1) T / G).  A CTA finds its start by a scan over the batch and a search inside one
// sequence, so the schedule needs no host lengths and no planning launch, and every CTA gets the same number
// of tiles whatever the lengths are.  An item cut by a CTA boundary leaves unnormalised fp32 partials with
// the running max and sum of each row; paged_combine_kernel joins them in segment order.
// Tiles run from the last key to the first: under ALiBi the largest scores come first, so that the running
// max hardly moves after the first tile and O is not rescaled (first to last rescaled it at every tile).
//
// Pipeline of a CTA (one per SM), NB blocks:
//   warps 0 .. 4 NB - 1   softmax of block b, thread r owns row r (TMEM lane r)
//   then a warp each      TMA producer of the K ring, of the V ring (lane i gathers box i of a tile through
//                         the block table), and the tcgen05 issuer: S_b = Q K^T, O_b += P_b V with P_b read
//                         from TMEM over S_b, P V in two halves of the keys
//
// What bounds it: a block's chain of softmax (some 2900 cycles for 128 keys, of which 1024 to 2048 are ex2, the tensor
// pipe's 512 to 1024 aside) and, with two S buffers, P V and the next Q K^T (1700).  The two blocks overlap; tensor
// pipe and ex2 unit both run at 38 % of their cycles (2 x 2048 new tokens over 8000 keys), DRAM at 4 %.
// Measured: 3 chunks of up to 4096 over 20000 keys, 32 / 8 heads, d 128: 2.24 to 2.6 ms, 820 to 960 TFLOP/s, by the
// clock that the power cap leaves.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <type_traits>

#include "paged_common.cuh"

namespace ala {

namespace {

// Blocks per segment list in the combine grid.  2, 4, 8, 16 and 32 of them: 4 chunks of 115 to 150 tokens over 1100 keys
// 61, 52, 52, 52 and 56 us, the decoding rows and chunks of D = 64 394, 392, 388, 389 and 392, long chunks alike.
constexpr int kCombineY = 4;

// The rings fill what shared memory leaves: a tile arrives a few thousand cycles after its load is issued, so
// depth is what keeps HBM busy.
// NQ: blocks of Q rows.  With one (items of at most 128 rows), the second's room goes to the rings.
template <typename T, int D_, int NQ_>
struct Cfg {
  static constexpr int D = D_, NQ = NQ_;
  static constexpr int NB = D == 256 ? 1 : 2;     // blocks of 128 rows
  static constexpr int TK = D == 256 ? 64 : 128;  // keys per tile
  static constexpr int THREADS = NB * 128 + 128;
  static constexpr int CB = D / 64;               // 128-byte column blocks of a row
  static constexpr int Q_BYTES = 128 * D * 2;     // one block
  static constexpr int KV_BYTES = TK * D * 2;
  static constexpr int NSK = D == 64 ? 5 : D == 128 ? 4 - NQ : 3;
  static constexpr int NSV = D == 64 ? 6 : D == 128 ? 3 : 2;
  static constexpr int SCRATCH = NQ * Q_BYTES;    // the Q buffers between items: what the joins pass through
  // S buffers.  A third, where tensor memory has room for it, takes the scores of a block's next tile while the block's
  // softmax still works on this one: chunks of D = 64 beside decoding rows 441 -> 407 us.
  static constexpr int NBUF = D == 64 ? 3 : 2;
  static constexpr int N_BARS = 1 + 2 * NSK + 2 * NSV + 5 * NBUF + 2 + 1;
  static constexpr int SMEM = 1024 + NQ * Q_BYTES + (NSK + NSV) * KV_BYTES + 256 * 4 + N_BARS * 8 + 16;  // 256 floats: sM
  static constexpr uint32_t S_COL(int k) { return k * TK; }
  static constexpr uint32_t O_COL(int b) { return NBUF * TK + (NB == 2 ? b * D : 0); }
  static constexpr uint32_t TMEM_COLS = 512;
  static_assert(SCRATCH / (NB * 4 * 32 * 4) % 32 == 0, "the joins take 32 columns at a time");
  static_assert(NBUF * TK + NB * D <= TMEM_COLS, "tensor memory budget");
};

// ---------------------------------------------------------------------------------------------- softmax

template <int NC>
__device__ __forceinline__ void load_cols(uint32_t col, float (&x)[NC]) {
  uint32_t r[NC / 32][32];
#pragma unroll
  for (int i = 0; i < NC / 32; ++i) tmem_ld32(col + i * 32, r[i]);
  tmem_ld_wait();  // one wait for all loads
#pragma unroll
  for (int c = 0; c < NC; ++c) x[c] = __uint_as_float(r[c >> 5][c & 31]);
}

// What a row keeps over an item.
struct RowState {
  float m, l;        // running max (log2 units; the one P is computed against; kNoKey before any key) and sum
  int last_key;      // keys j <= last_key are allowed (-1: none)
  int pos;           // absolute position of the row's token
  float slope_log2;
};

// Scores of the NC columns from key `first` of a row, in log2 units (raw where raw_max says so); returns their
// maximum in log2 units.
template <int NC>
__device__ __forceinline__ float scores(const PagedParams& p, const RowState& rs, float (&x)[NC], int first, bool raw_max) {
  const int mt = p.mask_type;
  const float scale = p.scale_log2;
  const int lim = rs.last_key - first;  // columns c <= lim are allowed
  if (mt == 3 || mt == 5) {
    // right- and left-aligned bias differ by a per-row constant; both use (j - pos)
    const float b0 = rs.slope_log2 * static_cast<float>(first - rs.pos);
#pragma unroll
    for (int c = 0; c < NC; ++c) x[c] = fmaf(x[c], scale, fmaf(rs.slope_log2, static_cast<float>(c), b0));
  } else if (mt == 4) {
    const float d0 = static_cast<float>(rs.pos - first);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      x[c] = fmaf(x[c], scale, -rs.slope_log2 * sqrt_approx(fmaxf(d0 - static_cast<float>(c), 0.f)));
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
  const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
  return raw_max ? mx * scale : mx;
}

// Takes a tile's maximum into the running one.  Returns the factor that O and l must be rescaled by (1: none).
__device__ __forceinline__ float grow(RowState& rs, float mx) {
  const float m_new = fmaxf(rs.m, mx);
  if (!(m_new - rs.m > kRescaleThreshold)) return 1.f;
  const float alpha = fast_exp2(rs.m - m_new);
  rs.m = m_new;
  return alpha;
}

// P = 2^(x - m) of N columns from C0 on, packed; adds to the four partial sums.  P is rounded to the operand type of
// the tensor core; the sum takes the unrounded values, so a row's rounding errors (at most half a step of each
// weight) average out instead of biasing the normalisation.  In a difference of two maps what they have in common
// cancels and their rounding errors do not, so there (CARRY) a second P carries what rounding drops, and P V is exact
// to 2^-17 or so.  Measured on chunks in f16: error 0.00032 -> 0.00021 of the output, which is its own rounding, and
// 413 to 437 -> 448 us.
template <typename T, int C0, int N, bool CARRY, int NC>
__device__ __forceinline__ void exponentials(const float (&x)[NC], uint64_t scale2, uint64_t negm2, uint64_t (&acc)[4],
                                             uint32_t (&pk)[N / 2], uint32_t (&rest)[N / 2]) {
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    float e0, e1;
    f2unpack(fma_x2(f2pack(x[C0 + c], x[C0 + c + 1]), scale2, negm2), e0, e1);
    e0 = fast_exp2(e0);
    e1 = fast_exp2(e1);
    acc[(c >> 1) & 3] = add_x2(acc[(c >> 1) & 3], f2pack(e0, e1));
    pk[c / 2] = pack2(e0, e1, (T*)nullptr);
    if constexpr (CARRY) {
      const float2 h = unpack2(pk[c / 2], (T*)nullptr);
      rest[c / 2] = pack2(e0 - h.x, e1 - h.y, (T*)nullptr);
    }
  }
}

__device__ __forceinline__ float sum4(const uint64_t (&acc)[4]) {
  float s0, s1;
  f2unpack(add_x2(add_x2(acc[0], acc[1]), add_x2(acc[2], acc[3])), s0, s1);
  return s0 + s1;
}

// 16 columns at a time, so that few packed weights are live at once.
template <typename T, int C0, bool CARRY, int NC>
__device__ __forceinline__ void columns_16(const float (&x)[NC], uint64_t scale2, uint64_t negm2, uint64_t (&acc)[4], uint32_t col) {
  uint32_t pk[8], rest[8];
  exponentials<T, C0, 16, CARRY>(x, scale2, negm2, acc, pk, rest);
  tmem_st8(col + C0 / 2, pk);
  if constexpr (CARRY) tmem_st8(col + NC / 2 + C0 / 2, rest);
  if constexpr (C0 + 16 < NC) columns_16<T, C0 + 16, CARRY>(x, scale2, negm2, acc, col);
}

// P of NC columns over the scores they came from: the rounded weights, then (CARRY) what rounding dropped.  Returns the
// sum.
template <typename T, bool CARRY, int NC>
__device__ __forceinline__ float write_p(const float (&x)[NC], uint64_t scale2, uint64_t negm2, uint32_t col) {
  uint64_t acc[4] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f), f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
  if constexpr (!CARRY && NC == 64) {
    uint32_t pk[32];
    exponentials<T, 0, 64, false>(x, scale2, negm2, acc, pk, pk);
    tmem_st32(col, pk);
  } else {
    columns_16<T, 0, CARRY>(x, scale2, negm2, acc, col);
  }
  return sum4(acc);
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

template <typename T, int D, int NQ, int MAPS>
__global__ void __launch_bounds__(Cfg<T, D, NQ>::THREADS, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const PagedParams p) {
  using C = Cfg<T, D, NQ>;
  constexpr int TK = C::TK, NSK = C::NSK, NSV = C::NSV, NB = C::NB, NBUF = C::NBUF;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                        // [NQ][Q_BYTES]; between items the scratch of the joins
  uint8_t* sK = sQ + NQ * C::Q_BYTES;        // [NSK][KV_BYTES]
  uint8_t* sV = sK + NSK * C::KV_BYTES;      // [NSV][KV_BYTES]
  float* sM = reinterpret_cast<float*>(sV + NSV * C::KV_BYTES);  // [256] maxima and sums of the joins
  uint64_t* bars = reinterpret_cast<uint64_t*>(sM + 256);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;
  uint64_t* k_empty = k_full + NSK;
  uint64_t* v_full = k_empty + NSK;
  uint64_t* v_empty = v_full + NSV;
  uint64_t* s_full = v_empty + NSV;     // [NBUF] per S buffer
  uint64_t* p_lo = s_full + NBUF;       // [NBUF] P of the tile's first half of keys written
  uint64_t* p_full = p_lo + NBUF;       // [NBUF] all of P
  uint64_t* lo_done = p_full + NBUF;    // [NBUF] the product of P's first half
  uint64_t* pv_done = lo_done + NBUF;   // [NBUF]
  uint64_t* o_done = pv_done + NBUF;    // [2] per block: the item's last product
  uint64_t* fin = o_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BARS);
  __shared__ Start st;
  __shared__ int64_t red[2 * C::THREADS / 32];
  static_assert(C::SMEM + sizeof(st) + sizeof(red) <= 232448, "shared memory budget");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  int* status = p.status;
  constexpr int kWarpK = NB * 4, kWarpV = kWarpK + 1, kWarpMma = kWarpK + 2;

  if (threadIdx.x == 0) {
    mbar_init(q_full, NB * 128);
    for (int s = 0; s < NSK; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(k_empty + s, 1);
    }
    for (int s = 0; s < NSV; ++s) {
      mbar_init(v_full + s, 1);
      mbar_init(v_empty + s, 1);
    }
    for (int s = 0; s < NBUF; ++s) {
      mbar_init(s_full + s, 1);
      mbar_init(p_lo + s, 128);
      mbar_init(p_full + s, 128);
      mbar_init(lo_done + s, 1);
      mbar_init(pv_done + s, 1);
    }
    mbar_init(o_done, 1);
    mbar_init(o_done + 1, 1);
    mbar_init(fin, 1);
    fence_mbar_init();
  }
  dependency_wait();
  const int failed = wait_failed(p);
  find_start<TK, C::THREADS>(p, &st, red);
  if (__syncthreads_or(failed) || st.b < 0) {  // fewer tiles than CTAs
    if (threadIdx.x == 0) p.desc[blockIdx.x].n_seg = 0;
    return;
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  Walker<TK> w;
  w.begin(p, st);

  // An item of cnt tiles is U steps: step u fills S buffer u % NBUF and multiplies its P.  With two blocks of rows,
  // steps 2i and 2i + 1 are tile i for block 0 and 1; otherwise step u is tile u, for block u & 1 of the two that
  // hold the same rows (NB = 1: for the one block).  Ring phases run on across items by a counter of tiles (slot
  // g % depth, phase g / depth), those of a buffer by its count of steps, q_full and o_done by items.
  uint32_t used[NBUF] = {};  // steps of each S buffer in the items before
  auto phase_of = [&](int u) {  // of step u's buffer
    uint32_t c = used[0];
    if (NBUF == 3 ? u % 3 == 1 : (u & 1)) c = used[1];
    if (NBUF == 3 && u % 3 == 2) c = used[NBUF - 1];
    return (c + u / NBUF) & 1;
  };
  auto count_steps = [&](int U) {
#pragma unroll
    for (int k = 0; k < NBUF; ++k) used[k] += (U - k + NBUF - 1) / NBUF;
  };
  auto is_two = [&]() { return NQ == 2 && w.tokens(p) * p.group > 128; };
  // register split for NB = 2: the softmax warps take 216 each, the others keep 72 (256 * 216 + 128 * 72 =
  // 64512 = 384 * 168, all that the block is launched with)
  if (warp >= kWarpK) {
    if constexpr (NB == 2) regs_decrease<72>();
  }
  if (warp == kWarpK || warp == kWarpV) {
    // -------------------------------------------------------------- producers
    const bool is_k = warp == kWarpK;
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
      int pg = ((w.t1 - 1) * TK + lane * box) / bs;
      int blk = has_box && pg < pages ? __ldg(bt + pg) : -1;
      for (int j = w.t1 - 1; j >= w.t0; --j, ++g) {
        const int slot = g % depth;
        const int pos = j * TK + lane * box;
        int row = oob_row;  // past the last page: the load fills zeros
        if (has_box && pg < pages) {
          if (blk >= 0 && blk < p.num_blocks) row = blk * bs + (pos - pg * bs);
          else atomicCAS(status + 1, 0, kDevBadBlockIndex);
        }
        if (j > w.t0) {
          pg = (pos - TK) / bs;
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
        __syncwarp();
      }
    } while (ok && w.next(p));
    // never leave the CTA while loads this warp issued are still landing in shared memory
    for (uint32_t i = g >= (uint32_t)depth ? g - depth : 0; i < g; ++i)
      mbar_wait(full_bar + (i % depth), (i / depth) & 1, status, is_k ? kDevTimeoutKFull : kDevTimeoutVFull);
    __syncwarp();
  } else if (warp == kWarpMma) {
    // -------------------------------------------------------------- MMA issuer: a warp in step, one lane issues
    const uint32_t lead = elect_one();
    const uint64_t dq = smem_desc_sw128(smem_addr(sQ), 16, 1024);
    const uint64_t dk = smem_desc_sw128(smem_addr(sK), 16, 1024);
    const uint64_t dv = smem_desc_sw128(smem_addr(sV), TK * 128, 1024);  // MN-major
    constexpr uint64_t kQStep = C::Q_BYTES >> 4, kStep = C::KV_BYTES >> 4;
    constexpr uint32_t kIdescQk = instr_desc(ElemFmt<T>::fmt, false, false, 128, TK);
    // P V makes the row's columns only, rounded up to the instruction's step of 16
    const uint32_t idesc_pv = instr_desc(ElemFmt<T>::fmt, false, true, 128, (p.row + 15) & ~15);
    constexpr bool per_map = MAPS == 2;  // with two blocks a block is a map
    const int steps_row = (p.row + 15) / 16;
    auto wait_all = [&](uint64_t* bar, uint32_t parity, int code) { return wait_warp(bar, parity, status, code); };
    bool ok = true;
    uint32_t item = 0;
    uint32_t ks = 0, kp = 0, vs = 0, vp = 0;  // ring positions: slot and phase
    do {
      const int cnt = __shfl_sync(0xffffffffu, w.t1 - w.t0, 0);
      const bool two = __any_sync(0xffffffffu, is_two());
      const int U = two ? 2 * cnt : cnt;
      // K of step u has arrived (the second block finds its tile there)
      auto wait_k = [&](int u) { return (two && (u & 1)) || wait_all(k_full + ks, kp, kDevTimeoutKFull); };
      auto issue_qk = [&](int u) -> bool {
        const int b = u & 1, k = u % NBUF;
        // the buffer's previous P has been multiplied (before the item: q_full says so)
        if (u >= NBUF && !wait_all(pv_done + k, phase_of(u - NBUF), kDevTimeoutODone)) return false;
        tc_fence_after();
        const uint64_t a0 = dq + (two && b ? kQStep : 0), b0 = dk + ks * kStep;
        const uint32_t d = tmem + C::S_COL(k);
        auto step = [&](int kk, bool acc) {
          const uint32_t in = (kk % 4) * (32 >> 4);
          mma_ss_by(lead, d, a0 + ((kk / 4) * ((128 * 128) >> 4) + in), b0 + ((kk / 4) * ((TK * 128) >> 4) + in), kIdescQk, acc);
        };
        if (two && per_map) {  // the columns of the block's map alone
          const int lo = b * p.dq / 16, hi = ((b + 1) * p.dq + 15) / 16;
#pragma unroll 1
          for (int kk = lo; kk < hi; ++kk) step(kk, kk > lo);
        } else if (steps_row == D / 16) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) step(kk, kk > 0);
        } else {
#pragma unroll 1
          for (int kk = 0; kk < steps_row; ++kk) step(kk, kk > 0);
        }
        mma_commit_by(lead, s_full + k);
        if (!two || b == 1) {
          mma_commit_by(lead, k_empty + ks);
          if (++ks == NSK) {
            ks = 0;
            kp ^= 1;
          }
        }
        return true;
      };
      // Q is written after the previous item's last product, so the S buffers and O are free from here on
      ok = wait_all(q_full, item & 1, kDevTimeoutQ);
      for (int u = 0; u < NBUF && u < U && ok; ++u) ok = wait_k(u) && issue_qk(u);
      for (int u = 0; u < U && ok; ++u) {
        const int b = u & 1;
        const int k = u % NBUF;
        const uint32_t ph = phase_of(u);
        const uint64_t v0 = dv + vs * kStep;
        const uint32_t o = tmem + C::O_COL(b), pcol = tmem + C::S_COL(k);
        auto issue_pv = [&](int half) {
          constexpr int NC = TK / 2, KH = NC / 16;  // a half's columns of S and steps
#pragma unroll
          for (int kk = 0; kk < KH; ++kk)
            mma_ts_by(lead, o, pcol + half * NC + kk * 8, v0 + (((half * KH + kk) * 16 * 128) >> 4), idesc_pv,
                      (u >= NB || half > 0 || kk > 0) ? 1u : 0u);
          if (per_map) {  // what rounding P dropped
#pragma unroll
            for (int kk = 0; kk < KH; ++kk)
              mma_ts_by(lead, o, pcol + half * NC + NC / 2 + kk * 8, v0 + (((half * KH + kk) * 16 * 128) >> 4), idesc_pv, 1u);
          }
        };
        ok = two && b == 1 ? wait_all(p_lo + k, ph, kDevTimeoutPFull)
                           : wait_warp2(v_full + vs, vp, kDevTimeoutVFull, p_lo + k, ph, kDevTimeoutPFull, status);
        if (!ok) break;
        tc_fence_after();
        issue_pv(0);
        mma_commit_by(lead, lo_done + k);
        ok = u + NBUF >= U || (two && ((u + NBUF) & 1)) ? wait_all(p_full + k, ph, kDevTimeoutPFull)
                                                        : wait_warp2(k_full + ks, kp, kDevTimeoutKFull, p_full + k, ph, kDevTimeoutPFull, status);
        if (!ok) break;
        tc_fence_after();
        issue_pv(1);
        mma_commit_by(lead, pv_done + k);
        if (!two || b == 1) {
          mma_commit_by(lead, v_empty + vs);
          if (++vs == NSV) {
            vs = 0;
            vp ^= 1;
          }
        }
        if (u + NB >= U) mma_commit_by(lead, o_done + (NB == 2 ? b : 0));
        if (u + NBUF < U) ok = issue_qk(u + NBUF);
      }
      count_steps(U);
      ++item;
    } while (ok && w.next(p));
    // all tensor-core work this warp issued has finished before TMEM is released
    mma_commit_by(lead, fin);
    wait_all(fin, 0, kDevTimeoutFinal);
  } else if (warp < kWarpK) {
    // -------------------------------------------------------------- softmax and epilogue
    if constexpr (NB == 2) regs_increase<216>();
    const int blk = warp >> 2, wq = warp & 3;
    const int r = threadIdx.x & 127;  // TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t o_col = tmem + lanes + C::O_COL(blk);
    const int group = p.group, gh = group / MAPS;
    const bool raw_max = (p.mask_type == 0 || p.mask_type == 9) && p.scale_log2 > 0.f;  // scale folded into the exponent
    const uint64_t scale2 = raw_max ? f2pack(p.scale_log2, p.scale_log2) : f2pack(1.f, 1.f);
    uint32_t g0 = 0, items = 0;  // tiles; items that this block took part in
    bool owner = false;
    // After a failed wait a warp skips what is left of the tiles, but goes on through the items, so that the
    // warps meet as often as ever.
    bool ok = true;
    int64_t line = st.line;
    auto meet = [&]() { named_barrier_sync(1, NB * 128); };
    do {
      const int cnt = w.t1 - w.t0, tokens = w.tokens(p);
      const bool two = is_two();
      const int steps = NB == 1 || two ? cnt : (cnt + 1 - blk) >> 1;  // this block's
      const int off = w.s.kv - w.s.seq;
      // this thread's row: its token in the tile and query head
      int tok, qh;
      bool valid;
      if (two && MAPS == 2) {
        tok = r / gh;
        qh = (w.h * gh + r % gh) * 2 + blk;
        valid = tok < tokens;
      } else {
        tok = r / group + (two ? blk * p.tb1 : 0);
        qh = w.h * group + r % group;
        valid = tok < tokens && (!two || blk == 1 || r / group < p.tb1);
      }
      const int64_t token0 = w.cu + (int64_t)w.rt * p.tb, token = token0 + tok;
      RowState rs;
      rs.m = kNoKey;
      rs.l = 0.f;
      rs.pos = w.rt * p.tb + tok + off;
      rs.last_key = !valid ? -1 : p.mask_type == 0 ? w.s.kv - 1 : min(rs.pos, w.s.kv - 1);
      rs.slope_log2 = (valid && p.slopes) ? p.slopes[qh] * kLog2e : 0.f;
      // ---- Q row to shared memory, K-major with the 128-byte swizzle; blocks of the same rows write half of it each
      if (valid) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + token * p.q_stride + (int64_t)qh * p.dq);
        const int lo = MAPS == 2 ? (qh & 1) * (p.dq / 8) : 0, hi = lo + p.dq / 8;  // map 2 in the upper half
        const bool share = NB == 2 && !two;
        const uint32_t dst = smem_addr(sQ) + (two ? blk * C::Q_BYTES : 0) + r * 128;
        const int c0 = share ? blk * (D / 16) : 0;
        constexpr int G = 8;  // 16-byte loads in flight
#pragma unroll
        for (int i0 = 0; i0 < D / 8; i0 += G) {
          if (share && i0 >= D / 16) break;
          uint4 v[G];
#pragma unroll
          for (int i = 0; i < G; ++i) {
            const int c = c0 + i0 + i;
            v[i] = c >= lo && c < hi ? ld_query(src + (c - lo)) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < G; ++i) {
            const int c = c0 + i0 + i;
            if (!share || i0 + i < D / 16) st_shared_v4(dst + (c >> 3) * (128 * 128) + (((c & 7) ^ (r & 7)) << 4), v[i]);
          }
        }
      }
      __syncwarp();
      fence_proxy_async_smem();
      tc_fence_before();  // the previous item's loads of O come before the product that overwrites it
      mbar_arrive(q_full);
      // ---- key tiles, from the last
      const bool warp_rows = __any_sync(0xffffffffu, valid);
      for (int s = 0; s < steps && ok; ++s) {
        const int u = NB == 2 ? 2 * s + blk : s;  // step of the item
        const int sb = u % NBUF;                  // its S buffer
        const uint32_t ph = phase_of(u);
        const int i = NB == 1 || two ? s : 2 * s + blk;  // tile of the item
        const int j0 = (w.t1 - 1 - i) * TK;
        const uint32_t s_col = tmem + lanes + C::S_COL(sb);
        ok = __all_sync(0xffffffffu, mbar_wait(s_full + sb, ph, status, kDevTimeoutSFull));
        if (!ok) break;
        tc_fence_after();
        if (s == 0 && blk == 0 && j0 + TK > w.s.kv) {
          // slots past kvSeqLen may hold anything, NaN included, and 0 * NaN is not 0: clear their V rows.  Block 0
          // has the first product of the item's first tile, so it does so for both.
          const int slot = g0 % NSV;
          ok = __all_sync(0xffffffffu, mbar_wait(v_full + slot, (g0 / NSV) & 1, status, kDevTimeoutVFull));
          if (!ok) break;
          if (r < TK && j0 + r >= w.s.kv) {
            const uint32_t dst = smem_addr(sV + slot * C::KV_BYTES) + r * 128;
#pragma unroll
            for (int cb = 0; cb < C::CB; ++cb)
#pragma unroll
              for (int c = 0; c < 8; ++c) st_shared_v4(dst + cb * TK * 128 + c * 16, make_uint4(0, 0, 0, 0));
          }
          __syncwarp();
          fence_proxy_async_smem();
        }
        if (warp_rows) {
          // The tile's halves, of which P V takes one after the other, in turn.  A half's P is computed against the
          // running maximum as it stands, while its own maximum is found; only where that is more than 2^8 above,
          // the maximum moves, O and l are rescaled and the half is computed again.
          constexpr int NC = TK / 2;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            float x[NC];
            load_cols<NC>(s_col + half * NC, x);
            const float mx = scores<NC>(p, rs, x, j0 + half * NC, raw_max);
            float alpha = 1.f;
            if (s == 0 && half == 0) grow(rs, mx);  // nothing to rescale yet
            float sum;
#pragma unroll 1
            for (;;) {
              const uint64_t negm2 = f2pack(-rs.m, -rs.m);
              sum = write_p<T, MAPS == 2>(x, scale2, negm2, s_col + half * NC);
              if (!__any_sync(0xffffffffu, mx - rs.m > kRescaleThreshold)) break;
              alpha = grow(rs, mx);
              // O must be at rest: after the product of the first half, or of the block's step before
              const int before = NB == 2 ? u - 2 : u - 1;
              ok = __all_sync(0xffffffffu, half == 1 ? mbar_wait(lo_done + sb, ph, status, kDevTimeoutODone)
                                                     : mbar_wait(pv_done + (before + NBUF) % NBUF, phase_of(before), status, kDevTimeoutODone));
              if (!ok) break;
              tc_fence_after();
              scale_rows<D>(o_col, alpha);
            }
            if (!ok) break;
            rs.l = rs.l * alpha + sum;
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive((half ? p_full : p_lo) + sb);
          }
          if (!ok) break;
        } else {  // no row of the tile: what the lanes hold of P and O is read by nobody
          mbar_arrive(p_lo + sb);
          mbar_arrive(p_full + sb);
        }
      }
      g0 += cnt;
      count_steps(two ? 2 * cnt : cnt);
      // o_done has one phase per item that the block took part in and is waited for once in each, so no wait can
      // meet the phase before or after its own
      if (steps > 0) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(o_done + blk, items & 1, status, kDevTimeoutODone));
        ++items;
      }
      tc_fence_after();
      const bool whole = w.t0 == 0 && w.t1 == w.n;
      // partials: slot 1 when the item starts here, 0 when it began in an earlier CTA
      const int64_t prow0 = ((int64_t)blockIdx.x * 2 + (w.t0 == 0 ? 1 : 0)) * (NB * 128);
      if (!whole && w.t0 == 0 && threadIdx.x == 0) {
        PagedDesc d;
        d.n_seg = st.part_of(line + w.n - 1) - (int)blockIdx.x + 1;
        d.token0 = (int)token0;
        d.tokens = tokens;
        d.kv_head = w.h;
        d.pos0 = w.rt * p.tb + off;
        d.two = two;
        p.desc[blockIdx.x] = d;
        owner = true;
      }
      line += cnt;
      bool has_rows = warp_rows;
      float* exchange = reinterpret_cast<float*>(sQ);  // a row of XCOLS floats for each thread, chunks swizzled by the row
      constexpr int XCOLS = C::SCRATCH / (128 * 4) < D ? C::SCRATCH / (128 * 4) : D;
      auto slot4 = [&](int c4) { return reinterpret_cast<float4*>(exchange + (size_t)r * XCOLS) + (c4 ^ (r & 7)); };
      if (NB == 2 && !two) {
        // ---- the blocks hold the same rows: block 1 hands its row to block 0, through the Q buffers, once block 0's
        // last score product has read those too
        float f0 = 1.f, f1 = 0.f;
#pragma unroll 1
        for (int x0 = 0; x0 < D; x0 += XCOLS) {
          meet();
          if (blk == 1) {
            if (x0 == 0) {
              sM[r] = rs.m;
              sM[128 + r] = rs.l;
            }
            if (warp_rows) {
#pragma unroll 1
              for (int c32 = 0; c32 < XCOLS / 32; ++c32) {
                uint32_t regs[32];
                if (steps > 0) {
                  tmem_ld32(o_col + x0 + c32 * 32, regs);
                  tmem_ld_wait();
                }
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  *slot4(c32 * 8 + c) = steps == 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                   : make_float4(__uint_as_float(regs[4 * c]), __uint_as_float(regs[4 * c + 1]),
                                                                 __uint_as_float(regs[4 * c + 2]), __uint_as_float(regs[4 * c + 3]));
              }
            }
          }
          meet();
          if (blk == 0 && warp_rows) {
            if (x0 == 0) {
              const float m1 = sM[r], l1 = sM[128 + r], top = fmaxf(rs.m, m1);
              f0 = fast_exp2(rs.m - top);
              f1 = fast_exp2(m1 - top);
              rs.l = rs.l * f0 + l1 * f1;
              rs.m = top;
            }
#pragma unroll 1
            for (int c32 = 0; c32 < XCOLS / 32; ++c32) {
              uint32_t regs[32];
              tmem_ld32(o_col + x0 + c32 * 32, regs);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float4 v = *slot4(c32 * 8 + c);
                regs[4 * c] = __float_as_uint(fmaf(v.x, f1, __uint_as_float(regs[4 * c]) * f0));
                regs[4 * c + 1] = __float_as_uint(fmaf(v.y, f1, __uint_as_float(regs[4 * c + 1]) * f0));
                regs[4 * c + 2] = __float_as_uint(fmaf(v.z, f1, __uint_as_float(regs[4 * c + 2]) * f0));
                regs[4 * c + 3] = __float_as_uint(fmaf(v.w, f1, __uint_as_float(regs[4 * c + 3]) * f0));
              }
              tmem_st32(o_col + x0 + c32 * 32, regs);
            }
            tmem_st_wait();
          }
        }
        meet();  // the exchange has been read: the next item's Q may go there
        has_rows = has_rows && blk == 0;
      }
      // ---- epilogue, a thread a row
      has_rows = has_rows && ok;
      const float inv_l = rs.l > 0.f ? 1.f / rs.l : 0.f;  // a row without keys gets 0
      if (!whole) {
        if (has_rows) {
          const int64_t prow = prow0 + (two ? blk * 128 : 0) + r;
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
            __syncwarp();
          }
        }
      } else if constexpr (MAPS == 1) {
        if (has_rows) {
          T* orow = static_cast<T*>(p.out) + (token * p.heads + qh) * p.row;
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
            __syncwarp();
          }
          if (valid && p.lse) {
            float lse = rs.l != 0.f ? rs.m * kLn2 + logf(rs.l) : -INFINITY;
            if (p.mask_type == 5) lse += p.slopes[qh] * static_cast<float>(rs.pos);  // left-aligned = right-aligned + slope * pos
            p.lse[token * p.heads + qh] = lse;
          }
        }
      } else {
        // the difference of the maps, in 16-column groups: of neighbouring lanes (even: map 1) where they are
        // neighbouring rows, the even lane finishing the first 16 columns of each 32 and the odd lane the others;
        // of the two blocks' rows, through the exchange, where a block is a map
        const int oh = qh >> 1;
        const float f = !valid ? 0.f : (qh & 1) ? -p.lambda[oh] * inv_l : inv_l;
        const bool odd = !two && (lane & 1);
        if (two) {
          if (blk == 1 && has_rows) {
#pragma unroll 1
            for (int c32 = 0; c32 < D / 32; ++c32) {
              uint32_t regs[32];
              tmem_ld32(o_col + c32 * 32, regs);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *slot4(c32 * 8 + c) = make_float4(__uint_as_float(regs[4 * c]) * f, __uint_as_float(regs[4 * c + 1]) * f,
                                                  __uint_as_float(regs[4 * c + 2]) * f, __uint_as_float(regs[4 * c + 3]) * f);
            }
          }
          meet();
        }
        if (has_rows && !(two && blk == 1)) {
          constexpr int kMost = 32;
          float y[kMost];
          // y: the columns of this thread from c32 * 32 (two blocks: all 32; else 16 of them)
          auto diff = [&](int c32) {
            uint32_t regs[32];
            tmem_ld32(o_col + c32 * 32, regs);
            tmem_ld_wait();
            if (two) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float4 v = *slot4(c32 * 8 + c);
                y[4 * c] = fmaf(__uint_as_float(regs[4 * c]), f, v.x);
                y[4 * c + 1] = fmaf(__uint_as_float(regs[4 * c + 1]), f, v.y);
                y[4 * c + 2] = fmaf(__uint_as_float(regs[4 * c + 2]), f, v.z);
                y[4 * c + 3] = fmaf(__uint_as_float(regs[4 * c + 3]), f, v.w);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float a = __uint_as_float(regs[i]) * f, b = __uint_as_float(regs[16 + i]) * f;
                y[i] = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
              }
            }
          };
          float post = p.out_scale;
          if (p.norm_weight) {
            float ss = 0.f;
#pragma unroll 1
            for (int c32 = 0; c32 < D / 32; ++c32) {
              if (c32 * 32 >= p.row) break;
              diff(c32);
#pragma unroll
              for (int i = 0; i < kMost; ++i) {
                const int col = c32 * 32 + (odd ? 16 : 0) + i;
                if ((two || i < 16) && col < p.row) ss = fmaf(y[i], y[i], ss);
              }
            }
            if (!two) ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            post *= inv_rms(p, ss);
          }
          T* orow = static_cast<T*>(p.out) + (token * (p.heads / 2) + oh) * p.row;
#pragma unroll 1
          for (int c32 = 0; c32 < D / 32; ++c32) {
            if (c32 * 32 >= p.row) break;
            diff(c32);
#pragma unroll
            for (int i16 = 0; i16 < 2; ++i16) {
              const int col = c32 * 32 + (odd ? 16 : i16 * 16);
              if (!valid || col >= p.row || (!two && i16 == 1)) continue;
              uint32_t o[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float a = y[i16 * 16 + 2 * i] * post, b = y[i16 * 16 + 2 * i + 1] * post;
                if (p.norm_weight) {
                  a *= __ldg(p.norm_weight + col + 2 * i);
                  b *= __ldg(p.norm_weight + col + 2 * i + 1);
                }
                o[i] = pack2(a, b, (T*)nullptr);
              }
              st_global_v8(orow + col, o);
            }
            __syncwarp();
          }
        }
        if (two) meet();  // the exchange has been read
      }
    } while (w.next(p));
    if (threadIdx.x == 0 && !owner) p.desc[blockIdx.x].n_seg = 0;
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------------------------- combine

// Joins the segments of the items that CTA boundaries cut, one warp per output row.  A grid of its own: the rows of
// a chunk are too many for the CTAs that cut them to do it on the side.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedParams p) {
  dependency_wait();
  const PagedDesc d = p.desc[blockIdx.x];
  if (d.n_seg == 0) return;
  const int gh = p.group / p.maps();
  for (int u = blockIdx.y * 8 + (threadIdx.x >> 5); u < d.tokens * gh; u += kCombineY * 8)
    combine_row<T, D>(p, d, blockIdx.x, u / gh, u % gh);
}

template <typename T, int D, int NQ, int MAPS>
cudaError_t launch_attn_maps(const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedParams& p, cudaStream_t stream) {
  using C = Cfg<T, D, NQ>;
  // at least 120 KB so a second CTA never shares the SM (each CTA allocates all 512 TMEM columns)
  constexpr int kSmem = C::SMEM > 120 * 1024 ? C::SMEM : 120 * 1024;
  cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<T, D, NQ, MAPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_attn_kernel<T, D, NQ, MAPS>, dim3(kGrid), C::THREADS, kSmem, stream, tmK, tmV, p);
}

template <typename T, int D, int NQ>
cudaError_t launch_attn(const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedParams& p, cudaStream_t stream) {
  return p.maps() == 1 ? launch_attn_maps<T, D, NQ, 1>(tmK, tmV, p, stream) : launch_attn_maps<T, D, NQ, 2>(tmK, tmV, p, stream);
}

template <typename T, int D>
cudaError_t launch(const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedParams& p, bool two, cudaStream_t stream) {
  cudaError_t e;
  if constexpr (D == 256) e = launch_attn<T, D, 1>(tmK, tmV, p, stream);
  else if constexpr (D == 64) e = launch_attn<T, D, 2>(tmK, tmV, p, stream);
  else e = two ? launch_attn<T, D, 2>(tmK, tmV, p, stream) : launch_attn<T, D, 1>(tmK, tmV, p, stream);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_combine_kernel<T, D>, dim3(kGrid, kCombineY), 256, 0, stream, p);
}

cudaError_t launch_any(int32_t dtype, int D, const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedParams& p, bool two,
                       cudaStream_t stream) {
  const bool f16 = dtype == kF16;
  if (D == 64) return f16 ? launch<__half, 64>(tmK, tmV, p, two, stream) : launch<__nv_bfloat16, 64>(tmK, tmV, p, two, stream);
  if (D == 128) return f16 ? launch<__half, 128>(tmK, tmV, p, two, stream) : launch<__nv_bfloat16, 128>(tmK, tmV, p, two, stream);
  return f16 ? launch<__half, 256>(tmK, tmV, p, two, stream) : launch<__nv_bfloat16, 256>(tmK, tmV, p, two, stream);
}

uint64_t align256(uint64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

int paged_kernel_d(int64_t row) {
  if (row <= 0 || row % 8 != 0 || row > 256) return 0;
  return row <= 64 ? 64 : row <= 128 ? 128 : 256;
}

void paged_layout(PagedPlan* plan) {
  const int D = paged_kernel_d(plan->row), rows = D == 256 ? 128 : 256;
  plan->off_desc = kPagedHeaderBytes;
  plan->off_ml = align256(plan->off_desc + sizeof(PagedDesc) * kGrid);
  plan->off_part = align256(plan->off_ml + sizeof(float2) * kGrid * 2 * rows);
  plan->ws_size = plan->off_part + (uint64_t)sizeof(float) * kGrid * 2 * rows * D;
}

int paged_run(PagedPlan* plan, void* workspace, cudaStream_t stream, char* err, size_t errlen) {
  cudaError_t e = cudaSuccess;
  if (workspace != plan->bound_ws) e = cudaMemsetAsync(workspace, 0, kPagedHeaderBytes, stream);
  if (e != cudaSuccess) {
    snprintf(err, errlen, "status clear failed: %s", cudaGetErrorString(e));
    return ALA_CUDA_ERROR;
  }
  if (plan->n_tokens == 0 || plan->batch == 0) return ALA_OK;  // no rows to write
  const int D = paged_kernel_d(plan->row);
  const int box = kv_box_rows(plan->block_size, D == 256 ? 64 : 128);
  if (!plan->maps_ready) {
    const int64_t rows = (int64_t)plan->num_blocks * plan->block_size;
    // L2 fetches whole lines of a kv head's row and no more: a line that reaches into the next head's row is gone
    // from L2 when its turn comes
    const int bytes = plan->row * 2, promote = bytes % 256 == 0 ? 256 : bytes % 128 == 0 ? 128 : 0;
    if (!encode_rows_heads_d(&plan->tmK, plan->k, plan->dtype, rows, plan->kv_heads, plan->row, box, false, promote) ||
        !encode_rows_heads_d(&plan->tmV, plan->v, plan->dtype, rows, plan->kv_heads, plan->row, box, true, promote)) {
      snprintf(err, errlen, "cuTensorMapEncodeTiled failed");
      return ALA_CUDA_ERROR;
    }
    plan->maps_ready = true;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
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
  p.arrived = reinterpret_cast<int*>(ws + 256);
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
  p.dq = plan->d;
  p.row = plan->row;
  p.tb1 = 128 / p.group;
  p.scale_log2 = plan->qk_scale * kLog2e;
  p.norm_eps = plan->norm_eps;
  p.out_scale = plan->out_scale;
  p.box_rows = box;
  p.rows_min = 0;
  p.rows_max = INT32_MAX;
  // Which kernels run follows from the rows (tokens x heads of a kv head) that a sequence has on average, since its
  // length is on the device; any lengths run on either.  What a step needs may differ: single tokens under a plan of 4096
  // tokens take 19, 34 and 102 us for 1, 8 and 64 requests of 1350 to 2200 keys, against 15, 23 and 88 under their own.
  // Up to one tile of the kernel for few rows, and 4 rows for the padding of a batch: that kernel alone.
  // Measured, it against the other: 16 x 1 token of 16000 keys 85 against 112 us, 32 rows 219 against 249; 40 rows,
  // its second tile reading the keys again, 393 against 259.  The 4 rows, in batches of 4, 8, 16 and 32 over 8000 keys: where
  // they are padding 41, 66, 90 and 164 us against 54, 79, 110 and 179; where they are tokens 47, 85, 127 and 297 against
  // 54, 81, 128 and 221.
  // More, in a batch of 16 or more, where there are likely to be sequences of both kinds: each on the kernel that
  // suits its own rows (36 decoding beside 4 chunks 411 -> 403 us).  In a smaller one a launch that finds nothing
  // costs more than that gives (4 chunks of 225 tokens 71 -> 77 us).
  const int64_t rows = plan->n_tokens * p.group;
  const bool can_few = p.group <= kFewRows, few = can_few && rows <= (int64_t)36 * p.batch;
  const bool both = !few && can_few && p.batch >= 16;
  if (few || both) {
    if (both) p.rows_max = kFewRows;
    p.tb = kFewRows / p.group;
    // The heads of a token lie side by side in the cache, so they run side by side, too: CTA c takes head c % kvHeadNum.
    // DRAM pages are then read once, and rows that end inside a line find it in L2.  Below 140 busy SMs that would
    // cost more than it gives.  Measured with 8 kv heads, rows of 160 bytes 690 -> 427 us, of 128 bytes 418 -> 330, of
    // 256 bytes 626 -> 617, 32 query rows of them 219 -> 196.
    const int parts = kGrid / p.kv_heads;
    p.head_stride = parts * p.kv_heads >= 140 ? p.kv_heads : 1;
    const int64_t most = (p.n_tokens / p.tb + (int64_t)p.batch) * ((int64_t)p.max_blocks * p.block_size / 128 + 1) * p.kv_heads;
    p.small = p.batch <= 64 && most < 1 << 24 && p.n_tokens < 1 << 24;
    e = launch_paged_few(plan->dtype, D, plan->tmK, plan->tmV, p, stream);
  }
  if (!few && e == cudaSuccess) {
    // Two blocks of rows where sequences have more than one block's on average (256 rows: 218 us against 226 with one,
    // long chunks 2290 against 2518); at D = 64 there is room for both Q blocks and deep rings anyway.
    const bool two = D == 64 || (D == 128 && rows > (int64_t)128 * p.batch);
    if (both) p.rows_min = kFewRows + 1;
    p.rows_max = INT32_MAX;
    p.tb = !two ? p.tb1 : p.maps() == 2 ? 128 / (p.group / 2) : 2 * p.tb1;
    p.head_stride = 1;
    e = launch_any(plan->dtype, D, plan->tmK, plan->tmV, p, two, stream);
  }
  if (e != cudaSuccess) {
    snprintf(err, errlen, "kernel launch failed: %s", cudaGetErrorString(e));
    return ALA_CUDA_ERROR;
  }
  return ALA_OK;
}

}  // namespace ala
