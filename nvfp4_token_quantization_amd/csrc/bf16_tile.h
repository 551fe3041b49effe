// bf16_tile.h -- the block tile of the bf16 products (gfx950): operands brought
// to LDS by DMA, fragments, the MFMA loop.  The products grouped by expert and
// the vocabulary loss differ in their schedules and in what they do with a tile.
#pragma once

#include <type_traits>
#include <utility>

#include "gemm_common.h"
#include "rowwise.h"

namespace nvfp4 {

enum { BG_FORWARD = 0, BG_DGRAD = 1, BG_WGRAD = 2 };

// ---------------------------------------------------------------------------
// The tile kernel.  Four waves share a block tile of 64 TM x 64 TN outputs; a
// wave holds TM x TN tiles of v_mfma_f32_32x32x16_bf16 and takes the 32-row
// slabs 2 i + wr, so that a ragged tile's empty slabs fall on both wave rows
// alike and are left out in pairs (VS <= TM pairs hold rows).
//
// A stage is BK = 32 or 64 elements of the summed dimension of both operands,
// brought to LDS by DMA (buffer_load ... lds, 1 KiB an instruction) into a
// ring of NB stage buffers: the DMA of stage s + NB goes out when every wave
// has read stage s, NB - 1 stages ahead of its use.  Two layouts:
//   row operands (X, dY and W of the forward product, dY of dgrad), whose
//     summed dimension is contiguous: LDS rows of BK elements, one per output
//     row or column, their 16-byte chunks XOR-swizzled by bg_row_swz, read 8
//     summed elements a lane with ds_read_b128.  BK = 64 takes whole 128-byte
//     lines (forward, 8192 cubed, 256 x 256: 840 us against 858 with 32);
//   column operands (W of dgrad, dY and X of wgrad), whose output dimension
//     is contiguous: BK LDS rows, one per summed index, read with
//     ds_read_b64_tr_b16, which hands each lane 4 summed elements of its
//     column.  Chunks are XOR-swizzled by row so that the four rows of 16
//     lanes (and of 32) lie in different banks.
// Row reads show no bank conflicts in the counters; with column reads they
// take 3% of the LDS cycles in dgrad (one column operand) and 13% in wgrad (two).
// Rows, columns and summed elements that do not exist get an offset past the
// resource, for which the DMA writes zeros.
constexpr uint32_t BG_OOB = 0x80000000u;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// chunk swizzle of a row operand's LDS row of BK elements (4 or 8 chunks)
template <int BK>
__device__ __forceinline__ int bg_row_swz(int r) {
  return BK == 64 ? (r >> 1) & 7 : ((r >> 2) + (r & 2)) & 3;
}
// chunk swizzle of a column operand's LDS row of 8 TN chunks
template <int TN>
__device__ __forceinline__ int bg_col_swz(int r) {
  return TN == 1 ? (r & 2) << 1 : ((r & 3) << 2) ^ (r & 2);
}

// The same for 16 x 16 x 32 fragments of 2 or more slabs, whose lanes 16 .. 31
// read rows 8 further on: those take the other 32 bytes of each 64.
__device__ __forceinline__ int bg_col_swz16(int r) { return ((r & 3) << 2) ^ ((r >> 2) & 2); }

template <int MODE> struct BgMode {
  static constexpr bool a_cols = MODE == BG_WGRAD;     // A is a column operand
  static constexpr bool b_cols = MODE != BG_FORWARD;   // B is a column operand
};

// One operand of a block tile, T slabs of 64 rows or columns.
template <int T>
struct BgOperand {
  i32x4 rsrc;
  const uint8_t* base;   // column operands: of summed index 0
  int64_t stride;        // column operands: bytes per summed index
  uint32_t voff[2 * T];  // this lane's byte offset for its DMA i
};

// Rows [row_lo, row_hi) of the layout (a wgrad's summed rows), the tile's
// first output column n0, wgrad's first output row m0 (a column of dY), and
// the length of the sum.
struct BgTile {
  int64_t row_lo, row_hi, m0, n0, K;
  int g;
};

__device__ __forceinline__ i32x4 bg_rsrc(const void* p, int64_t bytes) {
  i32x4 r = make_rsrc(p, bytes);
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_readfirstlane(r[i]);
  return r;
}

// Fragment of 32 rows or columns (slab `sl` of the operand) for summed
// elements [16 t + 8 h, +8) of the stage at `st`.
template <int BK>
__device__ __forceinline__ bf16x8 bg_frag_rows(const uint8_t* st, int sl, int t, int li, int h) {
  const int chunk = (2 * t + h) ^ bg_row_swz<BK>(li);
  return *reinterpret_cast<const bf16x8*>(st + sl * (64 * BK) + li * (2 * BK) + chunk * 16);
}
template <int T>
__device__ __forceinline__ bf16x8 bg_frag_cols(uint8_t* st, int sl, int t, int lane) {
  const int i = lane & 15, r4 = i >> 2;
  const int chunk = (4 * sl + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1)) ^ bg_col_swz<T>(r4);
  uint8_t* p = st + (16 * t + 8 * (lane >> 5) + r4) * (128 * T) + chunk * 16 + (i & 1) * 8;
  typedef __attribute__((address_space(3))) s16x4* lds4;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)p);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 4 * 128 * T));
  const s16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8, v);
}

// The same for v_mfma_f32_16x16x32_bf16: 16 rows or columns (half `sub` of slab
// `sl`), summed elements [32 t + 8 q, +8) for lane 16 q + i.
template <int BK>
__device__ __forceinline__ bf16x8 bg_frag16_rows(const uint8_t* st, int sl, int sub, int t, int lane) {
  const int i = lane & 15, chunk = (4 * t + (lane >> 4)) ^ bg_row_swz<BK>(i);
  return *reinterpret_cast<const bf16x8*>(st + sl * (64 * BK) + (16 * sub + i) * (2 * BK) + chunk * 16);
}
template <int T>
__device__ __forceinline__ bf16x8 bg_frag16_cols(uint8_t* st, int sl, int sub, int t, int lane) {
  const int i = lane & 15, r4 = i >> 2;
  const int row = 32 * t + 8 * (lane >> 4) + r4;
  const int chunk = (4 * sl + 2 * sub + ((i & 3) >> 1)) ^ bg_col_swz16(row);
  uint8_t* p = st + row * (128 * T) + chunk * 16 + (i & 1) * 8;
  typedef __attribute__((address_space(3))) s16x4* lds4;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)p);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 4 * 128 * T));
  const s16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8, v);
}

// f(0), f(1), .. f(N - 1) with constants: unrolled whatever the size of f
template <int... I, class F>
__device__ __forceinline__ void static_for_each(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_each(std::make_integer_sequence<int, N>(), f);
}

// MFMA shapes: 32 x 32 x 16 (F = 1) and 16 x 16 x 32 (F = 2 fragments a slab).
template <int SH> struct BgShape;
template <> struct BgShape<32> {
  typedef f32x16 acc;
  static constexpr int F = 1, KS = 16;
  static __device__ __forceinline__ acc mma(bf16x8 a, bf16x8 b, acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct BgShape<16> {
  typedef f32x4 acc;
  static constexpr int F = 2, KS = 32;
  static __device__ __forceinline__ acc mma(bf16x8 a, bf16x8 b, acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};

// Blocks of a tile shape that share a CU's 160 KiB, and the LDS each gets:
// the stage ring, and for a gathered wgrad each wave's ring of row indices.
template <int TM, int TN>
constexpr int bg_blocks() { return TM + TN > 6 ? 1 : (TM + TN > 2 ? 2 : 3); }
template <int MODE>
constexpr int bg_index_ring() { return MODE == BG_WGRAD ? 4 * 8 * 256 : 0; }
template <int TM, int TN>
constexpr int bg_lds() { return 160 * 1024 / bg_blocks<TM, TN>() / 1024 * 1024; }
// Stages of `bytes` the ring of one of KG wave groups holds: a tile with few
// rows keeps more of them in flight.
template <int MODE, int TM, int TN, int KG>
constexpr int bg_bufs(int bytes) {
  const int n = ((KG > 1 ? 160 * 1024 / KG : bg_lds<TM, TN>()) - bg_index_ring<MODE>()) / bytes;
  const int most = MODE == BG_WGRAD ? 4 : 6;
  return n < most ? n : most;
}

// The sums of a block tile: acc[i][j] holds rows 32 (2 i + wr) .. and columns
// 32 (TN wc + j) .. of the tile, wave w = 2 wr + wc of its group.  KG wave
// groups of four waves each sum their own range of `nst` stages, with a ring of
// their own, and the first adds the others' tiles in order: false for those
// others, which hold nothing.  On return every LDS byte from bg_sums() on is
// free.  p: the arguments' row_index and a_rows.
//
// Args with a member `blocks` hold A in blocks of 64 x 64 elements, 128 bytes a
// row, dz_row bytes from one to the next along its rows and dz_col along its
// columns: the offsets of oa.voff go from oa.base on, and both strides' steps are
// taken here.
template <class Args, class = void> constexpr bool bg_blocked = false;
template <class Args> constexpr bool bg_blocked<Args, std::void_t<decltype(Args::blocks)>> = true;
template <int VS, int TN, int KG>
constexpr int bg_sums() { return (KG - 1) * 4 * VS * TN * 16 * 64 * 4; }  // the other groups' accumulators
template <int MODE, int TM, int TN, int BK, int KG, int VS, int SH, class Args>
__device__ __forceinline__ bool bg_sum(const Args& p, const BgTile& tl, BgOperand<TM>& oa, BgOperand<TN>& ob,
                                       uint8_t* block_lds, int nst, int grp, int w, int lane,
                                       typename BgShape<SH>::acc (&acc)[BgShape<SH>::F * VS][BgShape<SH>::F * TN]) {
  constexpr int F = BgShape<SH>::F, FA = F * VS, FN = F * TN, READS = FA + FN;
  uint8_t* lds = block_lds + (KG > 1 ? grp * (160 * 1024 / KG) : 0);
  typedef BgMode<MODE> M;
  constexpr int TA = M::a_cols ? TM : VS;  // A slabs of a stage
  constexpr int NA = TA * BK / 32, NC = NA + TN * BK / 32;  // DMA instructions of this wave per stage
  constexpr int STAGE = NC * 4096;
  constexpr int NB = bg_bufs<MODE, TM, TN, KG>(STAGE);
  static_assert(NB >= 2, "a stage in use and one in flight");
  constexpr int AT = NA * 4096;  // the stage's B follows its A
  constexpr int NT = BK / BgShape<SH>::KS;  // MFMA steps of a stage
  const int li = lane & 31, h = lane >> 5, wr = w >> 1, wc = w & 1;
  const uint32_t lbase = (uint32_t)(uintptr_t)lds;
  const bool gather = MODE == BG_WGRAD && p.row_index != nullptr;
  // gathered wgrad: DMA of the row indices of stage s into this wave's ring
  const uint32_t ring = NB * STAGE + (uint32_t)w * 8 * 256;
  auto issue_index = [&](int s) {
    const int64_t left = min((int64_t)BK, max((int64_t)0, tl.K - (int64_t)s * BK));
    const i32x4 ri = bg_rsrc(p.row_index + tl.row_lo + (int64_t)s * BK, left * 4);
    dma4(ri, (uint32_t)lane * 4, 0, lbase + ring + (uint32_t)(s & 7) * 256);
  };
  // this lane's rows of its DMAs of B in a stage, from the ring
  constexpr int RPI = 8 / TN;  // summed rows an instruction covers
  auto gather_rows = [&](int s, int32_t (&idx)[NC - NA]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NC - NA; ++i) {
      const int r = (4 * i + w) * RPI + lane / (8 * TN);
      idx[i] = *reinterpret_cast<const int32_t*>(lds + ring + (s & 7) * 256 + r * 4);
    }
  };
  // What the DMAs of stage s share (a stage past the last has no summed
  // elements, so its DMAs write zeros), and DMA k of the stage.
  struct Issue {
    i32x4 ra, rb;
    uint32_t at, soff;
    bool in;  // row operands: this lane's chunk exists
    int s;
  };
  constexpr int CPR = BK / 8;  // chunks of a row operand's LDS row
  const int chunk8 = 8 * ((lane % CPR) ^ bg_row_swz<BK>(64 / CPR * w + lane / CPR));
  auto issue_at = [&](int s, int buf) __attribute__((always_inline)) {
    Issue q;
    q.s = s;
    q.at = lbase + (uint32_t)buf * STAGE + (uint32_t)w * 1024;
    q.soff = (uint32_t)s * (BK * 2);
    q.in = (int64_t)s * BK + chunk8 < tl.K;
    const int64_t left = min((int64_t)BK, max((int64_t)0, tl.K - (int64_t)s * BK));
    if constexpr (bg_blocked<Args>) {
      const int64_t first = (int64_t)s * BK;
      const uint8_t* at = M::a_cols ? oa.base + first / 64 * p.dz_row + first % 64 * 128 : oa.base + first / 64 * p.dz_col + first % 64 * 2;
      q.ra = bg_rsrc(at, left > 0 ? (TM - 1) * (M::a_cols ? p.dz_col : p.dz_row) + 8192 : 0);
    } else {
      q.ra = M::a_cols ? bg_rsrc(oa.base + (int64_t)s * BK * oa.stride, left * oa.stride) : oa.rsrc;
    }
    q.rb = M::b_cols && !gather ? bg_rsrc(ob.base + (int64_t)s * BK * ob.stride, left * ob.stride) : ob.rsrc;
    return q;
  };
  auto issue_one = [&](const Issue& q, const int32_t (&idx)[NC - NA], int k) __attribute__((always_inline)) {
    if (k < NA) {
      if constexpr (M::a_cols) dma16(q.ra, oa.voff[k], 0, q.at + k * 4096);
      else dma16(q.ra, q.in ? oa.voff[k] : BG_OOB, bg_blocked<Args> ? 0 : q.soff, q.at + k * 4096);
      return;
    }
    const int i = k - NA;
    const uint32_t at = q.at + AT + i * 4096;
    if constexpr (!M::b_cols) {
      dma16(q.rb, q.in ? ob.voff[i] : BG_OOB, q.soff, at);
    } else if (!gather) {
      dma16(q.rb, ob.voff[i], 0, at);
    } else {
      const int64_t r = (int64_t)q.s * BK + (4 * i + w) * RPI + lane / (8 * TN);
      const bool in = r < tl.K && idx[i] >= 0 && idx[i] < p.a_rows && ob.voff[i] != BG_OOB;
      dma16(q.rb, in ? (uint32_t)idx[i] * (uint32_t)ob.stride + ob.voff[i] : BG_OOB, 0, at);
    }
  };
  // fragment k (A slabs, then B slabs) of MFMA step t of the stage in buffer buf
  auto read_at = [&](uint8_t* st, uint8_t* sb, int t, bf16x8 (&fa)[FA], bf16x8 (&fb)[FN], int k) __attribute__((always_inline)) {
    if constexpr (SH == 32) {
      if (k < VS)
        fa[k] = M::a_cols ? bg_frag_cols<TM>(st, 2 * k + wr, t, lane) : bg_frag_rows<BK>(st, 2 * k + wr, t, li, h);
      else
        fb[k - VS] = M::b_cols ? bg_frag_cols<TN>(sb, TN * wc + k - VS, t, lane)
                               : bg_frag_rows<BK>(sb, TN * wc + k - VS, t, li, h);
    } else {
      if (k < FA) {
        const int sl = 2 * (k / F) + wr;
        fa[k] = M::a_cols ? bg_frag16_cols<TM>(st, sl, k % F, t, lane) : bg_frag16_rows<BK>(st, sl, k % F, t, lane);
      } else {
        const int sl = TN * wc + (k - FA) / F;
        fb[k - FA] = M::b_cols ? bg_frag16_cols<TN>(sb, sl, (k - FA) % F, t, lane)
                               : bg_frag16_rows<BK>(sb, sl, (k - FA) % F, t, lane);
      }
    }
  };
  auto read_one = [&](int buf, int t, bf16x8 (&fa)[FA], bf16x8 (&fb)[FN], int k) __attribute__((always_inline)) {
    uint8_t* st = lds + buf * STAGE;
    read_at(st, st + AT, t, fa, fb, k);
  };
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (typename BgShape<SH>::acc){0};
  // The MFMAs of one step with `items` other instructions spread among them,
  // pinned in this order: the matrix pipe never waits for a burst of LDS
  // reads or DMAs to issue.
  auto mma = [&](const bf16x8 (&fa)[FA], const bf16x8 (&fb)[FN], int items, auto&& item) {
    constexpr int S = FA * FN;
#pragma unroll
    for (int m = 0; m < S; ++m) {
      const int i = m / FN, j = m % FN;
      acc[i][j] = BgShape<SH>::mma(fa[i], fb[j], acc[i][j]);
#pragma unroll
      for (int k = m * items / S; k < (m + 1) * items / S; ++k) item(k);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // The same with the reads among the first three quarters of the MFMAs, so that
  // none is waited for at the step's end, B before A: row i of A is dead after
  // its MFMAs, so that the next step's A takes its registers over.
  auto mma_early = [&](const bf16x8 (&fa)[FA], const bf16x8 (&fb)[FN], auto&& read, auto dmas, auto&& dma) __attribute__((always_inline)) {
    constexpr int S = FA * FN, H = S * 3 / 4, DMAS = decltype(dmas)::value;
    static_for<S>([&](auto mc) __attribute__((always_inline)) {
      constexpr int m = decltype(mc)::value, i = m / FN, j = m % FN;
      acc[i][j] = BgShape<SH>::mma(fa[i], fb[j], acc[i][j]);
      if constexpr (m < H) {
        constexpr int k0 = m * READS / H, k1 = (m + 1) * READS / H;
        static_for<k1 - k0>([&](auto k) __attribute__((always_inline)) {
          constexpr int r = k0 + decltype(k)::value;
          read(r < FN ? FA + r : r - FN);
        });
      }
      constexpr int d0 = m * DMAS / S, d1 = (m + 1) * DMAS / S;
      static_for<d1 - d0>([&](auto k) __attribute__((always_inline)) { dma(d0 + decltype(k)::value); });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  int32_t idx[NC - NA] = {};
  if (gather) {
    for (int s = 0; s < NB; ++s) issue_index(s);
    wait_vmcnt<0>();
  }
  for (int s = 0; s < NB; ++s) {
    if (gather) gather_rows(s, idx);
    const Issue q = issue_at(s, s);
#pragma unroll
    for (int k = 0; k < NC; ++k) issue_one(q, idx, k);
    if (gather) issue_index(s + NB);
  }
  // Fragments are read LOOK MFMA steps ahead: two where a step has few MFMAs,
  // which would not cover the LDS latency.
  constexpr int LOOK = SH == 32 && VS <= 2 && NT == 4 ? 2 : 1, FB = 2 * LOOK;
  bf16x8 fa[FB][FA], fb[FB][FN];
  if (gather) wait_vmcnt<(NB - 1) * (NC + 1)>();
  else wait_vmcnt<(NB - 1) * NC>();
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int t = 0; t < LOOK; ++t)
#pragma unroll
    for (int k = 0; k < READS; ++k) read_one(0, t, fa[t], fb[t], k);
  int cur = 0;
  // 16 x 16 x 32, no gathered rows: stage s, whose first fragments are in set SET;
  // leaves those of the next stage in set SET + NT (of two).
  auto stage = [&](auto set, int s) __attribute__((always_inline)) {
    constexpr int SET = decltype(set)::value;
    const int nxt = cur + 1 == NB ? 0 : cur + 1;
#pragma unroll
    for (int t = 0; t < NT - 1; ++t)
      mma_early(fa[(SET + t) & 1], fb[(SET + t) & 1],
                [&](int k) __attribute__((always_inline)) { read_one(cur, t + 1, fa[(SET + t + 1) & 1], fb[(SET + t + 1) & 1], k); },
                std::integral_constant<int, 0>(), [](int) {});
    wait_lgkmcnt0();
    wait_vmcnt<(NB - 2) * NC>();
    asm volatile("s_barrier" ::: "memory");
    const Issue q = issue_at(s + NB, cur);
    mma_early(fa[(SET + NT - 1) & 1], fb[(SET + NT - 1) & 1],
              [&](int k) __attribute__((always_inline)) { read_one(nxt, 0, fa[(SET + NT) & 1], fb[(SET + NT) & 1], k); },
              std::integral_constant<int, NC>(), [&](int k) __attribute__((always_inline)) { issue_one(q, idx, k); });
    cur = nxt;
  };
  constexpr std::integral_constant<int, 0> s0{};
  if constexpr (SH == 16 && NT % 2 == 0) {
    for (int s = 0; s < nst; ++s) stage(s0, s);
  } else if constexpr (SH == 16) {  // the two sets change places from stage to stage
    constexpr std::integral_constant<int, 1> s1{};
    // an odd last stage is followed by one past the sum, which adds zeros
    for (int s = 0; s < nst; s += 2) {
      stage(s0, s);
      stage(s1, s + 1);
    }
  } else {
    for (int s = 0; s < nst; ++s) {
      const int nxt = cur + 1 == NB ? 0 : cur + 1;
      if (gather) gather_rows(s + NB, idx);
#pragma unroll
      for (int t = 0; t < NT - LOOK; ++t)
        mma(fa[t % FB], fb[t % FB], READS,
            [&](int k) { read_one(cur, t + LOOK, fa[(t + LOOK) % FB], fb[(t + LOOK) % FB], k); });
      // every read of stage s has landed and stage s + 1 is there: after the
      // barrier, for all four waves
      wait_lgkmcnt0();
      if (gather) wait_vmcnt<(NB - 2) * (NC + 1)>();
      else wait_vmcnt<(NB - 2) * NC>();
      asm volatile("s_barrier" ::: "memory");
      const Issue q = issue_at(s + NB, cur);
#pragma unroll
      for (int u = 0; u < LOOK; ++u) {
        const int t = NT - LOOK + u, d0 = NC * u / LOOK, d1 = NC * (u + 1) / LOOK;
        mma(fa[t % FB], fb[t % FB], READS + d1 - d0, [&](int k) {
          if (k < READS) read_one(nxt, u, fa[u], fb[u], k);
          else issue_one(q, idx, d0 + k - READS);
        });
      }
      if (gather) issue_index(s + 2 * NB);
      cur = nxt;
    }
  }
  wait_lgkmcnt0();
  wait_vmcnt<0>();
  asm volatile("s_barrier" ::: "memory");
  if constexpr (KG > 1) {
    static_assert(SH == 32, "only this shape's accumulators are laid out here");
    float* sums = reinterpret_cast<float*>(block_lds);
#pragma unroll
    for (int i = 0; i < VS; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (grp > 0) sums[((((grp - 1) * 4 + w) * VS * TN + i * TN + j) * 16 + r) * 64 + lane] = acc[i][j][r];
    __syncthreads();
    if (grp > 0) return false;
#pragma unroll
    for (int q = 0; q < KG - 1; ++q)
#pragma unroll
      for (int i = 0; i < VS; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            acc[i][j][r] += sums[(((q * 4 + w) * VS * TN + i * TN + j) * 16 + r) * 64 + lane];
  }
  return true;
}

}  // namespace nvfp4
