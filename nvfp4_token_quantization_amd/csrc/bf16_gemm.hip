// bf16_gemm.hip -- bf16 products grouped by expert, forward and both
// gradients, over the contiguous per-expert layout (gfx950).
//
//   forward  Y[i]  = X[r(i)] W_e^T      rows i of expert e, r(i) = row_index[i] or i
//   dgrad    dX[i] = dY[i] W_e
//   wgrad    dW_e  = add_e + sum_{i of e} dY[i]^T X[r(i)]
#include "gemm_common.h"
#include "rowwise.h"

namespace nvfp4 {

enum { BG_FORWARD = 0, BG_DGRAD = 1, BG_WGRAD = 2 };

struct Bf16Args {
  const uint16_t *a, *b;      // rows' operand (X or dY), weights or (wgrad) X
  int64_t a_rows;             // rows of the gathered operand
  const int32_t* row_index;
  const int32_t* offsets;
  int groups;
  int64_t m_total, n, k;      // weights are [groups, n, k]
  const void* add;
  void* y;
  bool y_bf;
  TileGrid t;
};

// ---------------------------------------------------------------------------
// The tile kernel.  Four waves share a block tile of 64 TM x 64 TN outputs; a
// wave holds TM x TN tiles of v_mfma_f32_32x32x16_bf16 and takes the 32-row
// slabs 2 i + wr, so that a ragged tile's empty slabs fall on both wave rows
// alike and are left out in pairs (VS <= TM pairs hold rows).
//
// A stage is 32 elements of the summed dimension of both operands, brought
// to LDS by DMA (buffer_load ... lds, 1 KiB an instruction) into a ring of
// four stage buffers: the DMA of stage s + 4 goes out when every wave has
// read stage s, three stages ahead of its use.  Two layouts:
//   row operands (X, dY and W of the forward product, dY of dgrad), whose
//     summed dimension is contiguous: LDS rows of 64 bytes, one per output
//     row or column, their 16-byte chunks XOR-swizzled by lds_swz, read 8
//     summed elements a lane with ds_read_b128;
//   column operands (W of dgrad, dY and X of wgrad), whose output dimension
//     is contiguous: 32 LDS rows, one per summed index, read with
//     ds_read_b64_tr_b16, which hands each lane 4 summed elements of its
//     column.  Chunks are XOR-swizzled by row so that the four rows of 16
//     lanes (and of 32) lie in different banks.
// Rows, columns and summed elements that do not exist get an offset past the
// resource, for which the DMA writes zeros.
constexpr int BG_BK = 32;
constexpr int BG_BUFS = 4;
constexpr uint32_t BG_OOB = 0x80000000u;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int bg_row_swz(int r) { return ((r >> 2) + (r & 2)) & 3; }
// chunk swizzle of a column operand's LDS row of 8 TN chunks
template <int TN>
__device__ __forceinline__ int bg_col_swz(int r) {
  return TN == 1 ? (r & 2) << 1 : ((r & 3) << 2) ^ (r & 2);
}

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
  uint32_t voff[T];      // this lane's byte offset for its DMA i
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
template <int T>
__device__ __forceinline__ bf16x8 bg_frag_rows(const uint8_t* st, int sl, int t, int li, int h) {
  const int chunk = (2 * t + h) ^ bg_row_swz(li & 15);
  return *reinterpret_cast<const bf16x8*>(st + sl * 2048 + li * 64 + chunk * 16);
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

template <int MODE, int TM, int TN>
constexpr int bg_stage() { return (TM + TN) * 4096; }
// LDS of a block: the stage ring, and for a gathered wgrad each wave's ring
// of the row indices of 8 stages
template <int MODE, int TM, int TN>
constexpr int bg_lds() { return BG_BUFS * bg_stage<MODE, TM, TN>() + (MODE == BG_WGRAD ? 4 * 8 * 256 : 0); }

template <int MODE, int TM, int TN, int VS>
__device__ __forceinline__ void bg_body(const Bf16Args& p, const BgTile& tl, BgOperand<TM>& oa, BgOperand<TN>& ob,
                                        uint8_t* lds, int w, int lane) {
  typedef BgMode<MODE> M;
  constexpr int STAGE = bg_stage<MODE, TM, TN>();
  constexpr int AT = TM * 4096;  // the stage's B follows its A
  constexpr int NA = M::a_cols ? TM : VS;
  const int li = lane & 31, h = lane >> 5, wr = w >> 1, wc = w & 1;
  const uint32_t lbase = (uint32_t)(uintptr_t)lds;
  const bool gather = MODE == BG_WGRAD && p.row_index != nullptr;
  const int nst = (int)((tl.K + BG_BK - 1) / BG_BK);
  // gathered wgrad: DMA of the row indices of stage s into this wave's ring
  const uint32_t ring = BG_BUFS * STAGE + (uint32_t)w * 8 * 256;
  auto issue_index = [&](int s) {
    const int64_t left = min((int64_t)BG_BK, max((int64_t)0, tl.K - (int64_t)s * BG_BK));
    const i32x4 ri = bg_rsrc(p.row_index + tl.row_lo + (int64_t)s * BG_BK, left * 4);
    dma4(ri, (uint32_t)lane * 4, 0, lbase + ring + (uint32_t)(s & 7) * 256);
  };
  // this lane's rows of its DMAs of B in a stage, from the ring
  constexpr int RPI = 8 / TN;  // summed rows an instruction covers
  auto gather_rows = [&](int s, int32_t (&idx)[TN]) {
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      const int r = (4 * i + w) * RPI + lane / (8 * TN);
      idx[i] = *reinterpret_cast<const int32_t*>(lds + ring + (s & 7) * 256 + r * 4);
    }
  };
  // What the DMAs of stage s share (a stage past the last has no summed
  // elements, so its DMAs write zeros), and DMA k of the stage.
  constexpr int NC = NA + TN;  // DMA instructions of this wave per stage
  struct Issue {
    i32x4 ra, rb;
    uint32_t at, soff;
    bool in;  // row operands: this lane's chunk exists
    int s;
  };
  const int chunk8 = 8 * ((lane & 3) ^ bg_row_swz(lane >> 2));
  auto issue_at = [&](int s) {
    Issue q;
    q.s = s;
    q.at = lbase + (uint32_t)(s & (BG_BUFS - 1)) * STAGE + (uint32_t)w * 1024;
    q.soff = (uint32_t)s * (BG_BK * 2);
    q.in = (int64_t)s * BG_BK + chunk8 < tl.K;
    const int64_t left = min((int64_t)BG_BK, max((int64_t)0, tl.K - (int64_t)s * BG_BK));
    q.ra = M::a_cols ? bg_rsrc(oa.base + (int64_t)s * BG_BK * oa.stride, left * oa.stride) : oa.rsrc;
    q.rb = M::b_cols && !gather ? bg_rsrc(ob.base + (int64_t)s * BG_BK * ob.stride, left * ob.stride) : ob.rsrc;
    return q;
  };
  auto issue_one = [&](const Issue& q, const int32_t (&idx)[TN], int k) {
    if (k < NA) {
      if constexpr (M::a_cols) dma16(q.ra, oa.voff[k], 0, q.at + k * 4096);
      else dma16(q.ra, q.in ? oa.voff[k] : BG_OOB, q.soff, q.at + k * 4096);
      return;
    }
    const int i = k - NA;
    const uint32_t at = q.at + AT + i * 4096;
    if constexpr (!M::b_cols) {
      dma16(q.rb, q.in ? ob.voff[i] : BG_OOB, q.soff, at);
    } else if (!gather) {
      dma16(q.rb, ob.voff[i], 0, at);
    } else {
      const int64_t r = (int64_t)q.s * BG_BK + (4 * i + w) * RPI + lane / (8 * TN);
      const bool in = r < tl.K && idx[i] >= 0 && idx[i] < p.a_rows && ob.voff[i] != BG_OOB;
      dma16(q.rb, in ? (uint32_t)idx[i] * (uint32_t)ob.stride + ob.voff[i] : BG_OOB, 0, at);
    }
  };
  // fragment k (A slabs, then B slabs) of half t of stage s
  auto read_one = [&](int s, int t, bf16x8 (&fa)[VS], bf16x8 (&fb)[TN], int k) {
    uint8_t* st = lds + (s & (BG_BUFS - 1)) * STAGE;
    if (k < VS)
      fa[k] = M::a_cols ? bg_frag_cols<TM>(st, 2 * k + wr, t, lane) : bg_frag_rows<TM>(st, 2 * k + wr, t, li, h);
    else
      fb[k - VS] = M::b_cols ? bg_frag_cols<TN>(st + AT, TN * wc + k - VS, t, lane)
                             : bg_frag_rows<TN>(st + AT, TN * wc + k - VS, t, li, h);
  };
  f32x16 acc[VS][TN];
#pragma unroll
  for (int i = 0; i < VS; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = (f32x16){0};
  // The MFMAs of one half stage with `items` other instructions spread among
  // them, pinned in this order: the matrix pipe never waits for a burst of
  // LDS reads or DMAs to issue.
  auto mma = [&](const bf16x8 (&fa)[VS], const bf16x8 (&fb)[TN], int items, auto&& item) {
    constexpr int S = VS * TN;
#pragma unroll
    for (int m = 0; m < S; ++m) {
      const int i = m / TN, j = m % TN;
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int k = m * items / S; k < (m + 1) * items / S; ++k) item(k);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  int32_t idx[TN] = {};
  if (gather) {
    for (int s = 0; s < 4; ++s) issue_index(s);
    wait_vmcnt<0>();
  }
  for (int s = 0; s < BG_BUFS; ++s) {
    if (gather) gather_rows(s, idx);
    const Issue q = issue_at(s);
#pragma unroll
    for (int k = 0; k < NC; ++k) issue_one(q, idx, k);
    if (gather) issue_index(s + 4);
  }
  bf16x8 fa[2][VS], fb[2][TN];
  if (gather) wait_vmcnt<3 * (NC + 1)>();
  else wait_vmcnt<3 * NC>();
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int k = 0; k < VS + TN; ++k) read_one(0, 0, fa[0], fb[0], k);
  for (int s = 0; s < nst; ++s) {
    if (gather) gather_rows(s + 4, idx);
    mma(fa[0], fb[0], VS + TN, [&](int k) { read_one(s, 1, fa[1], fb[1], k); });
    // every read of stage s has landed and stage s + 1 is there: after the
    // barrier, for all four waves
    wait_lgkmcnt0();
    if (gather) wait_vmcnt<2 * (NC + 1)>();
    else wait_vmcnt<2 * NC>();
    asm volatile("s_barrier" ::: "memory");
    const Issue q = issue_at(s + 4);
    mma(fa[1], fb[1], VS + TN + NC, [&](int k) {
      if (k < VS + TN) read_one(s + 1, 0, fa[0], fb[0], k);
      else issue_one(q, idx, k - VS - TN);
    });
    if (gather) issue_index(s + 8);
  }
  wait_lgkmcnt0();
  wait_vmcnt<0>();
  asm volatile("s_barrier" ::: "memory");

  // Epilogue through LDS, slab by slab, in a region of this wave's own: 16
  // bytes a lane and whole row segments per store instruction.
  constexpr int RS = 128 * TN + 32;  // bytes of an LDS row (the pad parts the lane halves' banks)
  static_assert(4 * 32 * RS <= bg_lds<MODE, TM, TN>(), "epilogue fits the ring");
  float* t = reinterpret_cast<float*>(lds + w * 32 * RS);
  const int64_t N = MODE == BG_FORWARD ? p.n : p.k;
  const int es = p.y_bf ? 2 : 4;
  const int64_t out_row = MODE == BG_WGRAD ? (int64_t)tl.g * p.n + tl.m0 : tl.row_lo;  // of the tile's first row
  const int64_t rows = MODE == BG_WGRAD ? min((int64_t)64 * TM, p.n - tl.m0) : tl.row_hi - tl.row_lo;
  const int64_t col0 = tl.n0 + 32 * TN * wc;
  uint8_t* yb = static_cast<uint8_t*>(p.y) + out_row * N * es;
  const uint32_t nb = (uint32_t)N * es;
  const __amdgpu_buffer_rsrc_t ry = out_rsrc(reinterpret_cast<float*>(yb), rows * N * es);
  const __amdgpu_buffer_rsrc_t radd =
      out_rsrc(reinterpret_cast<float*>(const_cast<uint8_t*>(static_cast<const uint8_t*>(p.add)) + (p.add ? out_row * N * es : 0)),
               p.add ? rows * N * es : 0);
#pragma unroll
  for (int i = 0; i < VS; ++i) {
    const int r0 = 32 * (2 * i + wr);
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        t[((8 * (r >> 2) + 4 * h + (r & 3)) * RS + (32 * j + li) * 4) / 4] = acc[i][j][r];
    wave_lds_sync();
    if (p.y_bf) {
      constexpr int LPR = 4 * TN;  // lanes a row, 8 columns each
      const int64_t col = col0 + 8 * (lane % LPR);
#pragma unroll
      for (int u = 0; u < 32 * LPR / 64; ++u) {
        const int r = u * (64 / LPR) + lane / LPR;
        const f32x4* q = reinterpret_cast<const f32x4*>(reinterpret_cast<const uint8_t*>(t) + r * RS + (lane % LPR) * 32);
        f32x4 a = q[0], b = q[1];
        const uint32_t off = col < N ? (uint32_t)(r0 + r) * nb + (uint32_t)col * 2 : BG_OOB;
        if (MODE == BG_WGRAD && p.add) {
          const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(radd, off, 0, 0);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            a[2 * c] += __uint_as_float(v[c] << 16);
            a[2 * c + 1] += __uint_as_float(v[c] & 0xFFFF0000u);
            b[2 * c] += __uint_as_float(v[2 + c] << 16);
            b[2 * c + 1] += __uint_as_float(v[2 + c] & 0xFFFF0000u);
          }
        }
        const u32x4 o = {pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3])};
        __builtin_amdgcn_raw_buffer_store_b128(o, ry, off, 0, 2);
      }
    } else {
      constexpr int LPR = 8 * TN;  // lanes a row, 4 columns each
      const int64_t col = col0 + 4 * (lane % LPR);
#pragma unroll
      for (int u = 0; u < 32 * LPR / 64; ++u) {
        const int r = u * (64 / LPR) + lane / LPR;
        f32x4 a = *reinterpret_cast<const f32x4*>(reinterpret_cast<const uint8_t*>(t) + r * RS + (lane % LPR) * 16);
        const uint32_t off = col < N ? (uint32_t)(r0 + r) * nb + (uint32_t)col * 4 : BG_OOB;
        if (MODE == BG_WGRAD && p.add) a += __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(radd, off, 0, 0));
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, a), ry, off, 0, 2);
      }
    }
    wave_lds_sync();
  }
}

template <int MODE, int TM, int TN>
__global__ __launch_bounds__(256) void bf16_tile_kernel(Bf16Args p) {
  typedef BgMode<MODE> M;
  constexpr int BM = 64 * TM, BN = 64 * TN;
  __shared__ __attribute__((aligned(16))) uint8_t lds[bg_lds<MODE, TM, TN>()];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  BgTile tl;
  BgOperand<TM> oa;
  BgOperand<TN> ob;
  int vs;
  if constexpr (MODE == BG_WGRAD) {
    // tiles of an expert one after another, its X columns fastest
    const int tn = (int)((p.n + BM - 1) / BM), tk = (int)((p.k + BN - 1) / BN);
    const int g = (int)(blockIdx.x / (unsigned)(tn * tk)), r = (int)(blockIdx.x % (unsigned)(tn * tk));
    const int64_t mt = p.m_total;
    const int64_t lo = min((int64_t)max(p.offsets[g], 0), mt), hi = min(max((int64_t)p.offsets[g + 1], lo), mt);
    tl.g = g;
    tl.row_lo = lo;
    tl.row_hi = hi;
    tl.K = hi - lo;
    tl.m0 = (int64_t)(r / tk) * BM;      // column of dY
    tl.n0 = (int64_t)(r % tk) * BN;  // column of X
    vs = (int)min((int64_t)TM, (p.n - tl.m0 + 63) / 64);
    // column operands: DMA i covers the summed rows (4 i + w) (8 / T) ..
    oa.stride = p.n * 2;
    oa.base = reinterpret_cast<const uint8_t*>(p.a + lo * p.n + tl.m0);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int row = (4 * i + w) * (8 / TM) + lane / (8 * TM);
      const int c = 8 * ((lane % (8 * TM)) ^ bg_col_swz<TM>(row));
      oa.voff[i] = tl.m0 + c < p.n ? (uint32_t)(row * oa.stride) + 2 * c : BG_OOB;
    }
    ob.stride = p.k * 2;
    ob.base = reinterpret_cast<const uint8_t*>(p.b + (p.row_index ? 0 : lo * p.k) + tl.n0);
    if (p.row_index) ob.rsrc = bg_rsrc(p.b, p.a_rows * p.k * 2);
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      const int row = (4 * i + w) * (8 / TN) + lane / (8 * TN);
      const int c = 8 * ((lane % (8 * TN)) ^ bg_col_swz<TN>(row));
      const uint32_t at = p.row_index ? (uint32_t)(tl.n0 * 2) : (uint32_t)(row * ob.stride);
      ob.voff[i] = tl.n0 + c < p.k ? at + 2 * c : BG_OOB;
    }
  } else {
    TileRange tr;
    static_assert(SCHED_LDS_WORDS * 4 <= bg_lds<MODE, TM, TN>(), "tile schedule fits");
    if (!schedule_tile<BM, BN>(p.t, lane, reinterpret_cast<int32_t*>(lds), tr)) return;  // block-uniform
    __syncthreads();  // the schedule's LDS words have been read
    tl.row_lo = tr.row_lo;
    tl.row_hi = tr.row_hi;
    tl.n0 = tr.n0;
    tl.g = tr.g;
    tl.K = MODE == BG_FORWARD ? p.k : p.n;
    vs = (int)((tl.row_hi - tl.row_lo + 63) / 64);
    // A: row operand, DMA i covers the tile's rows 16 (4 i + w) ..
    const uint32_t rowb = (uint32_t)tl.K * 2;
    const int swz = 16 * ((lane & 3) ^ bg_row_swz(lane >> 2));
    if (p.row_index) oa.rsrc = bg_rsrc(p.a, p.a_rows * (int64_t)rowb);
    else oa.rsrc = bg_rsrc(p.a + tl.row_lo * tl.K, (tl.row_hi - tl.row_lo) * (int64_t)rowb);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int64_t row = tl.row_lo + 16 * (4 * i + w) + (lane >> 2);
      int64_t src = gathered_row(p.row_index, p.a_rows, row, tl.row_hi);
      if (!p.row_index && src >= 0) src -= tl.row_lo;
      oa.voff[i] = src >= 0 ? (uint32_t)src * rowb + swz : BG_OOB;
    }
    if constexpr (M::b_cols) {
      ob.stride = p.k * 2;
      ob.base = reinterpret_cast<const uint8_t*>(p.b + (int64_t)tl.g * p.n * p.k + tl.n0);
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        const int row = (4 * i + w) * (8 / TN) + lane / (8 * TN);
        const int c = 8 * ((lane % (8 * TN)) ^ bg_col_swz<TN>(row));
        ob.voff[i] = tl.n0 + c < p.k ? (uint32_t)(row * ob.stride) + 2 * c : BG_OOB;
      }
    } else {
      const int64_t cols = min((int64_t)BN, p.n - tl.n0);
      ob.rsrc = bg_rsrc(p.b + ((int64_t)tl.g * p.n + tl.n0) * p.k, cols * p.k * 2);
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        const int c = 16 * (4 * i + w) + (lane >> 2);
        ob.voff[i] = c < cols ? (uint32_t)c * rowb + swz : BG_OOB;
      }
    }
  }
  if constexpr (TM == 4) {
    switch (vs) {
      case 4: bg_body<MODE, TM, TN, 4>(p, tl, oa, ob, lds, w, lane); break;
      case 3: bg_body<MODE, TM, TN, 3>(p, tl, oa, ob, lds, w, lane); break;
      case 2: bg_body<MODE, TM, TN, 2>(p, tl, oa, ob, lds, w, lane); break;
      default: bg_body<MODE, TM, TN, 1>(p, tl, oa, ob, lds, w, lane); break;
    }
  } else if constexpr (TM == 2) {
    if (vs == 2) bg_body<MODE, TM, TN, 2>(p, tl, oa, ob, lds, w, lane);
    else bg_body<MODE, TM, TN, 1>(p, tl, oa, ob, lds, w, lane);
  } else {
    bg_body<MODE, TM, TN, 1>(p, tl, oa, ob, lds, w, lane);
  }
}

template <int MODE, int TM, int TN>
static void launch_tiles(const Bf16Args& a, hipStream_t str) {
  Bf16Args p = a;
  int64_t blocks;
  if (MODE == BG_WGRAD) {
    blocks = (int64_t)p.groups * ((p.n + 64 * TM - 1) / (64 * TM)) * ((p.k + 64 * TN - 1) / (64 * TN));
  } else {
    p.t.m_total = p.m_total;
    p.t.offsets = p.offsets;
    p.t.groups = p.groups;
    blocks = plan_tiles<64 * TM, 64 * TN>(p.t, MODE == BG_FORWARD ? p.n : p.k, true, 1, p.row_index != nullptr);
  }
  hipLaunchKernelGGL((bf16_tile_kernel<MODE, TM, TN>), dim3((unsigned)blocks), dim3(256), 0, str, p);
}

template <int MODE>
static int launch_bf16(const Bf16Args& p, hipStream_t str) {
  launch_tiles<MODE, 4, 4>(p, str);
  return nvfp4host::launch_status();
}

}  // namespace nvfp4

using nvfp4host::aligned;

// What the three products refuse alike; `gathered`: bytes of an operand read through row_index.
static int bf16_check(int64_t groups, int64_t m_total, int64_t a_rows, int64_t n, int64_t k, const int32_t* offsets,
                      const int32_t* row_index, int64_t gathered_bytes, int y_type) {
  if (groups < 1 || m_total < 0 || a_rows < 0 || n < 0 || k < 0) return NVFP4_ERROR_INVALID_VALUE;
  if (y_type != NVFP4_TYPE_F32 && y_type != NVFP4_TYPE_BF16) return NVFP4_ERROR_INVALID_VALUE;
  if (n % 8 != 0 || k % 8 != 0 || groups > nvfp4::MAX_GROUPS) return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  const int64_t lim = (int64_t)1 << 31;
  if (m_total >= lim || a_rows >= lim || n > ((int64_t)1 << 20) || k > ((int64_t)1 << 20)) return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  if (row_index && gathered_bytes >= lim) return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  if (!offsets) return NVFP4_ERROR_INVALID_VALUE;
  if (!row_index && a_rows < m_total) return NVFP4_ERROR_INVALID_VALUE;
  if (!aligned(offsets, 4) || !aligned(row_index, 4)) return NVFP4_ERROR_MISALIGNED;
  return NVFP4_SUCCESS;
}

extern "C" int nvfp4_bf16_grouped_gemm(const uint16_t* x, int64_t a_rows, const int32_t* row_index, int64_t m_total,
                                       const int32_t* offsets, int64_t groups, const uint16_t* w, int64_t n, int64_t k,
                                       void* y, int y_type, void* stream) {
  int st = bf16_check(groups, m_total, a_rows, n, k, offsets, row_index, a_rows * k * 2, y_type);
  if (st) return st;
  if (m_total == 0 || n == 0) return NVFP4_SUCCESS;
  if (!y || (k > 0 && (!w || (a_rows > 0 && !x)))) return NVFP4_ERROR_INVALID_VALUE;
  if (!nvfp4::tile_grid_ok(m_total, groups, n)) return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16)) return NVFP4_ERROR_MISALIGNED;
  if ((st = nvfp4host::check_arch())) return st;
#if NVFP4_CHECKED
  {
    nvfp4check::Checks chk((hipStream_t)stream);
    chk.offsets(offsets, groups);
    if ((st = chk.result())) return st;
  }
#endif
  nvfp4::Bf16Args p{};
  p.a = x; p.b = w; p.a_rows = a_rows; p.row_index = row_index; p.offsets = offsets; p.groups = (int)groups;
  p.m_total = m_total; p.n = n; p.k = k; p.y = y; p.y_bf = y_type == NVFP4_TYPE_BF16;
  return nvfp4::launch_bf16<nvfp4::BG_FORWARD>(p, (hipStream_t)stream);
}

extern "C" int nvfp4_bf16_grouped_dgrad(const uint16_t* dy, int64_t m_total, const int32_t* offsets, int64_t groups,
                                        const uint16_t* w, int64_t n, int64_t k, void* dx, int dx_type, void* stream) {
  int st = bf16_check(groups, m_total, m_total, n, k, offsets, nullptr, 0, dx_type);
  if (st) return st;
  if (m_total == 0 || k == 0) return NVFP4_SUCCESS;
  if (!dx || (n > 0 && (!w || !dy))) return NVFP4_ERROR_INVALID_VALUE;
  if (!nvfp4::tile_grid_ok(m_total, groups, k)) return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  if (!aligned(dy, 16) || !aligned(w, 16) || !aligned(dx, 16)) return NVFP4_ERROR_MISALIGNED;
  if ((st = nvfp4host::check_arch())) return st;
#if NVFP4_CHECKED
  {
    nvfp4check::Checks chk((hipStream_t)stream);
    chk.offsets(offsets, groups);
    if ((st = chk.result())) return st;
  }
#endif
  nvfp4::Bf16Args p{};
  p.a = dy; p.b = w; p.a_rows = m_total; p.offsets = offsets; p.groups = (int)groups;
  p.m_total = m_total; p.n = n; p.k = k; p.y = dx; p.y_bf = dx_type == NVFP4_TYPE_BF16;
  return nvfp4::launch_bf16<nvfp4::BG_DGRAD>(p, (hipStream_t)stream);
}

extern "C" int nvfp4_bf16_grouped_wgrad(const uint16_t* dy, int64_t m_total, const uint16_t* x, int64_t a_rows,
                                        const int32_t* row_index, const int32_t* offsets, int64_t groups, int64_t n,
                                        int64_t k, const void* add, void* dw, int dw_type, void* stream) {
  int st = bf16_check(groups, m_total, a_rows, n, k, offsets, row_index, a_rows * k * 2, dw_type);
  if (st) return st;
  if (n == 0 || k == 0) return NVFP4_SUCCESS;
  if (!dw || (m_total > 0 && (!dy || (a_rows > 0 && !x)))) return NVFP4_ERROR_INVALID_VALUE;
  if (!nvfp4::tile_grid_ok(groups * n, 0, k)) return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dw, 16) || !aligned(add, 16)) return NVFP4_ERROR_MISALIGNED;
  if ((st = nvfp4host::check_arch())) return st;
#if NVFP4_CHECKED
  {
    nvfp4check::Checks chk((hipStream_t)stream);
    chk.offsets(offsets, groups);
    if ((st = chk.result())) return st;
  }
#endif
  nvfp4::Bf16Args p{};
  p.a = dy; p.b = x; p.a_rows = a_rows; p.row_index = row_index; p.offsets = offsets; p.groups = (int)groups;
  p.m_total = m_total; p.n = n; p.k = k; p.add = add; p.y = dw; p.y_bf = dw_type == NVFP4_TYPE_BF16;
  return nvfp4::launch_bf16<nvfp4::BG_WGRAD>(p, (hipStream_t)stream);
}
