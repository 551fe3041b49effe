// bf16_gemm.hip -- bf16 products grouped by expert, forward and both
// gradients, over the contiguous per-expert layout (gfx950).
//
//   forward  Y[i]  = X[r(i)] W_e^T      rows i of expert e, r(i) = row_index[i] or i
//   dgrad    dX[i] = dY[i] W_e
//   wgrad    dW_e  = add_e + sum_{i of e} dY[i]^T X[r(i)]
//
// bf16 products are exact in fp32 and summed there by the MFMAs; an output is
// rounded once.  One expert of 8192 rows, n = k = 8192 (bf16 output): forward
// 1298 TFLOP/s, dgrad 1196, wgrad 1190, where a large library product
// reaches 1377.  Ragged layouts are bound by what they move through HBM, panels
// read more than once among it, and by padding to 64-row slabs: 32768 rows over
// 128 Zipf experts, n = 1536, k = 2048, fp32 output: forward 295 to 314 us (682
// TFLOP/s at 302; reads 1.32 GB where 0.78 GB are the operands), wgrad 441 to
// 458 us (reads 0.95 GB for 0.12 GB and writes 1.61 GB).
#include <type_traits>

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
};

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

// KG wave groups of four waves each sum their own range of `nst` stages, with a
// ring of their own, and the first adds the others' tiles in order.
template <int MODE, int TM, int TN, int BK, int KG, int VS>
__device__ __forceinline__ void bg_body(const Bf16Args& p, const BgTile& tl, BgOperand<TM>& oa, BgOperand<TN>& ob,
                                        uint8_t* block_lds, int nst, int grp, int w, int lane) {
  uint8_t* lds = block_lds + (KG > 1 ? grp * (160 * 1024 / KG) : 0);
  typedef BgMode<MODE> M;
  constexpr int TA = M::a_cols ? TM : VS;  // A slabs of a stage
  constexpr int NA = TA * BK / 32, NC = NA + TN * BK / 32;  // DMA instructions of this wave per stage
  constexpr int STAGE = NC * 4096;
  constexpr int NB = bg_bufs<MODE, TM, TN, KG>(STAGE);
  static_assert(NB >= 2, "a stage in use and one in flight");
  constexpr int AT = NA * 4096;  // the stage's B follows its A
  constexpr int NT = BK / 16;    // MFMA steps of a stage
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
  auto gather_rows = [&](int s, int32_t (&idx)[NC - NA]) {
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
  auto issue_at = [&](int s, int buf) {
    Issue q;
    q.s = s;
    q.at = lbase + (uint32_t)buf * STAGE + (uint32_t)w * 1024;
    q.soff = (uint32_t)s * (BK * 2);
    q.in = (int64_t)s * BK + chunk8 < tl.K;
    const int64_t left = min((int64_t)BK, max((int64_t)0, tl.K - (int64_t)s * BK));
    q.ra = M::a_cols ? bg_rsrc(oa.base + (int64_t)s * BK * oa.stride, left * oa.stride) : oa.rsrc;
    q.rb = M::b_cols && !gather ? bg_rsrc(ob.base + (int64_t)s * BK * ob.stride, left * ob.stride) : ob.rsrc;
    return q;
  };
  auto issue_one = [&](const Issue& q, const int32_t (&idx)[NC - NA], int k) {
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
      const int64_t r = (int64_t)q.s * BK + (4 * i + w) * RPI + lane / (8 * TN);
      const bool in = r < tl.K && idx[i] >= 0 && idx[i] < p.a_rows && ob.voff[i] != BG_OOB;
      dma16(q.rb, in ? (uint32_t)idx[i] * (uint32_t)ob.stride + ob.voff[i] : BG_OOB, 0, at);
    }
  };
  // fragment k (A slabs, then B slabs) of MFMA step t of the stage in buffer buf
  auto read_one = [&](int buf, int t, bf16x8 (&fa)[VS], bf16x8 (&fb)[TN], int k) {
    uint8_t* st = lds + buf * STAGE;
    if (k < VS)
      fa[k] = M::a_cols ? bg_frag_cols<TM>(st, 2 * k + wr, t, lane) : bg_frag_rows<BK>(st, 2 * k + wr, t, li, h);
    else
      fb[k - VS] = M::b_cols ? bg_frag_cols<TN>(st + AT, TN * wc + k - VS, t, lane)
                             : bg_frag_rows<BK>(st + AT, TN * wc + k - VS, t, li, h);
  };
  f32x16 acc[VS][TN];
#pragma unroll
  for (int i = 0; i < VS; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = (f32x16){0};
  // The MFMAs of one step with `items` other instructions spread among them,
  // pinned in this order: the matrix pipe never waits for a burst of LDS
  // reads or DMAs to issue.
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
  constexpr int LOOK = VS <= 2 && NT == 4 ? 2 : 1, FB = 2 * LOOK;
  bf16x8 fa[FB][VS], fb[FB][TN];
  if (gather) wait_vmcnt<(NB - 1) * (NC + 1)>();
  else wait_vmcnt<(NB - 1) * NC>();
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int t = 0; t < LOOK; ++t)
#pragma unroll
    for (int k = 0; k < VS + TN; ++k) read_one(0, t, fa[t], fb[t], k);
  int cur = 0;
  for (int s = 0; s < nst; ++s) {
    const int nxt = cur + 1 == NB ? 0 : cur + 1;
    if (gather) gather_rows(s + NB, idx);
#pragma unroll
    for (int t = 0; t < NT - LOOK; ++t)
      mma(fa[t % FB], fb[t % FB], VS + TN,
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
      mma(fa[t % FB], fb[t % FB], VS + TN + d1 - d0, [&](int k) {
        if (k < VS + TN) read_one(nxt, u, fa[u], fb[u], k);
        else issue_one(q, idx, d0 + k - VS - TN);
      });
    }
    if (gather) issue_index(s + 2 * NB);
    cur = nxt;
  }
  wait_lgkmcnt0();
  wait_vmcnt<0>();
  asm volatile("s_barrier" ::: "memory");

  // Epilogue through LDS, slab by slab, in a region of this wave's own: 16
  // bytes a lane and whole row segments per store instruction.
  constexpr int RS = 128 * TN + 32;  // bytes of an LDS row (the pad parts the lane halves' banks)
  constexpr int SUMS = (KG - 1) * 4 * VS * TN * 16 * 64 * 4;  // the other groups' accumulators
  static_assert(SUMS + 4 * 32 * RS <= (KG > 1 ? 160 * 1024 : bg_lds<TM, TN>()), "epilogue fits the ring");
  if constexpr (KG > 1) {
    float* sums = reinterpret_cast<float*>(block_lds);
#pragma unroll
    for (int i = 0; i < VS; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (grp > 0) sums[((((grp - 1) * 4 + w) * VS * TN + i * TN + j) * 16 + r) * 64 + lane] = acc[i][j][r];
    __syncthreads();
    if (grp > 0) return;
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
  float* t = reinterpret_cast<float*>(block_lds + SUMS + w * 32 * RS);
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
  // pieces of 16 bytes a lane: columns of a piece, lanes a row, pieces a slab
  auto slab = [&](auto bf, int i, int r0) {
    constexpr bool BF = decltype(bf)::value;
    constexpr int CPP = BF ? 8 : 4, LPR = 32 * TN / CPP, U = 32 * LPR / 64;
    const int64_t col = col0 + CPP * (lane % LPR);
    uint32_t off[U];
    u32x4 av[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = u * (64 / LPR) + lane / LPR;
      off[u] = col < N ? (uint32_t)(r0 + r) * nb + (uint32_t)col * (BF ? 2 : 4) : BG_OOB;
      // all of the slab's addends before its first store: add may be y itself,
      // and one load after another would wait for memory U times
      if (MODE == BG_WGRAD && p.add) av[u] = __builtin_amdgcn_raw_buffer_load_b128(radd, off[u], 0, 0);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        t[((8 * (r >> 2) + 4 * h + (r & 3)) * RS + (32 * j + li) * 4) / 4] = acc[i][j][r];
    wave_lds_sync();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = u * (64 / LPR) + lane / LPR;
      const f32x4* q = reinterpret_cast<const f32x4*>(reinterpret_cast<const uint8_t*>(t) + r * RS + (lane % LPR) * 4 * CPP);
      u32x4 o;
      if (BF) {
        f32x4 a = q[0], b = q[1];
        if (MODE == BG_WGRAD && p.add) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            a[2 * c] += __uint_as_float(av[u][c] << 16);
            a[2 * c + 1] += __uint_as_float(av[u][c] & 0xFFFF0000u);
            b[2 * c] += __uint_as_float(av[u][2 + c] << 16);
            b[2 * c + 1] += __uint_as_float(av[u][2 + c] & 0xFFFF0000u);
          }
        }
        o = (u32x4){pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3])};
      } else {
        f32x4 a = q[0];
        if (MODE == BG_WGRAD && p.add) a += __builtin_bit_cast(f32x4, av[u]);
        o = __builtin_bit_cast(u32x4, a);
      }
      __builtin_amdgcn_raw_buffer_store_b128(o, ry, off[u], 0, 2);
    }
    wave_lds_sync();
  };
#pragma unroll
  for (int i = 0; i < VS; ++i) {
    if (p.y_bf) slab(std::true_type{}, i, 32 * (2 * i + wr));
    else slab(std::false_type{}, i, 32 * (2 * i + wr));
  }
}

// The block's tile.  Block b runs on XCD b % 8 (blocks are dealt round robin);
// an XCD takes an eighth of the heavy tiles (more than half of their 64-row
// slabs hold rows) and an eighth of the light ones, each in expert order,
// so that neighbours share operand panels in its L2 and the eighths cost
// alike.  Light tiles stream weights and heavy ones keep the MFMAs busy: the
// light ones are mixed evenly among the heavy ones, but for an eighth of all
// tiles kept for the end, where short tiles level the finish (32768 rows over
// 128 Zipf experts, n = 1536, k = 2048: 299 us; heavy ones first 324).  An
// expert's heavy tiles go in bands of 4 m-tiles; a W past an XCD's 4 MB of L2
// (6.3 MB here) is read again by each band and by the light remainder, a part
// of the 0.54 GB that this layout reads beyond its operands.  Every wave
// derives this from the device offsets by wave scans in registers (G experts
// in NSEG segments of 64 lanes).  False: no tile (block-uniform).
template <int NSEG, int TM, int TN>
__device__ __forceinline__ bool bg_schedule(const int32_t* offsets, int G, int64_t m_total, int tn, int lane, TileRange& out) {
  constexpr int BM = 64 * TM;
  const int32_t mt = (int32_t)m_total;
  int32_t lo[NSEG], hi[NSEG], eh[NSEG], el[NSEG];
#pragma unroll
  for (int i = 0; i < NSEG; ++i)
    if (64 * i < G) {
      lo[i] = offsets[min(64 * i + lane, G)];
      hi[i] = offsets[min(64 * i + lane + 1, G)];
    }
  int32_t nh = 0, nl = 0;
#pragma unroll
  for (int i = 0; i < NSEG; ++i) {
    eh[i] = el[i] = 0x7FFFFFFF;
    if (64 * i >= G) continue;
    const int32_t a = min(max(lo[i], 0), mt), rows = min(max(hi[i], a), mt) - a;
    lo[i] = a;
    hi[i] = a + rows;
    const int32_t slabs = rows / 64 + (rows % 64 != 0), rem = slabs % TM;
    const bool in = 64 * i + lane < G;
    const int32_t ch = in ? slabs / TM + (2 * rem > TM) : 0, cl = in && rem > 0 && 2 * rem <= TM;
    const int32_t ih = wave_incl_scan(ch), il = wave_incl_scan(cl);
    if (in) {
      eh[i] = nh + ih - ch;
      el[i] = nl + il - cl;
    }
    nh += __builtin_amdgcn_readlane(ih, 63);
    nl += __builtin_amdgcn_readlane(il, 63);
  }
  const int x = (int)(blockIdx.x % 8), j = (int)(blockIdx.x / 8);
  const int64_t th = (int64_t)nh * tn, tl = (int64_t)nl * tn;
  const int h0 = (int)(th * x / 8), H = (int)(th * (x + 1) / 8) - h0;
  const int l0 = (int)(tl * x / 8), L = (int)(tl * (x + 1) / 8) - l0;
  if (j >= H + L) return false;
  const int mixed = H + L - min(L, (H + L) / 8);  // H <= mixed
  // heavy tiles among the first j: ceil(j H / mixed)
  auto before = [&](int q) { return q >= mixed ? H : (int)(((int64_t)q * H + mixed - 1) / mixed); };
  const int hb = before(j);
  const bool heavy = before(j + 1) > hb;
  const int idx = heavy ? h0 + hb : l0 + j - hb;
  int m = idx / tn, n = idx % tn;
  int count = 0;
#pragma unroll
  for (int i = 0; i < NSEG; ++i)
    if (64 * i < G) count += __popcll(__ballot((heavy ? eh[i] : el[i]) <= m));
  const int g = max(count - 1, 0), ln = g & 63;
  int32_t lo_s = lo[0], hi_s = hi[0], eh_s = eh[0];
#pragma unroll
  for (int i = 1; i < NSEG; ++i)
    if ((g >> 6) == i) { lo_s = lo[i]; hi_s = hi[i]; eh_s = eh[i]; }
  const int32_t rlo = __builtin_amdgcn_readlane(lo_s, ln), rhi = __builtin_amdgcn_readlane(hi_s, ln);
  int64_t first;
  if (heavy) {
    const int32_t e0 = __builtin_amdgcn_readlane(eh_s, ln);
    const int32_t slabs = (rhi - rlo) / 64 + ((rhi - rlo) % 64 != 0);
    const int mts = slabs / TM + (2 * (slabs % TM) > TM);
    const int q = idx - e0 * tn;  // within the expert's mts x tn heavy tiles
    if (q < 0 || q >= mts * tn) return false;  // never for non-decreasing offsets
    const int band = q / (4 * tn), within = q % (4 * tn), bh = min(4, mts - 4 * band);
    m = 4 * band + within % bh;
    n = within / bh;
    first = (int64_t)rlo + (int64_t)m * BM;
  } else {
    const int32_t slabs = (rhi - rlo) / 64 + ((rhi - rlo) % 64 != 0);
    first = (int64_t)rlo + (int64_t)(slabs / TM) * BM;
  }
  out.g = g;
  out.row_lo = first;
  out.row_hi = min((int64_t)rhi, first + BM);
  out.n0 = (int64_t)n * 64 * TN;
  return out.row_lo < out.row_hi;
}

// wgrad: the block's expert and tile (index within the expert's `tiles`).
// Tiles of experts with more than 128 rows multiply, the others mostly write
// their dW.  The long ones go first, so that the short ones level the finish
// (32768 rows over 128 Zipf experts, n = 1536, k = 2048, fp32, inputs changing
// from call to call: 445 us; short ones first 478, mixed evenly 545: the
// writes push the panels that an expert's tiles share out of the L2s; in
// expert order 513).  XCD x takes every eighth tile of both lists, so that an
// expert's tiles of one block of X columns share an L2 where the columns
// come in eighths; every XCD then reads all of dY (eight times 100 MB there).
template <int NSEG>
__device__ __forceinline__ bool bg_schedule_wgrad(const int32_t* offsets, int G, int64_t m_total, int tiles, int lane,
                                                  int64_t& row_lo, int64_t& row_hi, int& g, int& tile) {
  const int32_t mt = (int32_t)m_total;
  int32_t lo[NSEG], hi[NSEG], eh[NSEG];
#pragma unroll
  for (int i = 0; i < NSEG; ++i)
    if (64 * i < G) {
      lo[i] = offsets[min(64 * i + lane, G)];
      hi[i] = offsets[min(64 * i + lane + 1, G)];
    }
  int32_t nh = 0;
  uint32_t heavy_of = 0;  // bit i: this lane's expert of segment i is heavy
#pragma unroll
  for (int i = 0; i < NSEG; ++i) {
    if (64 * i >= G) continue;
    lo[i] = min(max(lo[i], 0), mt);
    hi[i] = min(max(hi[i], lo[i]), mt);
    const bool h = 64 * i + lane < G && hi[i] - lo[i] > 128;
    heavy_of |= (uint32_t)h << i;
    const int32_t incl = wave_incl_scan(h ? 1 : 0);
    eh[i] = nh + incl - (h ? 1 : 0);  // heavy experts before this one
    nh += __builtin_amdgcn_readlane(incl, 63);
  }
  const int x = (int)(blockIdx.x % 8), j = (int)(blockIdx.x / 8);
  const int64_t th = (int64_t)nh * tiles, tl = (int64_t)(G - nh) * tiles;
  const int H = (int)((th - x + 7) / 8), L = (int)((tl - x + 7) / 8);
  if (j >= H + L) return false;
  const bool heavy = j < H;
  const int64_t idx = 8 * (int64_t)(heavy ? j : j - H) + x;
  const int e = (int)(idx / tiles);  // of the list's experts
  tile = (int)(idx % tiles);
  g = 0;
  row_lo = row_hi = 0;
#pragma unroll
  for (int i = 0; i < NSEG; ++i) {
    if (64 * i >= G) continue;
    const int ex = 64 * i + lane;
    const bool h = (heavy_of >> i) & 1u;
    const unsigned long long b = __ballot(ex < G && h == heavy && (h ? eh[i] : ex - eh[i]) == e);
    if (b) {
      const int ln = __builtin_ctzll(b);
      g = 64 * i + ln;
      row_lo = __builtin_amdgcn_readlane(lo[i], ln);
      row_hi = __builtin_amdgcn_readlane(hi[i], ln);
    }
  }
  return true;
}

template <int MODE, int TM, int TN, int BK, int KG>
__global__ __launch_bounds__(256 * KG, (KG > 1 ? KG : bg_blocks<TM, TN>())) void bf16_tile_kernel(Bf16Args p) {
  typedef BgMode<MODE> M;
  constexpr int BM = 64 * TM, BN = 64 * TN;
  __shared__ __attribute__((aligned(16))) uint8_t lds[KG > 1 ? 160 * 1024 : bg_lds<TM, TN>()];
  constexpr int D = BK / 32, CPR = BK / 8;  // DMAs per slab and wave; chunks of a row operand's LDS row
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = wave & 3, grp = wave >> 2;
  BgTile tl;
  BgOperand<TM> oa;
  BgOperand<TN> ob;
  int vs;
  if constexpr (MODE == BG_WGRAD) {
    // an expert's tiles: X columns fastest
    const int tn = (int)((p.n + BM - 1) / BM), tk = (int)((p.k + BN - 1) / BN);
    int r;
    const bool some = p.groups <= 256
        ? bg_schedule_wgrad<4>(p.offsets, p.groups, p.m_total, tn * tk, lane, tl.row_lo, tl.row_hi, tl.g, r)
        : bg_schedule_wgrad<16>(p.offsets, p.groups, p.m_total, tn * tk, lane, tl.row_lo, tl.row_hi, tl.g, r);
    if (!some) return;  // block-uniform
    const int64_t lo = tl.row_lo;
    tl.K = tl.row_hi - lo;
    tl.m0 = (int64_t)(r / tk) * BM;  // column of dY
    tl.n0 = (int64_t)(r % tk) * BN;  // column of X
    vs = (int)min((int64_t)TM, (p.n - tl.m0 + 63) / 64);
    // column operands: DMA i covers the summed rows (4 i + w) (8 / T) ..
    oa.stride = p.n * 2;
    oa.base = reinterpret_cast<const uint8_t*>(p.a + lo * p.n + tl.m0);
#pragma unroll
    for (int i = 0; i < TM * D; ++i) {
      const int row = (4 * i + w) * (8 / TM) + lane / (8 * TM);
      const int c = 8 * ((lane % (8 * TM)) ^ bg_col_swz<TM>(row));
      oa.voff[i] = tl.m0 + c < p.n ? (uint32_t)(row * oa.stride) + 2 * c : BG_OOB;
    }
    ob.stride = p.k * 2;
    ob.base = reinterpret_cast<const uint8_t*>(p.b + (p.row_index ? 0 : lo * p.k) + tl.n0);
    if (p.row_index) ob.rsrc = bg_rsrc(p.b, p.a_rows * p.k * 2);
#pragma unroll
    for (int i = 0; i < TN * D; ++i) {
      const int row = (4 * i + w) * (8 / TN) + lane / (8 * TN);
      const int c = 8 * ((lane % (8 * TN)) ^ bg_col_swz<TN>(row));
      const uint32_t at = p.row_index ? (uint32_t)(tl.n0 * 2) : (uint32_t)(row * ob.stride);
      ob.voff[i] = tl.n0 + c < p.k ? at + 2 * c : BG_OOB;
    }
  } else {
    TileRange tr;
    const int tn = (int)(((MODE == BG_FORWARD ? p.n : p.k) + BN - 1) / BN);
    const bool some = p.groups <= 256 ? bg_schedule<4, TM, TN>(p.offsets, p.groups, p.m_total, tn, lane, tr)
                                      : bg_schedule<16, TM, TN>(p.offsets, p.groups, p.m_total, tn, lane, tr);
    if (!some) return;  // block-uniform
    tl.row_lo = tr.row_lo;
    tl.row_hi = tr.row_hi;
    tl.n0 = tr.n0;
    tl.g = tr.g;
    tl.K = MODE == BG_FORWARD ? p.k : p.n;
    vs = (int)((tl.row_hi - tl.row_lo + 63) / 64);
    // A: row operand, DMA i covers the tile's rows 64 / CPR (4 i + w) ..
    const uint32_t rowb = (uint32_t)tl.K * 2;
    const int swz = 16 * ((lane % CPR) ^ bg_row_swz<BK>(64 / CPR * w + lane / CPR));
    if (p.row_index) oa.rsrc = bg_rsrc(p.a, p.a_rows * (int64_t)rowb);
    else oa.rsrc = bg_rsrc(p.a + tl.row_lo * tl.K, (tl.row_hi - tl.row_lo) * (int64_t)rowb);
#pragma unroll
    for (int i = 0; i < TM * D; ++i) {
      const int64_t row = tl.row_lo + 64 / CPR * (4 * i + w) + lane / CPR;
      int64_t src = gathered_row(p.row_index, p.a_rows, row, tl.row_hi);
      if (!p.row_index && src >= 0) src -= tl.row_lo;
      oa.voff[i] = src >= 0 ? (uint32_t)src * rowb + swz : BG_OOB;
    }
    if constexpr (M::b_cols) {
      ob.stride = p.k * 2;
      ob.base = reinterpret_cast<const uint8_t*>(p.b + (int64_t)tl.g * p.n * p.k + tl.n0);
#pragma unroll
      for (int i = 0; i < TN * D; ++i) {
        const int row = (4 * i + w) * (8 / TN) + lane / (8 * TN);
        const int c = 8 * ((lane % (8 * TN)) ^ bg_col_swz<TN>(row));
        ob.voff[i] = tl.n0 + c < p.k ? (uint32_t)(row * ob.stride) + 2 * c : BG_OOB;
      }
    } else {
      const int64_t cols = min((int64_t)BN, p.n - tl.n0);
      ob.rsrc = bg_rsrc(p.b + ((int64_t)tl.g * p.n + tl.n0) * p.k, cols * p.k * 2);
#pragma unroll
      for (int i = 0; i < TN * D; ++i) {
        const int c = 64 / CPR * (4 * i + w) + lane / CPR;
        ob.voff[i] = c < cols ? (uint32_t)c * rowb + swz : BG_OOB;
      }
    }
  }
  int nst = (int)((tl.K + BK - 1) / BK);
  if constexpr (KG > 1) {  // this group's range of the sum
    nst = (nst + KG - 1) / KG;
    const int64_t start = (int64_t)grp * nst * BK;
    tl.K = min((int64_t)nst * BK, max((int64_t)0, tl.K - start));
    if constexpr (M::a_cols) {
      oa.base += start * oa.stride;
    } else {
#pragma unroll
      for (int i = 0; i < TM * D; ++i)
        if (oa.voff[i] != BG_OOB) oa.voff[i] += (uint32_t)start * 2;
    }
    if constexpr (!M::b_cols) {
#pragma unroll
      for (int i = 0; i < TN * D; ++i)
        if (ob.voff[i] != BG_OOB) ob.voff[i] += (uint32_t)start * 2;
    } else if (MODE == BG_DGRAD || !p.row_index) {
      ob.base += start * ob.stride;
    }
    if (MODE == BG_WGRAD) tl.row_lo += start;  // the first summed row
  }
  if constexpr (TM == 4) {
    switch (vs) {
      case 4: bg_body<MODE, TM, TN, BK, KG, 4>(p, tl, oa, ob, lds, nst, grp, w, lane); break;
      case 3: bg_body<MODE, TM, TN, BK, KG, 3>(p, tl, oa, ob, lds, nst, grp, w, lane); break;
      case 2: bg_body<MODE, TM, TN, BK, KG, 2>(p, tl, oa, ob, lds, nst, grp, w, lane); break;
      default: bg_body<MODE, TM, TN, BK, KG, 1>(p, tl, oa, ob, lds, nst, grp, w, lane); break;
    }
  } else if constexpr (TM == 3) {
    if (vs == 3) bg_body<MODE, TM, TN, BK, KG, 3>(p, tl, oa, ob, lds, nst, grp, w, lane);
    else if (vs == 2) bg_body<MODE, TM, TN, BK, KG, 2>(p, tl, oa, ob, lds, nst, grp, w, lane);
    else bg_body<MODE, TM, TN, BK, KG, 1>(p, tl, oa, ob, lds, nst, grp, w, lane);
  } else if constexpr (TM == 2) {
    if (vs == 2) bg_body<MODE, TM, TN, BK, KG, 2>(p, tl, oa, ob, lds, nst, grp, w, lane);
    else bg_body<MODE, TM, TN, BK, KG, 1>(p, tl, oa, ob, lds, nst, grp, w, lane);
  } else {
    bg_body<MODE, TM, TN, BK, KG, 1>(p, tl, oa, ob, lds, nst, grp, w, lane);
  }
}

template <int MODE, int TM, int TN, int BK, int KG = 1>
static void launch_tiles(const Bf16Args& a, hipStream_t str) {
  Bf16Args p = a;
  int64_t blocks;
  if (MODE == BG_WGRAD) {
    // every XCD's share of the two lists rounded up
    blocks = (int64_t)p.groups * ((p.n + 64 * TM - 1) / (64 * TM)) * ((p.k + 64 * TN - 1) / (64 * TN));
    blocks = 8 * ((blocks + 7) / 8 + 1);
  } else {
    // at most a partial m-tile per expert that has rows, and an XCD's two
    // ranges each rounded up
    const int64_t mts = (p.m_total + 64 * TM - 1) / (64 * TM) + (p.groups < p.m_total ? p.groups : p.m_total);
    blocks = 8 * ((mts * (((MODE == BG_FORWARD ? p.n : p.k) + 64 * TN - 1) / (64 * TN)) + 7) / 8 + 2);
  }
  hipLaunchKernelGGL((bf16_tile_kernel<MODE, TM, TN, BK, KG>), dim3((unsigned)blocks), dim3(256 * KG), 0, str, p);
}

// Tiles of a call in units of the CUs (an upper estimate: every expert may add
// a partial m-tile), and the choice of tile from it.  The largest tile that
// still gives every CU work is the fastest: it reads each operand least and
// keeps the MFMAs busiest (one expert of 8192 rows, n = k = 8192: 256 x 256
// 840 us, 192 x 128 938, 128 x 128 983, 64 x 128 1223, 64 x 64 1567), but a
// grid of few tiles is bound by one tile's chain of stages, which is shorter
// for a small tile (32 rows over 8 experts, n = k = 2048: 256 x 256 22 us,
// 64 x 64 14).
//  - forward: two 192 x 128 tiles a CU level ragged experts and hide each
//    other's epilogues where the grid has fewer than three 256 x 256 tiles
//    a CU (4096 rows over 8 experts, n = k = 2048: 44 us against 54), and
//    experts with few rows are streams of weights, for which more blocks a CU
//    hide more latency (1024 rows over 32 experts: 64 x 128 32 us against 52).
//  - dgrad: W is read in rows of the output's columns, 512 contiguous bytes
//    for 256 columns; two 128 x 256 tiles a CU beat one 256 x 256 tile
//    (32768 rows over 128 experts, n = 2048, k = 768: 165 us against 189).
//  - wgrad: two 256 x 128 tiles a CU: one writes its dW while the other
//    multiplies (32768 rows over 128 experts, n = 1536, k = 2048, bf16: 354 us
//    against 432 for 256 x 256); with one tile a CU and long sums, smaller
//    tiles lose nothing where experts have equal rows and spread the largest
//    one's work where they do not (32768 rows over 8 Zipf experts, n = k =
//    1024: 128 x 128 192 us against 244; equal experts 93 and 92).
//  - few tiles and a long sum: two wave groups of a block halve the chain (64
//    rows, n = k = 4096: 18.3 us against 21.5, where its bytes alone take 6;
//    wgrad of 15262 rows over 3 experts, n = 784, k = 104: 71 against 108, its
//    bytes 5: few CUs have work; four groups gain no more: a CU's loads bound
//    them).
template <int MODE>
static int launch_bf16(const Bf16Args& p, hipStream_t str) {
  const int64_t cus = nvfp4host::num_cus();
  const int64_t rows = p.m_total / p.groups;  // of an expert, on average
  auto tiles = [&](int TM, int TN) -> int64_t {
    if (MODE == BG_WGRAD) return p.groups * ((p.n + 64 * TM - 1) / (64 * TM)) * ((p.k + 64 * TN - 1) / (64 * TN));
    const int64_t partial = (p.groups < p.m_total ? p.groups : p.m_total) - 1;
    return ((p.m_total + 64 * TM - 1) / (64 * TM) + partial) *
           (((MODE == BG_FORWARD ? p.n : p.k) + 64 * TN - 1) / (64 * TN));
  };
  if constexpr (MODE == BG_FORWARD) {
    if (tiles(4, 4) >= 3 * cus && rows >= 24) launch_tiles<MODE, 4, 4, 64>(p, str);
    else if (tiles(3, 2) >= cus && rows >= 128) launch_tiles<MODE, 3, 2, 64>(p, str);
    else if (tiles(2, 2) >= 2 * cus) launch_tiles<MODE, 2, 2, 64>(p, str);
    else if (2 * tiles(1, 2) >= cus && rows >= 24) launch_tiles<MODE, 1, 2, 64>(p, str);
    else if (2 * tiles(1, 1) <= cus && p.k >= 2048) launch_tiles<MODE, 1, 1, 64, 2>(p, str);
    else launch_tiles<MODE, 1, 1, 64>(p, str);
  } else if constexpr (MODE == BG_DGRAD) {
    if (tiles(2, 4) >= cus) launch_tiles<MODE, 2, 4, 32>(p, str);
    else if (2 * tiles(1, 2) >= cus && rows >= 24) launch_tiles<MODE, 1, 2, 64>(p, str);
    else if (2 * tiles(1, 1) <= cus && p.n >= 2048) launch_tiles<MODE, 1, 1, 64, 2>(p, str);
    else launch_tiles<MODE, 1, 1, 64>(p, str);
  } else {
    if (tiles(4, 2) >= (rows < 1024 ? cus : 2 * cus)) launch_tiles<MODE, 4, 2, 32>(p, str);
    else if (tiles(2, 2) >= cus) launch_tiles<MODE, 2, 2, 64>(p, str);
    else if (tiles(1, 2) >= cus) launch_tiles<MODE, 1, 2, 64>(p, str);
    else if (tiles(1, 1) <= cus && rows >= 1024) launch_tiles<MODE, 1, 1, 64, 2>(p, str);
    else launch_tiles<MODE, 1, 1, 64>(p, str);
  }
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
