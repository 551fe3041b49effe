// vocab_loss.hip -- the negative log-probability of a row's target over a large
// vocabulary, without the logits, and its gradients (gfx950).
//
//   z[r, v] = scale <h[r], w[v]>,  lse[r] = log sum_v e^z[r, v]
//   loss[r] = lse[r] - z[r, t_r]
//   dz[r, v] = scale d_loss[r] (e^(z[r, v] - lse[r]) - [v = t_r])
//   dh = dz w,  dw = add + dz^T h
//
// Rows without a target (t_r outside the vocabulary) are taken out first: a
// scan numbers the others, and every product runs over those alone, gathered
// from h by that numbering, so that prompt and padding rows cost nothing and
// whatever they hold reaches no gradient.
//
// Forward: the block tiles of the bf16 products, with an epilogue that leaves
// one partial sum a row and tile.  The sums are taken relative to a reference
// that every tile knows: the target's own logit, one dot product a row before
// the tiles start.  Then no tile needs its maximum first (a reduction across
// lanes as long as the sum's) and no term that matters can vanish, since lse
// >= z[r, t_r].  Where a tile's sum leaves fp32 all the same (a logit 88 above
// the target's), that tile takes its own maximum instead.
//
// Backward, a piece of the vocabulary at a time: the logits' tiles again, now
// turned into dz and rounded to bf16 for the two products that read them (a
// relative 2^-9 a term, as every gradient that the bf16 products take), then
// dh += dz w summed over the pieces in fp32, and dw = dz^T h, which is whole
// for the piece's rows of w.  Few rows leave few tiles of dh: the sum over the
// vocabulary is then split over blocks, each with fp32 sums of its own, added
// in order at the end.
#include <type_traits>

#include "bf16_tile.h"

namespace nvfp4 {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct VocabArgs {
  const uint16_t *h, *w;
  const int32_t* targets;
  int64_t rows, vocab, k;
  float scale;
  // workspace: number of the rows that have a target, the row of each number,
  // the number of each row (-1: none), and by number
  int32_t *count, *row_index, *number;
  int32_t* target;   // its target
  float* ref;        // forward: scale log2(e) <h, w_t>; backward: lse log2(e)
  float* coef;       // backward: scale d_loss
  float2* part;      // forward: [tiles][rows] exponent and sum of a tile
  float *loss, *lse;
  // backward
  const float *lse_in, *d_loss;
  uint16_t* dz;      // [rows, ld] of the piece
  int64_t ld, v0, width;  // the piece: vocabulary rows [v0, v0 + width)
  float* sums;       // [splits][rows, k]
  int splits;
  int64_t per_split; // vocabulary rows a split sums
  bool first;        // piece: the sums start here
  uint16_t* dh;
  const void* add;
  void* dw;
  bool dw_bf;
};

// -------------------------------------------------------------- numbering --

__device__ __forceinline__ bool has_target(const VocabArgs& p, int64_t r) {
  const int32_t t = p.targets[r];
  return t >= 0 && t < p.vocab;
}

// Block 0 numbers the rows with a target in order; the other blocks (forward)
// take the targets' logits, a wave a row, into ref by row.
__global__ __launch_bounds__(1024) void vocab_rows_kernel(VocabArgs p) {
  __shared__ int s_wave[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (blockIdx.x > 0) {
    for (int64_t r = (int64_t)(blockIdx.x - 1) * 16 + wave; r < p.rows; r += (int64_t)(gridDim.x - 1) * 16) {
      const int32_t t = p.targets[r];
      if (t < 0 || t >= p.vocab) continue;
      float acc = 0.0f;
      for (int64_t e = 8 * lane; e < p.k; e += 512) {
        float a[8], b[8];
        load8<true>(p.h + r * p.k + e, true, 8, 0, 64, 0, a);
        load8<true>(p.w + (int64_t)t * p.k + e, true, 8, 0, 64, 0, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc = __builtin_fmaf(a[i], b[i], acc);
      }
      acc = wave_sum_f32(acc);
      if (lane == 0) p.ref[r] = acc * (p.scale * LOG2E);
    }
    return;
  }
  int base = 0;
  for (int64_t r0 = 0; r0 < p.rows; r0 += 1024) {
    const int64_t r = r0 + tid;
    const bool has = r < p.rows && has_target(p, r);
    const uint64_t b = __ballot(has);
    if (lane == 0) s_wave[wave] = __popcll(b);
    __syncthreads();
    int at = base, total = 0;
    for (int w = 0; w < 16; ++w) {
      if (w < wave) at += s_wave[w];
      total += s_wave[w];
    }
    at += __popcll(b & ((1ull << lane) - 1));
    if (r < p.rows) {
      if (p.number) p.number[r] = has ? at : -1;
      if (has) {
        p.row_index[at] = (int32_t)r;
        if (p.coef) {
          p.target[at] = p.targets[r];
          p.ref[at] = p.lse_in[r] * LOG2E;
          p.coef[at] = p.d_loss[r] * p.scale;
        }
      }
    }
    base += total;
    __syncthreads();
  }
  if (tid == 0) *p.count = base;
}

// ------------------------------------------------------------------ tiles --

// Tile (m, n) of a grid of tm x tn for block b of it: block b runs on XCD
// b % 8, an XCD takes an eighth of the tiles in order, and the order goes
// through bands of up to 8 tiles along m, m fastest, so that the tiles an XCD
// works on at a time share panels of both operands in its L2.
__device__ __forceinline__ bool vocab_tile(int64_t tm, int64_t tn, int64_t b, int64_t& m, int64_t& n) {
  const int64_t x = b % 8, j = b / 8, tiles = tm * tn;
  const int64_t lo = tiles * x / 8, hi = tiles * (x + 1) / 8;
  if (lo + j >= hi) return false;
  const int64_t t = lo + j, band = t / (8 * tn), in = t % (8 * tn), bh = min((int64_t)8, tm - 8 * band);
  m = 8 * band + in % bh;
  n = in / bh;
  return true;
}

// Row operand: DMA offsets of T slabs of rows [row0, rows) of a matrix whose
// rows are `rowb` bytes, from the resource's base; `index`: gathered rows.
template <int T, int BK>
__device__ __forceinline__ void rows_operand(BgOperand<T>& o, const int32_t* index, int64_t index_rows, int64_t row0,
                                             int64_t rows, uint32_t rowb, int w, int lane) {
  constexpr int CPR = BK / 8;
  const int swz = 16 * ((lane % CPR) ^ bg_row_swz<BK>(64 / CPR * w + lane / CPR));
#pragma unroll
  for (int i = 0; i < T * BK / 32; ++i) {
    const int64_t row = row0 + 64 / CPR * (4 * i + w) + lane / CPR;
    int64_t src = gathered_row(index, index_rows, row, rows);
    if (!index && src >= 0) src -= row0;
    o.voff[i] = src >= 0 ? (uint32_t)src * rowb + swz : BG_OOB;
  }
}
// Column operand: DMA offsets of T slabs of columns [col0, cols), summed rows
// `stride` bytes apart (gathered: only the column's part).
template <int T, int BK>
__device__ __forceinline__ void cols_operand(BgOperand<T>& o, bool gathered, int64_t col0, int64_t cols, int w, int lane) {
#pragma unroll
  for (int i = 0; i < T * BK / 32; ++i) {
    const int row = (4 * i + w) * (8 / T) + lane / (8 * T);
    const int c = 8 * ((lane % (8 * T)) ^ bg_col_swz<T>(row));
    const uint32_t at = gathered ? (uint32_t)(col0 * 2) : (uint32_t)(row * o.stride);
    o.voff[i] = col0 + c < cols ? at + 2 * c : BG_OOB;
  }
}

// sum over the 32 lanes of each half of a wave (every lane gets it)
__device__ __forceinline__ float half_sum(float v) {
  v += __uint_as_float(dpp_mov<0xB1>(__float_as_uint(v)));   // quad_perm [1,0,3,2]
  v += __uint_as_float(dpp_mov<0x4E>(__float_as_uint(v)));   // quad_perm [2,3,0,1]
  v += __uint_as_float(dpp_mov<0x141>(__float_as_uint(v)));  // row_half_mirror
  v += __uint_as_float(dpp_mov<0x140>(__float_as_uint(v)));  // row_mirror
  return v + __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401F));
}

struct TileParams {  // what bg_sum reads of its arguments
  const int32_t* row_index;
  int64_t a_rows;
};

// The sums of a tile's valid slabs, then epi(acc) for VS of them.
template <int MODE, int TM, int TN, int BK, int KG, class Epi>
__device__ __forceinline__ void tile_sums(const TileParams& a, const BgTile& tl, BgOperand<TM>& oa, BgOperand<TN>& ob,
                                          uint8_t* lds, int vs, int nst, int grp, int w, int lane, Epi&& epi) {
  auto run = [&](auto n) {
    constexpr int VS = decltype(n)::value;
    f32x16 acc[VS][TN];
    if (bg_sum<MODE, TM, TN, BK, KG, VS>(a, tl, oa, ob, lds, nst, grp, w, lane, acc)) epi(acc);
  };
  if constexpr (TM == 4) {
    if (vs == 4) run(std::integral_constant<int, 4>());
    else if (vs == 3) run(std::integral_constant<int, 3>());
    else if (vs == 2) run(std::integral_constant<int, 2>());
    else run(std::integral_constant<int, 1>());
  } else if constexpr (TM == 2) {
    if (vs == 2) run(std::integral_constant<int, 2>());
    else run(std::integral_constant<int, 1>());
  } else {
    run(std::integral_constant<int, TM>());
  }
}

// Logits of a tile: DZ false leaves its partial sums, DZ true writes dz.
template <int TM, int TN, bool DZ>
__global__ __launch_bounds__(256, (bg_blocks<TM, TN>())) void vocab_logits_kernel(VocabArgs p) {
  constexpr int BM = 64 * TM, BN = 64 * TN, BK = 64;
  __shared__ __attribute__((aligned(16))) uint8_t lds[bg_lds<TM, TN>()];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t count = *p.count;
  int64_t m, n;
  if (!vocab_tile((count + BM - 1) / BM, (p.width + BN - 1) / BN, blockIdx.x, m, n)) return;  // block-uniform
  BgTile tl;
  BgOperand<TM> oa;
  BgOperand<TN> ob;
  tl.row_lo = m * BM;
  tl.row_hi = min(count, tl.row_lo + BM);
  tl.n0 = n * BN;
  tl.m0 = tl.g = 0;
  tl.K = p.k;
  const uint32_t rowb = (uint32_t)p.k * 2;
  oa.rsrc = bg_rsrc(p.h, p.rows * (int64_t)rowb);
  rows_operand<TM, BK>(oa, p.row_index, p.rows, tl.row_lo, tl.row_hi, rowb, w, lane);
  const int64_t cols = min((int64_t)BN, p.width - tl.n0);
  ob.rsrc = bg_rsrc(p.w + (p.v0 + tl.n0) * p.k, cols * rowb);
  rows_operand<TN, BK>(ob, nullptr, cols, 0, cols, rowb, w, lane);
  const int li = lane & 31, half = lane >> 5, wr = w >> 1, wc = w & 1;
  const int vs = (int)((tl.row_hi - tl.row_lo + 63) / 64), nst = (int)((p.k + BK - 1) / BK);
  const TileParams a = {p.row_index, p.rows};
  tile_sums<BG_FORWARD, TM, TN, BK, 1>(a, tl, oa, ob, lds, vs, nst, 0, w, lane, [&](auto& acc) {
    constexpr int VS = sizeof(acc) / sizeof(acc[0]);
    // the tile's rows: reference, and for dz coefficient and target column
    float* s_ref = reinterpret_cast<float*>(lds);
    float* s_coef = s_ref + BM;
    int* s_col = reinterpret_cast<int*>(s_coef + BM);
    for (int r = threadIdx.x; r < 64 * VS; r += 256) {
      const int64_t row = tl.row_lo + r;
      const bool in = row < tl.row_hi;
      if (DZ) {
        s_ref[r] = in ? p.ref[row] : 0.0f;
        s_coef[r] = in ? p.coef[row] : 0.0f;
        const int64_t c = in ? (int64_t)p.target[row] - p.v0 - tl.n0 : -1;
        s_col[r] = c >= 0 && c < BN ? (int)c : -1;
      } else {
        s_ref[r] = in ? p.ref[p.row_index[row]] : 0.0f;
      }
    }
    __syncthreads();
    const float f = p.scale * LOG2E;
    const int64_t left = p.width - tl.n0 - 32 * TN * wc - li;  // this lane's column of j exists: 32 j < left
    if constexpr (!DZ) {
      // partial sums of this wave's columns; the two column halves meet in LDS
      float2* s_part = reinterpret_cast<float2*>(lds + 16 * 1024);
#pragma unroll
      for (int i = 0; i < VS; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row0 = 32 * (2 * i + wr) + 8 * q + 4 * half;
          const f32x4 ref = *reinterpret_cast<const f32x4*>(s_ref + row0);
          float s[4], top[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            s[r] = 0.0f;
            top[r] = ref[r];
#pragma unroll
            for (int j = 0; j < TN; ++j)
              s[r] += 32 * j < left ? __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][4 * q + r], f, -ref[r])) : 0.0f;
          }
          bool over = false;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            s[r] = half_sum(s[r]);
            over |= !(s[r] < 0x1p120f);
          }
          if (__ballot(over)) {  // wave-uniform: relative to the row's maximum here
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float t = -__builtin_inff();
#pragma unroll
              for (int j = 0; j < TN; ++j)
                t = 32 * j < left ? __builtin_fmaxf(t, acc[i][j][4 * q + r] * f) : t;
#pragma unroll
              for (int o = 1; o < 32; o <<= 1) t = __builtin_fmaxf(t, __shfl_xor(t, o, 64));
              float u = 0.0f;
#pragma unroll
              for (int j = 0; j < TN; ++j)
                u += 32 * j < left && !(acc[i][j][4 * q + r] * f == -__builtin_inff())
                         ? __builtin_amdgcn_exp2f(acc[i][j][4 * q + r] * f - t) : 0.0f;
#pragma unroll
              for (int o = 1; o < 32; o <<= 1) u += __shfl_xor(u, o, 64);
              // of this row alone: its neighbours keep their bits
              if (!(s[r] < 0x1p120f)) {
                s[r] = u;
                top[r] = t;
              }
            }
          }
          if (li == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) s_part[wc * BM + row0 + r] = make_float2(top[r], s[r]);
          }
        }
      __syncthreads();
      for (int r = threadIdx.x; r < 64 * VS; r += 256) {
        if (tl.row_lo + r >= tl.row_hi) continue;
        const float2 a0 = s_part[r], a1 = s_part[BM + r];
        float2 o = make_float2(__builtin_fmaxf(a0.x, a1.x), 0.0f);
        if (a0.x == a1.x) o.y = a0.y + a1.y;
        else o.y = a0.y * __builtin_amdgcn_exp2f(a0.x - o.x) + a1.y * __builtin_amdgcn_exp2f(a1.x - o.x);
        p.part[n * p.rows + tl.row_lo + r] = o;
      }
    } else {
      // dz, 32 rows of this wave at a time through LDS: 16 bytes a lane and
      // whole row segments per store.  Columns past the vocabulary, which the
      // products read, are zero.
      constexpr int RS = 64 * TN + 16;  // bytes of an LDS row
      uint8_t* t = lds + 16 * 1024 + w * 32 * RS;
      const int64_t col0 = tl.n0 + 32 * TN * wc;
#pragma unroll
      for (int i = 0; i < VS; ++i) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row0 = 32 * (2 * i + wr) + 8 * q + 4 * half;
          const f32x4 ref = *reinterpret_cast<const f32x4*>(s_ref + row0);
          const f32x4 coef = *reinterpret_cast<const f32x4*>(s_coef + row0);
          typedef int i32x4v __attribute__((ext_vector_type(4)));
          const i32x4v col = *reinterpret_cast<const i32x4v*>(s_col + row0);
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
              const float pr = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][4 * q + r], f, -ref[r]));
              const float one = col[r] == 32 * (TN * wc + j) + li ? 1.0f : 0.0f;
              const float v = 32 * j < left ? coef[r] * (pr - one) : 0.0f;
              *reinterpret_cast<uint16_t*>(t + (8 * q + 4 * half + r) * RS + (32 * j + li) * 2) = to_bf16(v);
            }
        }
        wave_lds_sync();
        constexpr int LPR = 4 * TN, U = 32 * LPR / 64;  // lanes a row, stores a slab
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = u * (64 / LPR) + lane / LPR;
          const int64_t row = tl.row_lo + 32 * (2 * i + wr) + r, c = col0 + 8 * (lane % LPR);
          if (row < tl.row_hi && c < p.ld)
            *reinterpret_cast<u32x4*>(p.dz + row * p.ld + c) =
                *reinterpret_cast<const u32x4*>(t + r * RS + (lane % LPR) * 16);
        }
        wave_lds_sync();
      }
    }
  });
}

// Store of a tile through LDS, slab by slab: rows of `rows` that exist from
// out_row on, columns of N, fp32 or bf16, with `add` (may be y itself) added.
template <int VS, int TN, bool BF, class Row>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[VS][TN], uint8_t* lds, void* y, const void* add, int64_t N,
                                           int64_t col0, int w, int lane, Row&& row_at_slab) {
  constexpr int RS = 128 * TN + 32, CPP = BF ? 8 : 4, LPR = 32 * TN / CPP, U = 32 * LPR / 64, ES = BF ? 2 : 4;
  const int li = lane & 31, half = lane >> 5, wr = w >> 1;
  float* t = reinterpret_cast<float*>(lds + w * 32 * RS);
  const int64_t col = col0 + CPP * (lane % LPR);
#pragma unroll
  for (int i = 0; i < VS; ++i) {
    int64_t at[U];
    u32x4 av[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = row_at_slab(32 * (2 * i + wr) + u * (64 / LPR) + lane / LPR);
      at[u] = row >= 0 && col < N ? (row * N + col) * ES : -1;
      // all of the slab's addends before its first store: add may be y itself
      if (add && at[u] >= 0) av[u] = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(add) + at[u]);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) t[((8 * (r >> 2) + 4 * half + (r & 3)) * RS + (32 * j + li) * 4) / 4] = acc[i][j][r];
    wave_lds_sync();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = u * (64 / LPR) + lane / LPR;
      const f32x4* q = reinterpret_cast<const f32x4*>(reinterpret_cast<const uint8_t*>(t) + r * RS + (lane % LPR) * 4 * CPP);
      u32x4 o;
      if (BF) {
        f32x4 a = q[0], b = q[1];
        if (add) {
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
        if (add) a += __builtin_bit_cast(f32x4, av[u]);
        o = __builtin_bit_cast(u32x4, a);
      }
      if (at[u] >= 0)
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(static_cast<uint8_t*>(y) + at[u]));
    }
    wave_lds_sync();
  }
}

// sums[split] += dz w over the split's part of the piece (= in the first piece)
template <int TM, int TN, int BK>
__global__ __launch_bounds__(256, (bg_blocks<TM, TN>())) void vocab_dh_kernel(VocabArgs p) {
  constexpr int BM = 64 * TM, BN = 64 * TN;
  __shared__ __attribute__((aligned(16))) uint8_t lds[bg_lds<TM, TN>()];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t count = *p.count;
  // a split's tiles follow one another; a row's splits lie along m
  const int64_t tm = (count + BM - 1) / BM, tn = (p.k + BN - 1) / BN;
  int64_t m, n;
  if (!vocab_tile(tm * p.splits, tn, blockIdx.x, m, n)) return;  // block-uniform
  const int64_t split = m / tm, s0 = split * p.per_split;
  BgTile tl;
  BgOperand<TM> oa;
  BgOperand<TN> ob;
  tl.row_lo = (m % tm) * BM;
  tl.row_hi = min(count, tl.row_lo + BM);
  tl.n0 = n * BN;
  tl.m0 = tl.g = 0;
  tl.K = max((int64_t)0, min(p.per_split, p.width - s0));
  const uint32_t rowb = (uint32_t)p.ld * 2;
  // a split past a short last piece has nothing to sum: no byte of dz either
  oa.rsrc = bg_rsrc(p.dz + tl.row_lo * p.ld + s0, tl.K > 0 ? (tl.row_hi - tl.row_lo) * (int64_t)rowb - s0 * 2 : 0);
  rows_operand<TM, BK>(oa, nullptr, count, tl.row_lo, tl.row_hi, rowb, w, lane);
  ob.stride = p.k * 2;
  ob.base = reinterpret_cast<const uint8_t*>(p.w + (p.v0 + s0) * p.k + tl.n0);
  cols_operand<TN, BK>(ob, false, tl.n0, p.k, w, lane);
  const int vs = (int)((tl.row_hi - tl.row_lo + 63) / 64), nst = (int)((tl.K + BK - 1) / BK);
  const TileParams a = {nullptr, count};
  tile_sums<BG_DGRAD, TM, TN, BK, 1>(a, tl, oa, ob, lds, vs, nst, 0, w, lane, [&](auto& acc) {
    constexpr int VS = sizeof(acc) / sizeof(acc[0]);
    float* y = p.sums + split * p.rows * p.k;
    store_tile<VS, TN, false>(acc, lds, y, p.first ? nullptr : y, p.k, tl.n0 + 32 * TN * (w & 1), w, lane, [&](int r) {
      return tl.row_lo + r < tl.row_hi ? tl.row_lo + r : (int64_t)-1;
    });
  });
}

// dw of the piece's rows of w = add + dz^T h
template <int TM, int TN, int BK>
__global__ __launch_bounds__(256, (bg_blocks<TM, TN>())) void vocab_dw_kernel(VocabArgs p) {
  constexpr int BM = 64 * TM, BN = 64 * TN;
  __shared__ __attribute__((aligned(16))) uint8_t lds[bg_lds<TM, TN>()];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t count = *p.count;
  int64_t m, n;
  if (!vocab_tile((p.width + BM - 1) / BM, (p.k + BN - 1) / BN, blockIdx.x, m, n)) return;  // block-uniform
  BgTile tl;
  BgOperand<TM> oa;
  BgOperand<TN> ob;
  tl.row_lo = 0;
  tl.row_hi = tl.K = count;
  tl.m0 = m * BM;
  tl.n0 = n * BN;
  tl.g = 0;
  oa.stride = p.ld * 2;
  oa.base = reinterpret_cast<const uint8_t*>(p.dz + tl.m0);
  cols_operand<TM, BK>(oa, false, tl.m0, p.ld, w, lane);
  ob.stride = p.k * 2;
  ob.rsrc = bg_rsrc(p.h, p.rows * p.k * 2);
  cols_operand<TN, BK>(ob, true, tl.n0, p.k, w, lane);
  const int vs = (int)min((int64_t)TM, (p.width - tl.m0 + 63) / 64), nst = (int)((count + BK - 1) / BK);
  const TileParams a = {p.row_index, p.rows};
  tile_sums<BG_WGRAD, TM, TN, BK, 1>(a, tl, oa, ob, lds, vs, nst, 0, w, lane, [&](auto& acc) {
    constexpr int VS = sizeof(acc) / sizeof(acc[0]);
    auto row = [&](int r) { return tl.m0 + r < p.width ? p.v0 + tl.m0 + r : (int64_t)-1; };
    const int64_t col0 = tl.n0 + 32 * TN * (w & 1);
    if (p.dw_bf) store_tile<VS, TN, true>(acc, lds, p.dw, p.add, p.k, col0, w, lane, row);
    else store_tile<VS, TN, false>(acc, lds, p.dw, p.add, p.k, col0, w, lane, row);
  });
}

// ------------------------------------------------------------------- ends --

constexpr int JOIN_ROWS = 16;  // rows of a block, 64 threads each
__global__ __launch_bounds__(1024) void vocab_join_kernel(VocabArgs p, int64_t tiles) {
  __shared__ float2 s_part[64][JOIN_ROWS];
  const int r = threadIdx.x % JOIN_ROWS, sl = threadIdx.x / JOIN_ROWS;
  const int64_t count = *p.count, row = (int64_t)blockIdx.x * JOIN_ROWS + r;
  // rows without a target, by their own index
  if (sl == 0 && row < p.rows && !has_target(p, row)) p.loss[row] = p.lse[row] = 0.0f;
  auto add = [](float2& a, float2 b) {
    if (a.x == b.x || b.y == 0.0f) {  // the usual case: one reference
      a.y += b.y;
    } else {
      const float top = __builtin_fmaxf(a.x, b.x);
      a.y = (a.y == 0.0f ? 0.0f : a.y * __builtin_amdgcn_exp2f(a.x - top)) + b.y * __builtin_amdgcn_exp2f(b.x - top);
      a.x = top;
    }
  };
  float2 sum = make_float2(0.0f, 0.0f);
  if (row < count) {
    sum.x = p.ref[p.row_index[row]];
#pragma unroll 4
    for (int64_t t = sl; t < tiles; t += 64) add(sum, p.part[t * p.rows + row]);
  }
  s_part[sl][r] = sum;
  __syncthreads();
  for (int o = 32; o >= 1; o >>= 1) {
    if (sl < o) {
      add(sum, s_part[sl + o][r]);
      s_part[sl][r] = sum;
    }
    __syncthreads();
  }
  if (sl == 0 && row < count) {
    const int32_t at = p.row_index[row];
    const float ref = p.ref[at], l = __builtin_log2f(sum.y);
    p.lse[at] = (sum.x + l) * LN2;
    p.loss[at] = ((sum.x - ref) + l) * LN2;
  }
}

// dh of every row: its splits' sums added in order, zeros without a target
__global__ __launch_bounds__(256) void vocab_dh_join_kernel(VocabArgs p) {
  const int64_t slots = p.k / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.rows * slots; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / slots, e = 8 * (i % slots);
    const int32_t at = p.number[row];
    f32x4 a = {0, 0, 0, 0}, b = a;
    if (at >= 0)
      for (int s = 0; s < p.splits; ++s) {
        const f32x4* q = reinterpret_cast<const f32x4*>(p.sums + ((int64_t)s * p.rows + at) * p.k + e);
        a += q[0];
        b += q[1];
      }
    const u32x4 o = {pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3])};
    __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(p.dh + row * p.k + e));
  }
}

// ------------------------------------------------------------------- host --

static int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }
static int64_t tiles_of(int64_t rows, int64_t cols, int TM, int TN) {
  return ((rows + 64 * TM - 1) / (64 * TM)) * ((cols + 64 * TN - 1) / (64 * TN));
}
static dim3 tile_grid(int64_t tiles) { return dim3((unsigned)(8 * (tiles / 8 + 1))); }

// Columns (in 64s) of a tile of the logits.
static int logits_tn(int64_t rows) { return rows > 128 ? 4 : 2; }
static int64_t forward_tiles(int64_t rows, int64_t vocab) { return (vocab + 64 * logits_tn(rows) - 1) / (64 * logits_tn(rows)); }

template <bool DZ>
static void launch_logits(const VocabArgs& p, hipStream_t str) {
  if (p.rows > 128)
    hipLaunchKernelGGL((vocab_logits_kernel<4, 4, DZ>), tile_grid(tiles_of(p.rows, p.width, 4, 4)), dim3(256), 0, str, p);
  else if (p.rows > 64)
    hipLaunchKernelGGL((vocab_logits_kernel<2, 2, DZ>), tile_grid(tiles_of(p.rows, p.width, 2, 2)), dim3(256), 0, str, p);
  else
    hipLaunchKernelGGL((vocab_logits_kernel<1, 2, DZ>), tile_grid(tiles_of(p.rows, p.width, 1, 2)), dim3(256), 0, str, p);
}

// The pieces of the vocabulary in the backward pass and the splits of dh.
struct VocabPlan {
  int64_t width, ld, pieces, splits, per_split;
};
static VocabPlan vocab_plan(int64_t rows, int64_t vocab, int64_t k) {
  VocabPlan q;
  // dz of a piece stays below 128 MB, so that it is still in the memory-side
  // cache when the two products read it
  int64_t most = ((int64_t)1 << 26) / (rows > 0 ? rows : 1);
  most = most < 2048 ? 2048 : most;
  q.pieces = (vocab + most - 1) / most;
  q.pieces = q.pieces < 1 ? 1 : q.pieces;
  q.width = up((vocab + q.pieces - 1) / q.pieces, 256);
  q.width = q.width < 256 ? 256 : q.width;
  q.pieces = (vocab + q.width - 1) / q.width;
  q.pieces = q.pieces < 1 ? 1 : q.pieces;
  q.ld = q.width;
  const int64_t tiles = rows > 64 ? tiles_of(rows, k, 2, 4) : tiles_of(rows, k, 1, 2);
  q.splits = tiles > 0 && tiles < 256 ? (512 + tiles - 1) / tiles : 1;
  const int64_t room = q.width / 512 > 0 ? q.width / 512 : 1;  // a split sums 512 rows of w at least
  q.splits = q.splits < room ? q.splits : room;
  q.per_split = up((q.width + q.splits - 1) / q.splits, 64);
  return q;
}

static int64_t forward_bytes(int64_t rows, int64_t vocab) {
  return 16 + up(rows, 4) * 4 * 2 + forward_tiles(rows, vocab) * rows * 8;
}
static int64_t backward_bytes(int64_t rows, int64_t vocab, int64_t k) {
  const VocabPlan q = vocab_plan(rows, vocab, k);
  return 16 + up(rows, 4) * 4 * 5 + up(rows * q.ld * 2, 16) + q.splits * rows * k * 4;
}

}  // namespace nvfp4

using nvfp4host::aligned;

static int vocab_sizes(int64_t rows, int64_t vocab, int64_t k, float scale) {
  if (rows < 0 || vocab < 0 || k < 0 || !(scale - scale == 0.0f)) return NVFP4_ERROR_INVALID_VALUE;
  const int64_t lim = (int64_t)1 << 31;
  if (k % 8 != 0 || k > ((int64_t)1 << 20) || vocab > ((int64_t)1 << 24)) return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  if (rows >= lim || rows * (k > 0 ? k : 1) * 2 >= lim) return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  return NVFP4_SUCCESS;
}

extern "C" int64_t nvfp4_vocab_loss_workspace(int64_t rows, int64_t vocab, int64_t k) {
  return rows <= 0 || vocab_sizes(rows, vocab, k, 1.0f) ? 0 : nvfp4::forward_bytes(rows, vocab);
}

extern "C" int nvfp4_vocab_loss(const uint16_t* h, const uint16_t* w, const int32_t* targets, int64_t rows,
                                int64_t vocab, int64_t k, float scale, float* loss, float* lse, void* workspace,
                                int64_t workspace_bytes, void* stream) {
  int st = vocab_sizes(rows, vocab, k, scale);
  if (st) return st;
  if (rows == 0) return NVFP4_SUCCESS;
  if (!targets || !loss || !lse || (k > 0 && (!h || (vocab > 0 && !w)))) return NVFP4_ERROR_INVALID_VALUE;
  if (!workspace || workspace_bytes < nvfp4_vocab_loss_workspace(rows, vocab, k)) return NVFP4_ERROR_INVALID_VALUE;
  if (!nvfp4::tile_grid_ok(rows, 0, vocab)) return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  if (!aligned(h, 16) || !aligned(w, 16) || !aligned(targets, 4) || !aligned(loss, 4) || !aligned(lse, 4) ||
      !aligned(workspace, 16))
    return NVFP4_ERROR_MISALIGNED;
  if ((st = nvfp4host::check_arch())) return st;
  nvfp4::VocabArgs p{};
  p.h = h; p.w = w; p.targets = targets; p.rows = rows; p.vocab = vocab; p.k = k; p.scale = scale;
  p.loss = loss; p.lse = lse; p.width = vocab;
  int32_t* ws = static_cast<int32_t*>(workspace);
  const int64_t list = nvfp4::up(rows, 4);
  p.count = ws;
  p.row_index = ws + 4;
  p.ref = reinterpret_cast<float*>(ws + 4 + list);
  p.part = reinterpret_cast<float2*>(ws + 4 + 2 * list);
  hipStream_t str = (hipStream_t)stream;
  const int64_t cap = (int64_t)nvfp4host::num_cus() * 4, dots = (rows + 15) / 16;
  hipLaunchKernelGGL(nvfp4::vocab_rows_kernel, dim3((unsigned)(1 + (dots < cap ? dots : cap))), dim3(1024), 0, str, p);
  if (vocab > 0) nvfp4::launch_logits<false>(p, str);
  hipLaunchKernelGGL(nvfp4::vocab_join_kernel, dim3((unsigned)((rows + nvfp4::JOIN_ROWS - 1) / nvfp4::JOIN_ROWS)),
                     dim3(1024), 0, str, p, nvfp4::forward_tiles(rows, vocab));
  return nvfp4host::launch_status();
}

extern "C" int64_t nvfp4_vocab_loss_backward_workspace(int64_t rows, int64_t vocab, int64_t k) {
  return vocab_sizes(rows, vocab, k, 1.0f) ? 0 : nvfp4::backward_bytes(rows, vocab, k);
}

extern "C" int nvfp4_vocab_loss_backward(const uint16_t* h, const uint16_t* w, const int32_t* targets,
                                         const float* lse, const float* d_loss, int64_t rows, int64_t vocab, int64_t k,
                                         float scale, const void* add, uint16_t* dh, void* dw, int dw_type,
                                         void* workspace, int64_t workspace_bytes, void* stream) {
  if (dw_type != NVFP4_TYPE_F32 && dw_type != NVFP4_TYPE_BF16) return NVFP4_ERROR_INVALID_VALUE;
  int st = vocab_sizes(rows, vocab, k, scale);
  if (st) return st;
  if (!dh && !dw) return NVFP4_ERROR_INVALID_VALUE;
  if (k == 0 || (rows == 0 && (vocab == 0 || !dw))) return NVFP4_SUCCESS;
  if (rows > 0 && (!h || !targets || !lse || !d_loss)) return NVFP4_ERROR_INVALID_VALUE;
  if (vocab > 0 && !w) return NVFP4_ERROR_INVALID_VALUE;
  if (!workspace || workspace_bytes < nvfp4_vocab_loss_backward_workspace(rows, vocab, k)) return NVFP4_ERROR_INVALID_VALUE;
  if (!nvfp4::tile_grid_ok(rows, 0, vocab) || !nvfp4::tile_grid_ok(vocab, 0, k) || !nvfp4::tile_grid_ok(rows, 0, k))
    return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  if (!aligned(h, 16) || !aligned(w, 16) || !aligned(targets, 4) || !aligned(lse, 4) || !aligned(d_loss, 4) ||
      !aligned(add, 16) || !aligned(dh, 16) || !aligned(dw, 16) || !aligned(workspace, 16))
    return NVFP4_ERROR_MISALIGNED;
  if ((st = nvfp4host::check_arch())) return st;
  const nvfp4::VocabPlan q = nvfp4::vocab_plan(rows, vocab, k);
  nvfp4::VocabArgs p{};
  p.h = h; p.w = w; p.targets = targets; p.rows = rows; p.vocab = vocab; p.k = k; p.scale = scale;
  p.lse_in = lse; p.d_loss = d_loss; p.add = add; p.dh = dh; p.dw = dw; p.dw_bf = dw_type == NVFP4_TYPE_BF16;
  int32_t* ws = static_cast<int32_t*>(workspace);
  const int64_t list = nvfp4::up(rows, 4);
  p.count = ws;
  p.row_index = ws + 4;
  p.number = p.row_index + list;
  p.target = p.number + list;
  p.ref = reinterpret_cast<float*>(p.target + list);
  p.coef = p.ref + list;
  p.dz = reinterpret_cast<uint16_t*>(p.coef + list);
  p.sums = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(p.dz) + nvfp4::up(rows * q.ld * 2, 16));
  p.splits = (int)q.splits;
  p.per_split = q.per_split;
  hipStream_t str = (hipStream_t)stream;
  hipLaunchKernelGGL(nvfp4::vocab_rows_kernel, dim3(1), dim3(1024), 0, str, p);
  for (int64_t v0 = 0; v0 < vocab; v0 += q.width) {
    p.v0 = v0;
    p.width = vocab - v0 < q.width ? vocab - v0 : q.width;
    p.ld = nvfp4::up(p.width, 8);
    p.first = v0 == 0;
    if (rows > 0) nvfp4::launch_logits<true>(p, str);
    if (dh && rows > 0) {
      if (rows > 64)
        hipLaunchKernelGGL((nvfp4::vocab_dh_kernel<2, 4, 32>),
                           nvfp4::tile_grid(nvfp4::tiles_of(rows, k, 2, 4) * q.splits), dim3(256), 0, str, p);
      else
        hipLaunchKernelGGL((nvfp4::vocab_dh_kernel<1, 2, 64>),
                           nvfp4::tile_grid(nvfp4::tiles_of(rows, k, 1, 2) * q.splits), dim3(256), 0, str, p);
    }
    if (dw)
      hipLaunchKernelGGL((nvfp4::vocab_dw_kernel<4, 2, 32>), nvfp4::tile_grid(nvfp4::tiles_of(p.width, k, 4, 2)),
                         dim3(256), 0, str, p);
  }
  if (dh && rows > 0) {
    const int64_t blocks = (rows * (k / 8) + 255) / 256;
    if (vocab == 0) p.splits = 0;
    hipLaunchKernelGGL(nvfp4::vocab_dh_join_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, str, p);
  }
  return nvfp4host::launch_status();
}
