// residual_norm.hip -- RMS norms after and before a block, fused with the
// block's gate, the residual sum and the per-token NVFP4 quantization of the
// normed rows, and their backward pass (gfx950).
//
// Forward, for a block output b, residual r, gate g, scale a (all optional
// parts left out act as 1, or 0 for r):
//   n  = b rho1 w1,       rho1 = 1 / sqrt(mean(b^2) + eps)
//   r' = round(r + a g n)                (to the residual's type)
//   h  = bf16(r' rho2 w2), rho2 = 1 / sqrt(mean(r'^2) + eps), of the rounded r'
// Backward, from dh and dr' (the rounding of r' passes gradients unchanged):
//   t  = dr' + rho2 (w2 dh) - r' rho2^3 / d sum(w2 dh r')       dr = t
//   dn = a g t,  dg = a n t,  db = rho1 (w1 dn) - b rho1^3 / d sum(w1 dn b)
//   dw1 = sum_rows dn b rho1,  dw2 = sum_rows dh r' rho2
//
// HBM-bound: every row is read once and stays in registers (W = ceil(d / 512)
// waves hold 8 elements a thread, 16 past d = 8192).  The parameters are the
// same for every row, so a block keeps them in registers and walks rows; the
// next row's loads are issued before the current row's reductions.  Rows of
// 512 to 8192 come near the card's copy rate of 6.1 TB/s (16384 x 2560, fp32
// block output, bf16 residual, post norm, channel gate: forward 73 to 76 us, 5.6
// TB/s, 82 with the NVFP4 rows too; backward 114 to 117 us, 5.1 TB/s).  The
// backward pass keeps its column sums in registers too, and writes one
// partial row per block, which a second kernel adds in block order (no
// atomics: the same bits on every call).
#include "quant_rows.h"
#include "rowwise.h"

namespace nvfp4 {

struct NormArgs {
  const void *x, *residual, *post_w, *gate, *norm_w;
  void* r_out;
  uint16_t* h;
  float* amax;
  uint8_t *q, *sb;
  float* s;
  int64_t rows, d;
  float scale, eps, inv_d;
  bool x_bf, r_bf, p_bf;
  bool gate_rows;  // gate [rows, d], else [d]
  // backward
  const void *dh, *dr;
  void *dx, *dr_out, *dgate;
  bool dx_bf;
  float* part;  // [grid][2][d]: partial column sums
  float *dw1, *dw2, *dg;
};

// (mean + eps)^-1/2 within 2 ulp (the hardware's 1 ulp reciprocal root; below
// the normal range the correctly rounded operations)
__device__ __forceinline__ float rho_of(float sumsq, float inv_d, float eps) {
  const float v = __builtin_fmaf(sumsq, inv_d, eps);
  return v >= 0x1p-100f ? __builtin_amdgcn_rsqf(v) : 1.0f / __builtin_sqrtf(v);
}

// How a kernel reads its rows: KIND 0 element by element with types known at
// run time (any width and alignment), KIND 1 + x + 2 r in 16-byte pieces, x
// and r telling whether x and the residual are bf16.
template <int KIND>
struct Rows {
  static constexpr bool vec = KIND > 0;
  static __device__ __forceinline__ bool x_bf(const NormArgs& p) { return KIND ? ((KIND - 1) & 1) != 0 : p.x_bf; }
  static __device__ __forceinline__ bool r_bf(const NormArgs& p) { return KIND ? ((KIND - 1) & 2) != 0 : p.r_bf; }
};

// One slot of every row operand of a row: raw when it is fetched ahead.
struct NormSlots {
  RawSlot x, r, g, dh, dr;
};

template <int NV, int KIND, int MAXT>
__global__ __launch_bounds__(MAXT) void norm_forward_kernel(NormArgs p) {
  typedef Rows<KIND> R;
  constexpr bool VEC = R::vec;
  __shared__ BlockSums<1> sums;
  __shared__ uint32_t smax[2][16];
  const int T = blockDim.x, tid = threadIdx.x, W = T >> 6;
  const int64_t d = p.d;
  const bool xb = R::x_bf(p), rb = R::r_bf(p);
  float w1[NV][8], w2[NV][8], gc[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (p.post_w) load8<VEC>(p.post_w, p.p_bf, d, v, T, tid, w1[v]);
    if (p.norm_w) load8<VEC>(p.norm_w, p.p_bf, d, v, T, tid, w2[v]);
    if (p.gate && !p.gate_rows) load8<VEC>(p.gate, p.p_bf, d, v, T, tid, gc[v]);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) gc[v][i] = 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) gc[v][i] *= p.scale;
  }
  NormSlots nx[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      load_raw(row_at(p.x, xb, row, d), xb, d, v, T, tid, nx[v].x);
      if (p.residual) load_raw(row_at(p.residual, rb, row, d), rb, d, v, T, tid, nx[v].r);
      if (p.gate_rows) load_raw(row_at(p.gate, p.p_bf, row, d), p.p_bf, d, v, T, tid, nx[v].g);
    }
  };
  if (VEC) fetch(blockIdx.x);
  int slot = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    float b[NV][8], r[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[v][i] = 0.0f;
      if (VEC) {
        decode_raw(nx[v].x, xb, b[v]);
        if (p.residual) decode_raw(nx[v].r, rb, r[v]);
        if (p.gate_rows) decode_raw(nx[v].g, p.p_bf, gc[v]);
      } else {
        load8<false>(row_at(p.x, xb, row, d), xb, d, v, T, tid, b[v]);
        if (p.residual) load8<false>(row_at(p.residual, rb, row, d), rb, d, v, T, tid, r[v]);
        if (p.gate_rows) load8<false>(row_at(p.gate, p.p_bf, row, d), p.p_bf, d, v, T, tid, gc[v]);
      }
      if (p.gate_rows) {
#pragma unroll
        for (int i = 0; i < 8; ++i) gc[v][i] *= p.scale;
      }
    }
    if (VEC && row + gridDim.x < p.rows) fetch(row + gridDim.x);
    if (p.post_w) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = __builtin_fmaf(b[v][i], b[v][i], ss[0]);
      block_sum<1>(ss, W, slot, sums);
      slot ^= 1;
      const float rho = rho_of(ss[0], p.inv_d, p.eps);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) b[v][i] = b[v][i] * rho * w1[v][i];
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[v][i] = __builtin_fmaf(gc[v][i], b[v][i], r[v][i]);
        if (rb) r[v][i] = bf16_to_f32(to_bf16(r[v][i]));
      }
      if (p.r_out) store8<VEC>(row_at(p.r_out, rb, row, d), rb, d, v, T, tid, r[v]);
    }
    if (!p.norm_w) continue;
    float ss[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[0] = __builtin_fmaf(r[v][i], r[v][i], ss[0]);
    block_sum<1>(ss, W, slot, sums);
    const float rho = rho_of(ss[0], p.inv_d, p.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[v][i] = r[v][i] * rho * w2[v][i];
      if (p.h) store8<VEC>(p.h + row * d, true, d, v, T, tid, r[v]);
    }
    if (p.amax || p.s) {
      uint32_t m = 0, bm[NV];
      uint4 hb[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        hb[v] = make_uint4(pack_bf16(r[v][0], r[v][1]), pack_bf16(r[v][2], r[v][3]), pack_bf16(r[v][4], r[v][5]),
                           pack_bf16(r[v][6], r[v][7]));
        bm[v] = half_amax_bits(hb[v]);
        m = max(m, bm[v]);
      }
      m = group_max_u32<64>(m);
      if (W > 1) {
        if ((tid & 63) == 0) smax[slot][tid >> 6] = m;
        __syncthreads();
        m = 0;
        for (int k = 0; k < W; ++k) m = max(m, smax[slot][k]);
      }
      const float amax = __uint_as_float(m << 16);
      if (p.amax && tid == 0) p.amax[row] = amax;
      if (VEC && p.s) {  // d % 16 == 0: a block of 16 is a pair of lanes
        const RowScale rs = row_scale(amax);
        if (tid == 0) p.s[row] = rs.S;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          uint32_t code;
          float inv;
          block_scale(pair_max(bm[v]), rs, code, inv);
          const int64_t e = slot_elem<true>(v, 0, T, tid);
          if (e < d) {
            reinterpret_cast<uint32_t*>(p.q + row * (d / 2))[e / 8] = encode_half(hb[v], inv);
            if (!(tid & 1)) p.sb[row * (d / 16) + e / 16] = (uint8_t)code;
          }
        }
      }
    }
    slot ^= 1;
  }
}

// One pass, one reduction a row.  With q = a g w1 (a constant of a column) the
// sum that db needs, sum(w1 dn b), splits into sums that need none of the
// row's other results:
//   sum(w1 dn b) = A + rho2 B - c2 C,   A = sum(q b dr'), B = sum(q b w2 dh),
//   C = sum(q b r'),   c2 = rho2^3 / d sum(w2 dh r')
// so all six sums of a row (with sum b^2, sum r'^2) meet in one exchange.
// For a gate of the columns, dw1 and dg are both multiples of the column sums
// of t b rho1: one running sum a column serves both.
// A row's chain of dependent work, not its bytes, is what the waves of a CU
// have to hide: with two exchanges, divisions and branches for every optional
// part a row took about 3 us and 16384 x 2560 rows 250 us.  PLAIN: post and
// next norm, both gradients, no gate by rows, known when compiled, and at
// most 128 registers (four waves a SIMD).  The other forms are slower (16384 x
// 2560 without post norm and gate 193 us against 117), and 1024 threads leave
// them 128 registers too: they spill 1 to 27 of them for 4096 < d <= 8192 and
// 96 to 135 beyond, where PLAIN spills 3 to 10.
template <int NV, int KIND, int MAXT, bool PLAIN>
__global__ __launch_bounds__(MAXT, PLAIN || MAXT > 512 ? 4 : 3) void norm_backward_kernel(NormArgs p) {
  typedef Rows<KIND> R;
  constexpr bool VEC = R::vec;
  constexpr bool AHEAD = VEC && NV == 1;  // registers to fetch a row ahead
  __shared__ BlockSums<6> sums;
  const int T = blockDim.x, tid = threadIdx.x, W = T >> 6;
  const int64_t d = p.d;
  const bool xb = R::x_bf(p), rb = R::r_bf(p);
  const bool post = PLAIN || p.post_w, norm = PLAIN || p.norm_w, dr = PLAIN || p.dr, by_row = !PLAIN && p.gate_rows;
  // w2 and q (by rows: a w1) of this thread's columns: in registers, or past
  // d = 8192 in LDS, where each thread reads back what it wrote itself (with
  // them in registers too, 2048 x 16384 spilled and took 220 us)
  __shared__ f32x4 s_par[NV > 1 ? 4 * NV * MAXT : 1];
  float w2r[8], qr[8], a1[NV][8], a2[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a1[v][i] = a2[v][i] = 0.0f;
      w2r[i] = qr[i] = g[i] = 1.0f;
    }
    if (norm) load8<VEC>(p.norm_w, p.p_bf, d, v, T, tid, w2r);
    if (post) load8<VEC>(p.post_w, p.p_bf, d, v, T, tid, qr);
    if (p.gate && !by_row) load8<VEC>(p.gate, p.p_bf, d, v, T, tid, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) qr[i] *= g[i] * p.scale;
    if (NV > 1) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        s_par[(4 * v + k) * MAXT + tid] = (f32x4){w2r[4 * k], w2r[4 * k + 1], w2r[4 * k + 2], w2r[4 * k + 3]};
        s_par[(4 * v + 2 + k) * MAXT + tid] = (f32x4){qr[4 * k], qr[4 * k + 1], qr[4 * k + 2], qr[4 * k + 3]};
      }
    }
  }
  auto params = [&](int v, float (&w2)[8], float (&q)[8]) {
    if (NV > 1) asm volatile("" ::: "memory");  // read here, not kept in registers over the rows
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w2[i] = NV > 1 ? s_par[(4 * v + i / 4) * MAXT + tid][i % 4] : w2r[i];
      q[i] = NV > 1 ? s_par[(4 * v + 2 + i / 4) * MAXT + tid][i % 4] : qr[i];
    }
  };
  NormSlots nx[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      load_raw(row_at(p.x, xb, row, d), xb, d, v, T, tid, nx[v].x);
      if (norm) {
        load_raw(row_at(p.residual, rb, row, d), rb, d, v, T, tid, nx[v].r);
        load_raw(row_at(p.dh, true, row, d), true, d, v, T, tid, nx[v].dh);
      }
      if (dr) load_raw(row_at(p.dr, rb, row, d), rb, d, v, T, tid, nx[v].dr);
      if (by_row) load_raw(row_at(p.gate, p.p_bf, row, d), p.p_bf, d, v, T, tid, nx[v].g);
    }
  };
  if (AHEAD) fetch(blockIdx.x);
  int slot = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, slot ^= 1) {
    float b[NV][8], r[NV][8], dh[NV][8], t[NV][8], g[NV][8];
    if (VEC && !AHEAD) fetch(row);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!norm) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[v][i] = dh[v][i] = 0.0f;
      }
      if (!dr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[v][i] = 0.0f;
      }
      if (VEC) {
        decode_raw(nx[v].x, xb, b[v]);
        if (norm) {
          decode_raw(nx[v].r, rb, r[v]);
          decode_raw(nx[v].dh, true, dh[v]);
        }
        if (dr) decode_raw(nx[v].dr, rb, t[v]);
        if (by_row) decode_raw(nx[v].g, p.p_bf, g[v]);
      } else {
        load8<false>(row_at(p.x, xb, row, d), xb, d, v, T, tid, b[v]);
        if (norm) {
          load8<false>(row_at(p.residual, rb, row, d), rb, d, v, T, tid, r[v]);
          load8<false>(row_at(p.dh, true, row, d), true, d, v, T, tid, dh[v]);
        }
        if (dr) load8<false>(row_at(p.dr, rb, row, d), rb, d, v, T, tid, t[v]);
        if (by_row) load8<false>(row_at(p.gate, p.p_bf, row, d), p.p_bf, d, v, T, tid, g[v]);
      }
    }
    if (AHEAD && row + gridDim.x < p.rows) fetch(row + gridDim.x);
    float ss[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float w2[8], q[8];
      params(v, w2, q);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float up = dh[v][i] * w2[i];
        float qb = q[i] * b[v][i];
        if (by_row) qb *= g[v][i];
        ss[0] = __builtin_fmaf(b[v][i], b[v][i], ss[0]);
        ss[1] = __builtin_fmaf(r[v][i], r[v][i], ss[1]);
        ss[2] = __builtin_fmaf(up, r[v][i], ss[2]);
        ss[3] = __builtin_fmaf(qb, t[v][i], ss[3]);
        ss[4] = __builtin_fmaf(qb, up, ss[4]);
        ss[5] = __builtin_fmaf(qb, r[v][i], ss[5]);
      }
    }
    block_sum<6>(ss, W, slot, sums);
    const float rho1 = post ? rho_of(ss[0], p.inv_d, p.eps) : 1.0f;
    const float rho2 = norm ? rho_of(ss[1], p.inv_d, p.eps) : 0.0f;
    // one rho at a time: a bare rho^3 leaves fp32 for rows of about 1e13 and
    // 1e-13, long before their squares do
    const float c2 = rho2 * (rho2 * (rho2 * (ss[2] * p.inv_d)));
    const float s1 = __builtin_fmaf(-c2, ss[5], __builtin_fmaf(rho2, ss[4], ss[3]));
    const float c1 = post ? rho1 * (rho1 * (s1 * p.inv_d)) : 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float o[8], dg[8], w2[8], q[8];
      params(v, w2, q);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (norm) {
          const float up = dh[v][i] * w2[i];
          a2[v][i] = __builtin_fmaf(dh[v][i], r[v][i] * rho2, a2[v][i]);
          t[v][i] = __builtin_fmaf(-r[v][i], c2, __builtin_fmaf(rho2, up, t[v][i]));
        }
        const float tn = t[v][i] * (b[v][i] * rho1);
        float m = q[i] * t[v][i];
        if (by_row) {
          m *= g[v][i];
          dg[i] = q[i] * tn;  // q is a w1 here
          a1[v][i] = __builtin_fmaf(g[v][i], tn, a1[v][i]);
        } else {
          a1[v][i] += tn;
        }
        o[i] = rho1 * __builtin_fmaf(-b[v][i], c1, m);
      }
      if (VEC) {
        if (p.dr_out) store_raw(row_at(p.dr_out, rb, row, d), rb, d, v, T, tid, t[v]);
        store_raw(row_at(p.dx, p.dx_bf, row, d), p.dx_bf, d, v, T, tid, o);
        if (by_row && p.dgate) store_raw(row_at(p.dgate, p.p_bf, row, d), p.p_bf, d, v, T, tid, dg);
      } else {
        if (p.dr_out) store8<false>(row_at(p.dr_out, rb, row, d), rb, d, v, T, tid, t[v]);
        store8<false>(row_at(p.dx, p.dx_bf, row, d), p.dx_bf, d, v, T, tid, o);
        if (by_row && p.dgate) store8<false>(row_at(p.dgate, p.p_bf, row, d), p.p_bf, d, v, T, tid, dg);
      }
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (p.dw1 || p.dg) store8<VEC>(part, false, d, v, T, tid, a1[v]);
    if (p.dw2) store8<VEC>(part + d, false, d, v, T, tid, a2[v]);
  }
}

// Column sums of the blocks' partial rows in a fixed order: 64 columns a
// block, 16 waves each over a sixteenth of the partial rows (8 loads in
// flight), their sums added in order, and the columns' constants applied.
__global__ __launch_bounds__(1024) void norm_columns_kernel(NormArgs p, int blocks) {
  __shared__ float red[16][64];
  const int which = blockIdx.y;  // 0: sums of t b rho1, 1: of dh r' rho2
  if (which == 0 ? !(p.dw1 || p.dg) : !p.dw2) return;
  const int lane = threadIdx.x & 63, part = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  const int per = (blocks + 15) / 16, b0 = part * per, b1 = min(blocks, b0 + per);
  float sum = 0.0f;
  if (c < p.d) {
    const float* q = p.part + (int64_t)which * p.d + c;
    const int64_t step = 2 * p.d;
    int b = b0;
    for (; b + 8 <= b1; b += 8) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = q[(b + i) * step];
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[i];
    }
    for (; b < b1; ++b) sum += q[b * step];
  }
  red[part][lane] = sum;
  __syncthreads();
  if (part == 0 && c < p.d) {
    float t = 0.0f;
    for (int k = 0; k < 16; ++k) t += red[k][lane];
    if (which == 1) {
      p.dw2[c] = t;
      return;
    }
    auto at = [&](const void* w) {
      return p.p_bf ? bf16_to_f32(static_cast<const uint16_t*>(w)[c]) : static_cast<const float*>(w)[c];
    };
    const float st = p.scale * t;
    if (p.dw1) p.dw1[c] = p.gate && !p.gate_rows ? at(p.gate) * st : st;
    if (p.dg) p.dg[c] = p.post_w ? at(p.post_w) * st : st;
  }
}

constexpr int64_t NORM_MAX_D = 16384;

// waves that hold a row: 8 elements a thread up to d = 8192, then 16
static int norm_waves(int64_t d) {
  const int64_t per = d <= 8192 ? 512 : 1024;
  return (int)((d + per - 1) / per);
}

// Blocks of the backward pass: about ten waves a CU, since each block walks
// rows and leaves one partial row (16384 x 2560, fp32 x, bf16 residual: 1, 2, 3
// blocks a CU take 163, 118, 146 us, 4.97 TB/s at 2; 16384 x 1024: 106, 68, 58;
// 16384 x 4096: 166, 172, 176).
static int64_t norm_backward_blocks(int64_t rows, int64_t d) {
  const int64_t cap = (int64_t)nvfp4host::num_cus() * (norm_waves(d) <= 10 ? 10 / norm_waves(d) : 1);
  return rows < cap ? rows : cap;
}

template <int NV, int MAXT>
static void launch_forward(const NormArgs& p, int kind, dim3 grid, dim3 block, hipStream_t s) {
  switch (kind) {
    case 0: hipLaunchKernelGGL((norm_forward_kernel<NV, 0, MAXT>), grid, block, 0, s, p); break;
    case 1: hipLaunchKernelGGL((norm_forward_kernel<NV, 1, MAXT>), grid, block, 0, s, p); break;
    case 2: hipLaunchKernelGGL((norm_forward_kernel<NV, 2, MAXT>), grid, block, 0, s, p); break;
    case 3: hipLaunchKernelGGL((norm_forward_kernel<NV, 3, MAXT>), grid, block, 0, s, p); break;
    default: hipLaunchKernelGGL((norm_forward_kernel<NV, 4, MAXT>), grid, block, 0, s, p); break;
  }
}

template <int NV, int MAXT, bool PLAIN>
static void launch_backward(const NormArgs& p, int kind, dim3 grid, dim3 block, hipStream_t s) {
  switch (kind) {
    case 1: hipLaunchKernelGGL((norm_backward_kernel<NV, 1, MAXT, PLAIN>), grid, block, 0, s, p); break;
    case 2: hipLaunchKernelGGL((norm_backward_kernel<NV, 2, MAXT, PLAIN>), grid, block, 0, s, p); break;
    case 3: hipLaunchKernelGGL((norm_backward_kernel<NV, 3, MAXT, PLAIN>), grid, block, 0, s, p); break;
    case 4: hipLaunchKernelGGL((norm_backward_kernel<NV, 4, MAXT, PLAIN>), grid, block, 0, s, p); break;
    default: hipLaunchKernelGGL((norm_backward_kernel<NV, 0, MAXT, false>), grid, block, 0, s, p); break;
  }
}

static bool vec_rows(int64_t d, const void* const* ptrs, int n) {
  if (d % 8 != 0) return false;
  for (int i = 0; i < n; ++i)
    if (!nvfp4host::aligned(ptrs[i], 16)) return false;
  return true;
}

}  // namespace nvfp4

using nvfp4host::aligned;

static bool bad_type(int t) { return t != NVFP4_TYPE_F32 && t != NVFP4_TYPE_BF16; }
static bool bad_elem(const void* p, int t) { return !aligned(p, t == NVFP4_TYPE_BF16 ? 2 : 4); }

extern "C" int nvfp4_residual_norm(const void* x, int x_type, const void* residual, int residual_type,
                                   const void* post_weight, const void* gate, int gate_rows,
                                   const void* norm_weight, int param_type, int64_t rows, int64_t d,
                                   float scale, float eps, void* residual_out, uint16_t* h, float* amax,
                                   uint8_t* q, uint8_t* sb, float* s, void* stream) {
  if (rows < 0 || d < 1 || bad_type(x_type) || bad_type(residual_type) || bad_type(param_type))
    return NVFP4_ERROR_INVALID_VALUE;
  if (!(eps >= 0.0f) || !__builtin_isfinite(eps) || !__builtin_isfinite(scale)) return NVFP4_ERROR_INVALID_VALUE;
  if (d > nvfp4::NORM_MAX_D || (s && d % 16 != 0) || rows > ((int64_t)1 << 31)) return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  if (rows == 0) return NVFP4_SUCCESS;
  if (!x || (!q != !s) || (!sb != !s)) return NVFP4_ERROR_INVALID_VALUE;
  const bool wants_h = h || amax || s;
  if (!residual_out && !wants_h) return NVFP4_ERROR_INVALID_VALUE;
  if (wants_h && !norm_weight) return NVFP4_ERROR_INVALID_VALUE;
  if (gate_rows && !gate) return NVFP4_ERROR_INVALID_VALUE;
  if (bad_elem(x, x_type) || bad_elem(residual, residual_type) || bad_elem(residual_out, residual_type) ||
      bad_elem(post_weight, param_type) || bad_elem(gate, param_type) || bad_elem(norm_weight, param_type) ||
      !aligned(h, 2) || !aligned(amax, 4) || !aligned(s, 4) || (s && (!aligned(q, 16) || !aligned(x, 16))))
    return NVFP4_ERROR_MISALIGNED;
  const void* ptrs[] = {x, residual, post_weight, gate, norm_weight, residual_out, h};
  const bool vec = nvfp4::vec_rows(d, ptrs, 7);
  if (s && !vec) return NVFP4_ERROR_MISALIGNED;
  int st = nvfp4host::check_arch();
  if (st) return st;
#if NVFP4_CHECKED
  if (s || amax) {
    nvfp4check::Checks chk((hipStream_t)stream);
    auto finite = [&](const void* t, int type, int64_t n) {
      if (type == NVFP4_TYPE_BF16) chk.bf16_finite((const uint16_t*)t, n);
      else chk.f32_finite((const float*)t, n);
    };  // NULL: nothing to check
    finite(x, x_type, rows * d);
    finite(residual, residual_type, rows * d);
    finite(post_weight, param_type, d);
    finite(gate, param_type, gate_rows ? rows * d : d);
    finite(norm_weight, param_type, d);
    if ((st = chk.result())) return st;
  }
#endif
  nvfp4::NormArgs p{};
  p.x = x; p.residual = residual; p.post_w = post_weight; p.gate = gate; p.norm_w = wants_h ? norm_weight : nullptr;
  p.r_out = residual_out; p.h = h; p.amax = amax; p.q = q; p.sb = sb; p.s = s;
  p.rows = rows; p.d = d; p.scale = scale; p.eps = eps; p.inv_d = 1.0f / (float)d;
  p.x_bf = x_type == NVFP4_TYPE_BF16; p.r_bf = residual_type == NVFP4_TYPE_BF16;
  p.p_bf = param_type == NVFP4_TYPE_BF16; p.gate_rows = gate && gate_rows;
  const int W = nvfp4::norm_waves(d);
  // about 16 waves a CU (16384 x 2560, 2, 3, 4, 8 blocks a CU: 78, 76, 87, 86 us,
  // 5.5 TB/s at 3; 32768 x 512, 2, 4, 8, 16: 59, 35, 27, 26)
  const int64_t cap = (int64_t)nvfp4host::num_cus() * (16 / W);
  const dim3 grid((unsigned)(rows < cap ? rows : cap)), block(64 * W);
  hipStream_t str = (hipStream_t)stream;
  const int kind = vec ? 1 + (p.x_bf ? 1 : 0) + (p.r_bf ? 2 : 0) : 0;
  if (W <= 8) nvfp4::launch_forward<1, 512>(p, kind, grid, block, str);
  else if (d <= 8192) nvfp4::launch_forward<1, 1024>(p, kind, grid, block, str);
  else nvfp4::launch_forward<2, 1024>(p, kind, grid, block, str);
  return nvfp4host::launch_status();
}

extern "C" int64_t nvfp4_residual_norm_backward_workspace(int64_t rows, int64_t d) {
  if (rows < 1 || d < 1 || d > nvfp4::NORM_MAX_D) return 0;
  return nvfp4::norm_backward_blocks(rows, d) * 2 * d * (int64_t)sizeof(float);
}

extern "C" int nvfp4_residual_norm_backward(const void* x, int x_type, const void* residual_out, int residual_type,
                                            const void* post_weight, const void* gate, int gate_rows,
                                            const void* norm_weight, int param_type, const uint16_t* dh,
                                            const void* d_residual_out, int64_t rows, int64_t d, float scale,
                                            float eps, void* dx, int dx_type, void* d_residual, float* d_post_weight,
                                            void* d_gate, float* d_norm_weight, void* workspace,
                                            int64_t workspace_bytes, void* stream) {
  if (rows < 0 || d < 1 || bad_type(x_type) || bad_type(residual_type) || bad_type(param_type) || bad_type(dx_type))
    return NVFP4_ERROR_INVALID_VALUE;
  if (!(eps >= 0.0f) || !__builtin_isfinite(eps) || !__builtin_isfinite(scale)) return NVFP4_ERROR_INVALID_VALUE;
  if (d > nvfp4::NORM_MAX_D || rows > ((int64_t)1 << 31)) return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  if ((d_post_weight && !post_weight) || (d_norm_weight && !norm_weight) || (d_gate && !gate) || (gate_rows && !gate))
    return NVFP4_ERROR_INVALID_VALUE;
  const bool per_row_gate = gate && gate_rows;
  if (rows > 0 && (!x || !dx || (!dh && !d_residual_out))) return NVFP4_ERROR_INVALID_VALUE;
  if (rows > 0 && dh && (!norm_weight || !residual_out)) return NVFP4_ERROR_INVALID_VALUE;
  if (bad_elem(x, x_type) || bad_elem(residual_out, residual_type) || bad_elem(d_residual_out, residual_type) ||
      bad_elem(d_residual, residual_type) || bad_elem(post_weight, param_type) || bad_elem(gate, param_type) ||
      bad_elem(norm_weight, param_type) || !aligned(dh, 2) || bad_elem(dx, dx_type) || !aligned(d_post_weight, 4) ||
      !aligned(d_norm_weight, 4) || bad_elem(d_gate, per_row_gate ? param_type : NVFP4_TYPE_F32) ||
      !aligned(workspace, 16))
    return NVFP4_ERROR_MISALIGNED;
  nvfp4::NormArgs p{};
  p.x = x; p.residual = residual_out; p.post_w = post_weight; p.gate = gate; p.norm_w = dh ? norm_weight : nullptr;
  p.rows = rows; p.d = d; p.scale = scale; p.eps = eps; p.inv_d = 1.0f / (float)d;
  p.x_bf = x_type == NVFP4_TYPE_BF16; p.r_bf = residual_type == NVFP4_TYPE_BF16;
  p.p_bf = param_type == NVFP4_TYPE_BF16; p.gate_rows = per_row_gate;
  p.dh = dh; p.dr = d_residual_out; p.dx = dx; p.dx_bf = dx_type == NVFP4_TYPE_BF16; p.dr_out = d_residual;
  p.dgate = per_row_gate ? d_gate : nullptr;
  p.dw1 = d_post_weight; p.dw2 = d_norm_weight; p.dg = per_row_gate ? nullptr : (float*)d_gate;
  p.part = (float*)workspace;
  const bool columns = p.dw1 || p.dw2 || p.dg;
  if (rows == 0 && !columns) return NVFP4_SUCCESS;
  int st = nvfp4host::check_arch();
  if (st) return st;
  const int64_t blocks = rows > 0 ? nvfp4::norm_backward_blocks(rows, d) : 0;
  if (columns && rows > 0 && (!workspace || workspace_bytes < blocks * 2 * d * (int64_t)sizeof(float)))
    return NVFP4_ERROR_INVALID_VALUE;
  hipStream_t str = (hipStream_t)stream;
  if (rows > 0) {
    const void* ptrs[] = {x, residual_out, d_residual_out, d_residual, post_weight, gate, norm_weight, dh, dx, p.dgate};
    const bool vec = nvfp4::vec_rows(d, ptrs, 10);
    const int W = nvfp4::norm_waves(d);
    const dim3 grid((unsigned)blocks), block(64 * W);
    const int kind = vec ? 1 + (p.x_bf ? 1 : 0) + (p.r_bf ? 2 : 0) : 0;
    const bool plain = p.post_w && p.norm_w && p.dr && !p.gate_rows;
    if (W <= 8 && plain) nvfp4::launch_backward<1, 512, true>(p, kind, grid, block, str);
    else if (W <= 8) nvfp4::launch_backward<1, 512, false>(p, kind, grid, block, str);
    else if (d <= 8192 && plain) nvfp4::launch_backward<1, 1024, true>(p, kind, grid, block, str);
    else if (d <= 8192) nvfp4::launch_backward<1, 1024, false>(p, kind, grid, block, str);
    else if (plain) nvfp4::launch_backward<2, 1024, true>(p, kind, grid, block, str);
    else nvfp4::launch_backward<2, 1024, false>(p, kind, grid, block, str);
  }
  if (columns)
    hipLaunchKernelGGL(nvfp4::norm_columns_kernel, dim3((unsigned)((d + 63) / 64), 2), dim3(1024), 0, str, p,
                       (int)blocks);
  return nvfp4host::launch_status();
}
