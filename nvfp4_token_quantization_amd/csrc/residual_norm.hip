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
// next row's loads are issued before the current row's reductions.  The
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
  float scale, eps;
  bool x_bf, r_bf, p_bf;
  bool gate_rows;  // gate [rows, d], else [d]
  // backward
  const void *dh, *dr;
  void *dx, *dr_out, *dgate;
  bool dx_bf;
  float* part;  // [grid][3][d]: dw1, dw2, dg partial sums
  float *dw1, *dw2, *dg;
};

__device__ __forceinline__ float rho_of(float sumsq, float d, float eps) { return 1.0f / __builtin_sqrtf(sumsq / d + eps); }

template <int NV, bool VEC>
__global__ __launch_bounds__(1024) void norm_forward_kernel(NormArgs p) {
  __shared__ BlockSums<1> sums;
  __shared__ uint32_t smax[2][16];
  const int T = blockDim.x, tid = threadIdx.x, W = T >> 6;
  const int64_t d = p.d;
  const float fd = (float)d;
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
  int slot = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    float b[NV][8], r[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      load8<VEC>(row_at(p.x, p.x_bf, row, d), p.x_bf, d, v, T, tid, b[v]);
      if (p.residual) load8<VEC>(row_at(p.residual, p.r_bf, row, d), p.r_bf, d, v, T, tid, r[v]);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) r[v][i] = 0.0f;
      if (p.gate_rows) {
        float g[8];
        load8<VEC>(row_at(p.gate, p.p_bf, row, d), p.p_bf, d, v, T, tid, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) gc[v][i] = g[i] * p.scale;
      }
    }
    if (p.post_w) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = __builtin_fmaf(b[v][i], b[v][i], ss[0]);
      block_sum<1>(ss, W, slot, sums);
      slot ^= 1;
      const float rho = rho_of(ss[0], fd, p.eps);
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
        if (p.r_bf) r[v][i] = bf16_to_f32(to_bf16(r[v][i]));
      }
      if (p.r_out) store8<VEC>(row_at(p.r_out, p.r_bf, row, d), p.r_bf, d, v, T, tid, r[v]);
    }
    if (!p.norm_w) continue;
    float ss[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[0] = __builtin_fmaf(r[v][i], r[v][i], ss[0]);
    block_sum<1>(ss, W, slot, sums);
    const float rho = rho_of(ss[0], fd, p.eps);
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

template <int NV, bool VEC>
__global__ __launch_bounds__(1024) void norm_backward_kernel(NormArgs p) {
  __shared__ BlockSums<3> sums3;
  __shared__ BlockSums<1> sums1;
  const int T = blockDim.x, tid = threadIdx.x, W = T >> 6;
  const int64_t d = p.d;
  const float fd = (float)d;
  float w1[NV][8], w2[NV][8], gc[NV][8], a1[NV][8], a2[NV][8], ag[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a1[v][i] = a2[v][i] = ag[v][i] = 0.0f;
      w1[v][i] = w2[v][i] = gc[v][i] = 1.0f;
    }
    if (p.post_w) load8<VEC>(p.post_w, p.p_bf, d, v, T, tid, w1[v]);
    if (p.norm_w) load8<VEC>(p.norm_w, p.p_bf, d, v, T, tid, w2[v]);
    if (p.gate && !p.gate_rows) load8<VEC>(p.gate, p.p_bf, d, v, T, tid, gc[v]);
  }
  int slot = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, slot ^= 1) {
    float b[NV][8], r[NV][8], dh[NV][8], t[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) b[v][i] = r[v][i] = dh[v][i] = t[v][i] = 0.0f;
      load8<VEC>(row_at(p.x, p.x_bf, row, d), p.x_bf, d, v, T, tid, b[v]);
      if (p.norm_w) {
        load8<VEC>(row_at(p.residual, p.r_bf, row, d), p.r_bf, d, v, T, tid, r[v]);
        load8<VEC>(row_at(p.dh, true, row, d), true, d, v, T, tid, dh[v]);
      }
      if (p.dr) load8<VEC>(row_at(p.dr, p.r_bf, row, d), p.r_bf, d, v, T, tid, t[v]);
      if (p.gate_rows) load8<VEC>(row_at(p.gate, p.p_bf, row, d), p.p_bf, d, v, T, tid, gc[v]);
    }
    float ss[3] = {0.0f, 0.0f, 0.0f};  // sum b^2, sum r'^2, sum w2 dh r'
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss[0] = __builtin_fmaf(b[v][i], b[v][i], ss[0]);
        ss[1] = __builtin_fmaf(r[v][i], r[v][i], ss[1]);
        ss[2] = __builtin_fmaf(dh[v][i] * w2[v][i], r[v][i], ss[2]);
      }
    block_sum<3>(ss, W, slot, sums3);
    const float rho1 = p.post_w ? rho_of(ss[0], fd, p.eps) : 1.0f;
    if (p.norm_w) {
      const float rho2 = rho_of(ss[1], fd, p.eps);
      const float c2 = rho2 * rho2 * (ss[2] / fd);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a2[v][i] = __builtin_fmaf(dh[v][i], r[v][i] * rho2, a2[v][i]);
          t[v][i] = __builtin_fmaf(rho2, __builtin_fmaf(-r[v][i], c2, dh[v][i] * w2[v][i]), t[v][i]);
        }
    }
    float s1[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (p.dr_out) store8<VEC>(row_at(p.dr_out, p.r_bf, row, d), p.r_bf, d, v, T, tid, t[v]);
      float dgr[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n0 = b[v][i] * rho1;                 // n without its weight
        const float at = p.scale * t[v][i];
        dgr[i] = at * (n0 * w1[v][i]);
        ag[v][i] += dgr[i];
        const float dn = at * gc[v][i];
        a1[v][i] = __builtin_fmaf(dn, n0, a1[v][i]);
        t[v][i] = dn * w1[v][i];
        s1[0] = __builtin_fmaf(t[v][i], b[v][i], s1[0]);
      }
      if (p.gate_rows && p.dgate) store8<VEC>(row_at(p.dgate, p.p_bf, row, d), p.p_bf, d, v, T, tid, dgr);
    }
    if (p.post_w) {
      block_sum<1>(s1, W, slot, sums1);
      const float c1 = rho1 * rho1 * (s1[0] / fd);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) t[v][i] = rho1 * __builtin_fmaf(-b[v][i], c1, t[v][i]);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) store8<VEC>(row_at(p.dx, p.dx_bf, row, d), p.dx_bf, d, v, T, tid, t[v]);
  }
  float* part = p.part + (int64_t)blockIdx.x * 3 * d;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (p.dw1) store8<VEC>(part, false, d, v, T, tid, a1[v]);
    if (p.dw2) store8<VEC>(part + d, false, d, v, T, tid, a2[v]);
    if (p.dg) store8<VEC>(part + 2 * d, false, d, v, T, tid, ag[v]);
  }
}

// Column sums of the blocks' partial rows, in block order in fp32: 64 columns
// a block, 16 row ranges of the partials added in order at the end.
__global__ __launch_bounds__(1024) void norm_columns_kernel(NormArgs p, int blocks) {
  __shared__ float red[16][64];
  const int which = blockIdx.y;
  float* out = which == 0 ? p.dw1 : (which == 1 ? p.dw2 : p.dg);
  if (!out) return;
  const int lane = threadIdx.x & 63, part = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  const int per = (blocks + 15) / 16, b0 = part * per, b1 = min(blocks, b0 + per);
  float sum = 0.0f;
  if (c < p.d)
    for (int b = b0; b < b1; ++b) sum += p.part[((int64_t)b * 3 + which) * p.d + c];
  red[part][lane] = sum;
  __syncthreads();
  if (part == 0 && c < p.d) {
    float t = 0.0f;
    for (int k = 0; k < 16; ++k) t += red[k][lane];
    out[c] = t;
  }
}

constexpr int64_t NORM_MAX_D = 16384;

// waves that hold a row: 8 elements a thread up to d = 8192, then 16
static int norm_waves(int64_t d) {
  const int64_t per = d <= 8192 ? 512 : 1024;
  return (int)((d + per - 1) / per);
}

// blocks of the backward pass (each walks rows and leaves one partial row)
static int64_t norm_backward_blocks(int64_t rows, int64_t d) {
  const int64_t cap = (int64_t)nvfp4host::num_cus() * (norm_waves(d) <= 8 ? 4 : 2);
  return rows < cap ? rows : cap;
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
    if (x_type == NVFP4_TYPE_BF16) chk.bf16_finite((const uint16_t*)x, rows * d);
    else chk.f32_finite((const float*)x, rows * d);
    if (residual) {
      if (residual_type == NVFP4_TYPE_BF16) chk.bf16_finite((const uint16_t*)residual, rows * d);
      else chk.f32_finite((const float*)residual, rows * d);
    }
    if ((st = chk.result())) return st;
  }
#endif
  nvfp4::NormArgs p{};
  p.x = x; p.residual = residual; p.post_w = post_weight; p.gate = gate; p.norm_w = wants_h ? norm_weight : nullptr;
  p.r_out = residual_out; p.h = h; p.amax = amax; p.q = q; p.sb = sb; p.s = s;
  p.rows = rows; p.d = d; p.scale = scale; p.eps = eps;
  p.x_bf = x_type == NVFP4_TYPE_BF16; p.r_bf = residual_type == NVFP4_TYPE_BF16;
  p.p_bf = param_type == NVFP4_TYPE_BF16; p.gate_rows = gate && gate_rows;
  const int W = nvfp4::norm_waves(d);
  const int64_t cap = (int64_t)nvfp4host::num_cus() * (32 / W > 16 ? 16 : (32 / W < 2 ? 2 : 32 / W));
  const dim3 grid((unsigned)(rows < cap ? rows : cap)), block(64 * W);
  hipStream_t str = (hipStream_t)stream;
  if (d <= 8192) {
    if (vec) hipLaunchKernelGGL((nvfp4::norm_forward_kernel<1, true>), grid, block, 0, str, p);
    else hipLaunchKernelGGL((nvfp4::norm_forward_kernel<1, false>), grid, block, 0, str, p);
  } else {
    if (vec) hipLaunchKernelGGL((nvfp4::norm_forward_kernel<2, true>), grid, block, 0, str, p);
    else hipLaunchKernelGGL((nvfp4::norm_forward_kernel<2, false>), grid, block, 0, str, p);
  }
  return nvfp4host::launch_status();
}

extern "C" int64_t nvfp4_residual_norm_backward_workspace(int64_t rows, int64_t d) {
  if (rows < 1 || d < 1 || d > nvfp4::NORM_MAX_D) return 0;
  return nvfp4::norm_backward_blocks(rows, d) * 3 * d * (int64_t)sizeof(float);
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
  p.rows = rows; p.d = d; p.scale = scale; p.eps = eps;
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
  if (columns && rows > 0 && (!workspace || workspace_bytes < blocks * 3 * d * (int64_t)sizeof(float)))
    return NVFP4_ERROR_INVALID_VALUE;
  hipStream_t str = (hipStream_t)stream;
  if (rows > 0) {
    const void* ptrs[] = {x, residual_out, d_residual_out, d_residual, post_weight, gate, norm_weight, dh, dx, p.dgate};
    const bool vec = nvfp4::vec_rows(d, ptrs, 10);
    const dim3 grid((unsigned)blocks), block(64 * nvfp4::norm_waves(d));
    if (d <= 8192) {
      if (vec) hipLaunchKernelGGL((nvfp4::norm_backward_kernel<1, true>), grid, block, 0, str, p);
      else hipLaunchKernelGGL((nvfp4::norm_backward_kernel<1, false>), grid, block, 0, str, p);
    } else {
      if (vec) hipLaunchKernelGGL((nvfp4::norm_backward_kernel<2, true>), grid, block, 0, str, p);
      else hipLaunchKernelGGL((nvfp4::norm_backward_kernel<2, false>), grid, block, 0, str, p);
    }
  }
  if (columns)
    hipLaunchKernelGGL(nvfp4::norm_columns_kernel, dim3((unsigned)((d + 63) / 64), 3), dim3(1024), 0, str, p,
                       (int)blocks);
  return nvfp4host::launch_status();
}
