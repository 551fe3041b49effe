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
};

// One wave per 32 x 32 output tile, fragments gathered element by element.
template <int MODE>
__global__ __launch_bounds__(64) void bf16_simple_kernel(Bf16Args p) {
  const int lane = threadIdx.x, li = lane & 31, h = lane >> 5;
  const int e = blockIdx.y;
  const int64_t lo = min((int64_t)max(p.offsets[e], 0), p.m_total);
  const int64_t hi = min(max((int64_t)p.offsets[e + 1], lo), p.m_total);
  const int64_t N = MODE == BG_FORWARD ? p.n : p.k;          // output columns
  const int64_t M = MODE == BG_WGRAD ? p.n : hi - lo;        // output rows
  const int64_t K = MODE == BG_FORWARD ? p.k : (MODE == BG_DGRAD ? p.n : hi - lo);
  const int64_t c = (int64_t)blockIdx.x * 32 + li;
  for (int64_t m0 = (int64_t)blockIdx.z * 32; m0 < M; m0 += (int64_t)gridDim.z * 32) {
    const int64_t m = m0 + li;
    int64_t arow = -1;
    if (MODE != BG_WGRAD && m < M) arow = MODE == BG_FORWARD ? gathered_row(p.row_index, p.a_rows, lo + m, hi) : lo + m;
    f32x16 acc = {0};
    for (int64_t k0 = 0; k0 < K; k0 += 16) {
      bf16x8 fa, fb;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t kk = k0 + 8 * h + j;
        uint16_t va = 0, vb = 0;
        if (kk < K) {
          if (MODE == BG_FORWARD) {
            if (arow >= 0) va = p.a[arow * p.k + kk];
            if (c < N) vb = p.b[((int64_t)e * p.n + c) * p.k + kk];
          } else if (MODE == BG_DGRAD) {
            if (arow >= 0) va = p.a[arow * p.n + kk];
            if (c < N) vb = p.b[((int64_t)e * p.n + kk) * p.k + c];
          } else {
            const int64_t xr = gathered_row(p.row_index, p.a_rows, lo + kk, hi);
            if (m < M) va = p.a[(lo + kk) * p.n + m];
            if (c < N && xr >= 0) vb = p.b[xr * p.k + c];
          }
        }
        fa[j] = __builtin_bit_cast(__bf16, va);
        fb[j] = __builtin_bit_cast(__bf16, vb);
      }
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fb, acc, 0, 0, 0);
    }
    if (c >= N) continue;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int64_t mm = m0 + 8 * (r >> 2) + 4 * h + (r & 3);
      if (mm >= M) continue;
      const int64_t at = (MODE == BG_WGRAD ? (int64_t)e * p.n + mm : lo + mm) * N + c;
      float v = acc[r];
      if (p.y_bf) {
        if (MODE == BG_WGRAD && p.add) v += bf16_to_f32(static_cast<const uint16_t*>(p.add)[at]);
        static_cast<uint16_t*>(p.y)[at] = to_bf16(v);
      } else {
        if (MODE == BG_WGRAD && p.add) v += static_cast<const float*>(p.add)[at];
        static_cast<float*>(p.y)[at] = v;
      }
    }
  }
}

template <int MODE>
static int launch_bf16(const Bf16Args& p, hipStream_t str) {
  const int64_t N = MODE == BG_FORWARD ? p.n : p.k;
  const int64_t mz = ((MODE == BG_WGRAD ? p.n : p.m_total) + 31) / 32;
  hipLaunchKernelGGL(bf16_simple_kernel<MODE>, dim3((unsigned)((N + 31) / 32), (unsigned)p.groups, (unsigned)(mz < 64 ? mz : 64)),
                     dim3(64), 0, str, p);
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
