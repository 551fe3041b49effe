// moe_combine.hip -- a token's sum over its experts' rows and the gradient of
// that sum (gfx950), through the slot_of layout nvfp4_moe_route writes.
//
//   out[t] = sum_j p[t, j] y[slot_of[t, j]]                    (p = 1 when left out)
//   dy[slot_of[t, j]] = p[t, j] dout[t],   dp[t, j] = <dout[t], y[slot_of[t, j]]>
//
// HBM-bound: every routed row is read once, as whole contiguous rows, so the
// gather costs nothing beyond the slot lookups.  Forward: one wave per 512
// columns of a token (8 a lane), up to 8 choices' loads in flight before the
// first sum, choices added in order j in fp32 (the same bits on every call).
// Backward: one block per token; its waves walk the columns, hold the token's
// gradient piece once for all choices, and the dot products meet in LDS in
// wave order.  4096 tokens x 8 x 2048, fp32 y, bf16 dy, inputs changing from
// call to call: forward 52 us (5.5 TB/s), backward 82 us (5.1 TB/s; 81 with
// ordinary stores of dy).  On the same inputs again and again part of y is
// still in the memory-side cache: 42 and 65 us, there 85 with ordinary stores.
#include "rowwise.h"

namespace nvfp4 {

struct CombineArgs {
  const void* y;
  const int32_t* slot_of;
  const float* weights;
  void* out;
  const void* dout;
  void* dy;
  float* dw;
  int64_t y_rows, tokens, d;
  int topk;
  bool y_bf, o_bf, dy_bf;
};

constexpr int COMBINE_CHUNK = 8;  // choices whose rows are loaded together

template <bool VEC>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs p, int pieces) {
  const int lane = threadIdx.x & 63;
  const int64_t items = p.tokens * pieces;
  for (int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); item < items; item += (int64_t)gridDim.x * 4) {
    const int64_t t = item / pieces;
    const int piece = (int)(item % pieces);
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < p.topk; j0 += COMBINE_CHUNK) {
      // lane j holds choice j0 + j: its row (-1 when it has none) and weight
      const bool has = lane < COMBINE_CHUNK && j0 + lane < p.topk;
      int32_t sl = has ? p.slot_of[t * p.topk + j0 + lane] : -1;
      if (sl < 0 || sl >= p.y_rows) sl = -1;
      const float w = has ? (p.weights ? p.weights[t * p.topk + j0 + lane] : 1.0f) : 0.0f;
      float v[COMBINE_CHUNK][8];
#pragma unroll
      for (int j = 0; j < COMBINE_CHUNK; ++j) {
        const int32_t row = __builtin_amdgcn_readlane(sl, j);
        if (row >= 0) {
          load8<VEC>(row_at(p.y, p.y_bf, row, p.d), p.y_bf, p.d, piece, 64, lane, v[j]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < COMBINE_CHUNK; ++j) {
        if (__builtin_amdgcn_readlane(sl, j) < 0) continue;  // nothing added, whatever its weight
        const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), j));
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(wj, v[j][i], acc[i]);
      }
    }
    store8<VEC>(row_at(p.out, p.o_bf, t, p.d), p.o_bf, p.d, piece, 64, lane, acc);
  }
}

template <bool VEC>
__global__ __launch_bounds__(1024) void combine_backward_kernel(CombineArgs p, int pieces) {
  __shared__ float s_dot[16][COMBINE_CHUNK];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, W = blockDim.x >> 6;
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    for (int j0 = 0; j0 < p.topk; j0 += COMBINE_CHUNK) {
      const bool has = lane < COMBINE_CHUNK && j0 + lane < p.topk;
      int32_t sl = has ? p.slot_of[t * p.topk + j0 + lane] : -1;
      if (sl < 0 || sl >= p.y_rows) sl = -1;
      const float w = has ? (p.weights ? p.weights[t * p.topk + j0 + lane] : 1.0f) : 0.0f;
      float dot[COMBINE_CHUNK] = {};
      for (int piece = wave; piece < pieces; piece += W) {
        float g[8];
        load8<VEC>(row_at(p.dout, p.o_bf, t, p.d), p.o_bf, p.d, piece, 64, lane, g);
#pragma unroll
        for (int j = 0; j < COMBINE_CHUNK; ++j) {
          const int32_t row = __builtin_amdgcn_readlane(sl, j);
          if (row < 0) continue;
          const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), j));
          if (p.dw) {
            float v[8];
            load8<VEC>(row_at(p.y, p.y_bf, row, p.d), p.y_bf, p.d, piece, 64, lane, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[j] = __builtin_fmaf(g[i], v[i], dot[j]);
          }
          if (p.dy) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = wj * g[i];
            store8<VEC>(row_at(p.dy, p.dy_bf, row, p.d), p.dy_bf, p.d, piece, 64, lane, o);
          }
        }
      }
      if (!p.dw) continue;
#pragma unroll
      for (int j = 0; j < COMBINE_CHUNK; ++j) {
        const float s = wave_sum_f32(dot[j]);
        if (lane == 0) s_dot[wave][j] = s;
      }
      __syncthreads();
      if (wave == 0 && has) {
        float s = 0.0f;
        for (int k = 0; k < W; ++k) s += s_dot[k][lane];
        p.dw[t * p.topk + j0 + lane] = s;
      }
      __syncthreads();
    }
  }
}

static bool combine_vec(int64_t d, const void* a, const void* b, const void* c) {
  return d % 8 == 0 && nvfp4host::aligned(a, 16) && nvfp4host::aligned(b, 16) && nvfp4host::aligned(c, 16);
}

}  // namespace nvfp4

using nvfp4host::aligned;

static bool bad_type(int t) { return t != NVFP4_TYPE_F32 && t != NVFP4_TYPE_BF16; }
static bool bad_elem(const void* p, int t) { return !aligned(p, t == NVFP4_TYPE_BF16 ? 2 : 4); }

// sizes both calls share: 0 to go on, -1 nothing to do, else the error
static int combine_sizes(int64_t y_rows, int64_t tokens, int64_t topk, int64_t d) {
  if (y_rows < 0 || tokens < 0 || topk < 1 || d < 0) return NVFP4_ERROR_INVALID_VALUE;
  if (topk > 64 || tokens > ((int64_t)1 << 31) / topk || y_rows > ((int64_t)1 << 31) || d > ((int64_t)1 << 24))
    return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  return (tokens == 0 || d == 0) ? -1 : NVFP4_SUCCESS;
}

extern "C" int nvfp4_moe_combine(const void* y, int y_type, int64_t y_rows, const int32_t* slot_of,
                                 const float* weights, int64_t tokens, int64_t topk, int64_t d, void* out,
                                 int out_type, void* stream) {
  if (bad_type(y_type) || bad_type(out_type)) return NVFP4_ERROR_INVALID_VALUE;
  int st = combine_sizes(y_rows, tokens, topk, d);
  if (st) return st < 0 ? NVFP4_SUCCESS : st;
  if ((y_rows > 0 && !y) || !slot_of || !out) return NVFP4_ERROR_INVALID_VALUE;
  if (bad_elem(y, y_type) || bad_elem(out, out_type) || !aligned(slot_of, 4) || !aligned(weights, 4))
    return NVFP4_ERROR_MISALIGNED;
  const int pieces = (int)((d + 511) / 512);
  if ((st = nvfp4host::check_arch())) return st;
  nvfp4::CombineArgs p{};
  p.y = y; p.slot_of = slot_of; p.weights = weights; p.out = out;
  p.y_rows = y_rows; p.tokens = tokens; p.d = d; p.topk = (int)topk;
  p.y_bf = y_type == NVFP4_TYPE_BF16; p.o_bf = out_type == NVFP4_TYPE_BF16;
  const int64_t blocks = (tokens * pieces + 3) / 4;
  const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)));
  if (nvfp4::combine_vec(d, y, out, nullptr))
    hipLaunchKernelGGL(nvfp4::combine_kernel<true>, grid, dim3(256), 0, (hipStream_t)stream, p, pieces);
  else
    hipLaunchKernelGGL(nvfp4::combine_kernel<false>, grid, dim3(256), 0, (hipStream_t)stream, p, pieces);
  return nvfp4host::launch_status();
}

extern "C" int nvfp4_moe_combine_backward(const void* dout, int dout_type, const void* y, int y_type, int64_t y_rows,
                                          const int32_t* slot_of, const float* weights, int64_t tokens, int64_t topk,
                                          int64_t d, void* dy, int dy_type, float* d_weights, void* stream) {
  if (bad_type(dout_type) || bad_type(y_type) || bad_type(dy_type)) return NVFP4_ERROR_INVALID_VALUE;
  int st = combine_sizes(y_rows, tokens, topk, d);
  if (st > 0) return st;
  if (!dy && !d_weights) return NVFP4_ERROR_INVALID_VALUE;
  if (tokens == 0) return NVFP4_SUCCESS;
  if (!slot_of || (d > 0 && !dout) || (d > 0 && y_rows > 0 && d_weights && !y)) return NVFP4_ERROR_INVALID_VALUE;
  if (bad_elem(dout, dout_type) || bad_elem(y, y_type) || bad_elem(dy, dy_type) || !aligned(slot_of, 4) ||
      !aligned(weights, 4) || !aligned(d_weights, 4))
    return NVFP4_ERROR_MISALIGNED;
  if ((st = nvfp4host::check_arch())) return st;
  nvfp4::CombineArgs p{};
  p.y = y; p.slot_of = slot_of; p.weights = weights; p.dout = dout; p.dy = dy; p.dw = d_weights;
  p.y_rows = y_rows; p.tokens = tokens; p.d = d; p.topk = (int)topk;
  p.y_bf = y_type == NVFP4_TYPE_BF16; p.o_bf = dout_type == NVFP4_TYPE_BF16; p.dy_bf = dy_type == NVFP4_TYPE_BF16;
  const int pieces = (int)((d + 511) / 512);
  const int W = pieces < 1 ? 1 : (pieces > 16 ? 16 : pieces);
  const int64_t cap = (int64_t)nvfp4host::num_cus() * 64;
  const dim3 grid((unsigned)(tokens < cap ? tokens : cap)), block(64 * W);
  if (nvfp4::combine_vec(d, d_weights ? y : nullptr, dout, dy))
    hipLaunchKernelGGL(nvfp4::combine_backward_kernel<true>, grid, block, 0, (hipStream_t)stream, p, pieces);
  else
    hipLaunchKernelGGL(nvfp4::combine_backward_kernel<false>, grid, block, 0, (hipStream_t)stream, p, pieces);
  return nvfp4host::launch_status();
}
