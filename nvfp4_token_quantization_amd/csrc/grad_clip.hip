// grad_clip.hip -- the global norm of many gradient tensors and their
// clipping by it (gfx950).
//
//   N = sqrt(sum over tensors of sum g^2),  c = min(1, max_norm / (N + 1e-6)),
//   out = round(c g) in each tensor's own type.
//
// HBM-bound, in two passes over the data, since the factor needs every
// gradient.  Pass 1: a fixed set of blocks walks the tensors' chunks and each
// leaves one fp64 partial sum (squares of fp32 and bf16 values neither
// overflow nor vanish in fp64, and an fp64 FMA for every element is a small
// part of the memory time); pass 2: every block adds the partials in index
// order, derives the factor and scales its chunks.  Nothing is added by
// atomics: the same bits on every call.  The tensors' addresses and sizes
// travel in the kernel arguments, so nothing is staged in device memory and a
// captured graph holds them; a set larger than one launch's list takes
// several launches a pass.
#include "rowwise.h"

namespace nvfp4 {

constexpr int CLIP_LIST = 96;        // tensors in one launch's arguments
constexpr int CLIP_CHUNK = 8192;     // elements a block takes at a time
// Blocks, and partial sums, of one launch: three a CU (755 MB of fp32 and bf16
// gradients, 512, 768, 1024, 2048 blocks: 452, 410, 419, 450 us; as it stands
// 397 to 405 us into tensors of their own, 5.6 TB/s over the three passes, 408
// with ordinary stores, 423 in place; the norm alone 129 us, 5.8 TB/s).
constexpr int CLIP_BLOCKS = 768;

struct ClipList {
  const void* in[CLIP_LIST];
  void* out[CLIP_LIST];
  int64_t count[CLIP_LIST];
  int32_t first[CLIP_LIST + 1];  // first chunk of each tensor
  uint32_t bf16[(CLIP_LIST + 31) / 32];
  int n;
};

__device__ __forceinline__ int tensor_of(const ClipList& l, int chunk) {
  int lo = 0, hi = l.n;  // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (l.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double block_sum_f64(double v, double* s) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.0;
  for (int k = 0; k < (int)(blockDim.x >> 6); ++k) t += s[k];
  __syncthreads();
  return t;
}

__device__ __forceinline__ void chunk_at(const ClipList& l, int chunk, int& t, int64_t& lo, int64_t& hi) {
  t = tensor_of(l, chunk);
  lo = (int64_t)(chunk - l.first[t]) * CLIP_CHUNK;
  hi = min(l.count[t], lo + CLIP_CHUNK);
}

// Elements [lo, hi) of a tensor to `slot` 8 at a time where the memory is
// 16-byte aligned, and to `one` singly otherwise and at a ragged end.
template <class Slot, class One>
__device__ __forceinline__ void walk_chunk(int64_t lo, int64_t hi, bool wide, Slot&& slot, One&& one) {
  int64_t e = lo;
  if (wide) {
    if (hi - lo == CLIP_CHUNK) {
#pragma unroll
      for (int i = 0; i < CLIP_CHUNK / 2048; ++i) slot(lo + 8 * (i * 256 + (int)threadIdx.x));
      return;
    }
    const int n = (int)((hi - lo) / 8);
    for (int i = threadIdx.x; i < n; i += 256) slot(lo + 8 * i);
    e = lo + 8 * n;
  }
  for (e += threadIdx.x; e < hi; e += 256) one(e);
}

__global__ __launch_bounds__(256) void clip_squares_kernel(ClipList l, double* partial) {
  __shared__ double s[4];
  double acc[2] = {0.0, 0.0};
  for (int chunk = blockIdx.x; chunk < l.first[l.n]; chunk += gridDim.x) {
    int t;
    int64_t lo, hi;
    chunk_at(l, chunk, t, lo, hi);
    const bool bf = (l.bf16[t >> 5] >> (t & 31)) & 1u;
    const uint8_t* base = static_cast<const uint8_t*>(l.in[t]);
    walk_chunk(lo, hi, ((uintptr_t)base & 15) == 0,
               [&](int64_t e) {
                 float v[8];
                 load8<true>(base + e * (bf ? 2 : 4), bf, 8, 0, 256, 0, v);
#pragma unroll
                 for (int i = 0; i < 8; ++i) acc[i & 1] = __builtin_fma((double)v[i], (double)v[i], acc[i & 1]);
               },
               [&](int64_t e) {
                 const double v = bf ? bf16_to_f32(reinterpret_cast<const uint16_t*>(base)[e])
                                     : reinterpret_cast<const float*>(base)[e];
                 acc[0] = __builtin_fma(v, v, acc[0]);
               });
  }
  const double sum = block_sum_f64(acc[0] + acc[1], s);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// Walks the chunks last to first: what the first pass read last is what the
// memory-side cache still holds.
__global__ __launch_bounds__(256) void clip_scale_kernel(ClipList l, const double* partial, int partials,
                                                         float max_norm, float* norm_out) {
  __shared__ double s[4];
  double acc = 0.0;
  for (int i = threadIdx.x; i < partials; i += 256) acc += partial[i];
  const double norm = __builtin_sqrt(block_sum_f64(acc, s));
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm_out) *norm_out = (float)norm;
  const double f = (double)max_norm / (norm + 1e-6);
  // The factor is rounded once to 24 bits, c 2^e: e = 0 where it is a normal
  // fp32, else c lies in [0.5, 1] (as a subnormal fp32 it left gradients of
  // norm 3e38 clipped to 0.001 off by 1e-4, and as zero those clipped to 1e-9
  // zero).  A NaN norm gives a NaN factor.
  int e = 0;
  const bool small = f > 0.0 && f < 0x1p-126;
  const float c = (float)(f > 1.0 ? 1.0 : small ? __builtin_frexp(f, &e) : f);
  auto scaled = [&](float v) { return __builtin_ldexpf(v * c, e); };
  for (int chunk = l.first[l.n] - 1 - (int)blockIdx.x; chunk >= 0; chunk -= gridDim.x) {
    int t;
    int64_t lo, hi;
    chunk_at(l, chunk, t, lo, hi);
    const bool bf = (l.bf16[t >> 5] >> (t & 31)) & 1u;
    const uint8_t* in = static_cast<const uint8_t*>(l.in[t]);
    uint8_t* out = static_cast<uint8_t*>(l.out[t]);
    const bool wide = (((uintptr_t)in | (uintptr_t)out) & 15) == 0;
    if (wide && hi - lo == CLIP_CHUNK) {
#pragma unroll
      for (int i = 0; i < CLIP_CHUNK / 2048; ++i) {
        float v[8];
        load8<true>(in + lo * (bf ? 2 : 4), bf, CLIP_CHUNK, i, 256, threadIdx.x, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = scaled(v[k]);
        store8<true>(out + lo * (bf ? 2 : 4), bf, CLIP_CHUNK, i, 256, threadIdx.x, v);
      }
      continue;
    }
    walk_chunk(lo, hi, wide,
               [&](int64_t k) {
                 float v[8];
                 load8<true>(in + k * (bf ? 2 : 4), bf, 8, 0, 256, 0, v);
#pragma unroll
                 for (int i = 0; i < 8; ++i) v[i] = scaled(v[i]);
                 store8<true>(out + k * (bf ? 2 : 4), bf, 8, 0, 256, 0, v);
               },
               [&](int64_t k) {
                 if (bf) reinterpret_cast<uint16_t*>(out)[k] = to_bf16(scaled(bf16_to_f32(reinterpret_cast<const uint16_t*>(in)[k])));
                 else reinterpret_cast<float*>(out)[k] = scaled(reinterpret_cast<const float*>(in)[k]);
               });
  }
}

}  // namespace nvfp4

using nvfp4host::aligned;

extern "C" int64_t nvfp4_clip_grad_norm_workspace(int64_t tensors) {
  if (tensors < 1) return 0;
  return (tensors + nvfp4::CLIP_LIST - 1) / nvfp4::CLIP_LIST * nvfp4::CLIP_BLOCKS * (int64_t)sizeof(double);
}

extern "C" int nvfp4_clip_grad_norm(const void* const* grads, void* const* out, const int64_t* counts,
                                    const int32_t* types, int64_t tensors, float max_norm, float* norm,
                                    void* workspace, int64_t workspace_bytes, void* stream) {
  using namespace nvfp4;
  if (tensors < 0 || !(max_norm >= 0.0f)) return NVFP4_ERROR_INVALID_VALUE;
  if (tensors > 0 && (!grads || !counts || !types)) return NVFP4_ERROR_INVALID_VALUE;
  if (!norm && !out) return NVFP4_ERROR_INVALID_VALUE;
  if (tensors > (1 << 20)) return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  for (int64_t i = 0; i < tensors; ++i) {
    if (counts[i] < 0 || (types[i] != NVFP4_TYPE_F32 && types[i] != NVFP4_TYPE_BF16)) return NVFP4_ERROR_INVALID_VALUE;
    if (counts[i] > 0 && (!grads[i] || (out && !out[i]))) return NVFP4_ERROR_INVALID_VALUE;
    if (counts[i] > ((int64_t)1 << 36)) return NVFP4_ERROR_UNSUPPORTED_SHAPE;
    const int a = types[i] == NVFP4_TYPE_BF16 ? 2 : 4;
    if (!aligned(grads[i], a) || (out && !aligned(out[i], a))) return NVFP4_ERROR_MISALIGNED;
  }
  if (!aligned(norm, 4) || !aligned(workspace, 8)) return NVFP4_ERROR_MISALIGNED;
  const int64_t need = nvfp4_clip_grad_norm_workspace(tensors < 1 ? 1 : tensors);
  if (!workspace || workspace_bytes < need) return NVFP4_ERROR_INVALID_VALUE;
  int st = nvfp4host::check_arch();
  if (st) return st;
  hipStream_t str = (hipStream_t)stream;
  double* partial = static_cast<double*>(workspace);
  ClipList l;
  // the next list of up to CLIP_LIST tensors from i in direction `step`
  auto next_list = [&](int64_t& i, int step) -> int64_t {
    l.n = 0;
    l.first[0] = 0;
    for (uint32_t& b : l.bf16) b = 0u;
    int64_t chunks = 0;  // at most 96 x 2^23
    int64_t at[CLIP_LIST];
    for (; i >= 0 && i < tensors && l.n < CLIP_LIST; i += step)
      if (counts[i] > 0) at[l.n++] = i;
    for (int j = 0; j < l.n; ++j) {
      const int64_t k = at[step > 0 ? j : l.n - 1 - j];  // ascending either way
      l.in[j] = grads[k];
      l.out[j] = out ? out[k] : nullptr;
      l.count[j] = counts[k];
      if (types[k] == NVFP4_TYPE_BF16) l.bf16[j >> 5] |= 1u << (j & 31);
      chunks += (counts[k] + CLIP_CHUNK - 1) / CLIP_CHUNK;
      l.first[j + 1] = (int32_t)chunks;
    }
    return chunks < 1 ? 1 : (chunks < CLIP_BLOCKS ? chunks : CLIP_BLOCKS);
  };
  int partials = 0;
  int64_t i = 0;
  do {
    const int64_t blocks = next_list(i, 1);
    hipLaunchKernelGGL(clip_squares_kernel, dim3((unsigned)blocks), dim3(256), 0, str, l, partial + partials);
    partials += (int)blocks;
  } while (i < tensors);
  if (out) {
    i = tensors - 1;
    do {
      const int64_t blocks = next_list(i, -1);
      hipLaunchKernelGGL(clip_scale_kernel, dim3((unsigned)blocks), dim3(256), 0, str, l, partial, partials, max_norm, norm);
    } while (i >= 0);
  } else {
    l.n = 0;
    l.first[0] = 0;
    hipLaunchKernelGGL(clip_scale_kernel, dim3(1), dim3(256), 0, str, l, partial, partials, max_norm, norm);
  }
  return nvfp4host::launch_status();
}
