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
constexpr int CLIP_BLOCKS = 1024;    // partial sums of one launch

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

__global__ __launch_bounds__(256) void clip_squares_kernel(ClipList l, double* partial) {
  __shared__ double s[4];
  double acc = 0.0;
  for (int chunk = blockIdx.x; chunk < l.first[l.n]; chunk += gridDim.x) {
    int t;
    int64_t lo, hi;
    chunk_at(l, chunk, t, lo, hi);
    const bool bf = (l.bf16[t >> 5] >> (t & 31)) & 1u;
    const uint8_t* base = static_cast<const uint8_t*>(l.in[t]);
    if (((uintptr_t)base & 15) == 0 && hi - lo == CLIP_CHUNK) {
#pragma unroll 4
      for (int i = 0; i < CLIP_CHUNK / 2048; ++i) {
        float v[8];
        load8<true>(base + lo * (bf ? 2 : 4), bf, CLIP_CHUNK, i, 256, threadIdx.x, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc = __builtin_fma((double)v[e], (double)v[e], acc);
      }
    } else {
      for (int64_t e = lo + threadIdx.x; e < hi; e += 256) {
        const double v = bf ? bf16_to_f32(reinterpret_cast<const uint16_t*>(base)[e]) : reinterpret_cast<const float*>(base)[e];
        acc = __builtin_fma(v, v, acc);
      }
    }
  }
  acc = block_sum_f64(acc, s);
  if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

__global__ __launch_bounds__(256) void clip_scale_kernel(ClipList l, const double* partial, int partials,
                                                         float max_norm, float* norm_out) {
  __shared__ double s[4];
  double acc = 0.0;
  for (int i = threadIdx.x; i < partials; i += 256) acc += partial[i];
  const double norm = __builtin_sqrt(block_sum_f64(acc, s));
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm_out) *norm_out = (float)norm;
  const double f = (double)max_norm / (norm + 1e-6);
  const float c = (float)(f > 1.0 ? 1.0 : f);  // a NaN norm gives a NaN factor
  for (int chunk = blockIdx.x; chunk < l.first[l.n]; chunk += gridDim.x) {
    int t;
    int64_t lo, hi;
    chunk_at(l, chunk, t, lo, hi);
    const bool bf = (l.bf16[t >> 5] >> (t & 31)) & 1u;
    const uint8_t* in = static_cast<const uint8_t*>(l.in[t]);
    uint8_t* out = static_cast<uint8_t*>(l.out[t]);
    if ((((uintptr_t)in | (uintptr_t)out) & 15) == 0 && hi - lo == CLIP_CHUNK) {
#pragma unroll 4
      for (int i = 0; i < CLIP_CHUNK / 2048; ++i) {
        float v[8];
        load8<true>(in + lo * (bf ? 2 : 4), bf, CLIP_CHUNK, i, 256, threadIdx.x, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= c;
        store8<true>(out + lo * (bf ? 2 : 4), bf, CLIP_CHUNK, i, 256, threadIdx.x, v);
      }
    } else {
      for (int64_t e = lo + threadIdx.x; e < hi; e += 256) {
        if (bf) reinterpret_cast<uint16_t*>(out)[e] = to_bf16(bf16_to_f32(reinterpret_cast<const uint16_t*>(in)[e]) * c);
        else reinterpret_cast<float*>(out)[e] = reinterpret_cast<const float*>(in)[e] * c;
      }
    }
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
  int partials = 0;
  ClipList l;
  // pass 0 sums squares, pass 1 scales (with nothing to scale: the norm only)
  for (int pass = 0; pass < 2; ++pass) {
    int64_t i = 0;
    do {
      l.n = 0;
      l.first[0] = 0;
      for (uint32_t& b : l.bf16) b = 0u;
      int64_t chunks = 0;  // at most 96 x 2^23
      for (; i < tensors && l.n < CLIP_LIST; ++i) {
        if (counts[i] == 0) continue;
        const int64_t c = (counts[i] + CLIP_CHUNK - 1) / CLIP_CHUNK;
        l.in[l.n] = grads[i];
        l.out[l.n] = out ? out[i] : nullptr;
        l.count[l.n] = counts[i];
        if (types[i] == NVFP4_TYPE_BF16) l.bf16[l.n >> 5] |= 1u << (l.n & 31);
        chunks += c;
        l.first[++l.n] = (int32_t)chunks;
      }
      const int64_t blocks = chunks < 1 ? 1 : (chunks < CLIP_BLOCKS ? chunks : CLIP_BLOCKS);
      if (pass == 0) {
        hipLaunchKernelGGL(clip_squares_kernel, dim3((unsigned)blocks), dim3(256), 0, str, l, partial + partials);
        partials += (int)blocks;
      } else {
        if (!out) l.n = 0, l.first[0] = 0;
        hipLaunchKernelGGL(clip_scale_kernel, dim3(out ? (unsigned)blocks : 1u), dim3(256), 0, str, l, partial, partials,
                           max_norm, norm);
        if (!out) break;
      }
    } while (i < tensors);
  }
  return nvfp4host::launch_status();
}
