// rowwise.h -- loads, stores and reductions of the kernels that hold one row
// in the registers of W waves (residual norms, expert combine), gfx950.
//
// A row of d elements is cut into slots of 8: slot v of thread t (of T = 64 W)
// holds 8 consecutive elements from 8 (v T + t) when the rows can be read in
// 16-byte pieces (VEC: d % 8 == 0 and 16-byte aligned rows), and otherwise the
// elements (8 v + i) T + t, so that every scalar access of a wave is
// contiguous too.
#pragma once

#include "nvfp4_internal.h"

namespace nvfp4 {

typedef __bf16 bf16_2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_to_f32(uint32_t b) { return __uint_as_float(b << 16); }

// fp32 -> bf16 bits, nearest even, NaN kept (the hardware converter)
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16_2 p = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ uint16_t to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

template <bool VEC>
__device__ __forceinline__ int64_t slot_elem(int v, int i, int T, int tid) {
  return VEC ? 8 * ((int64_t)v * T + tid) + i : ((int64_t)8 * v + i) * T + tid;
}

// 8 elements of slot v of the row at `row`, as fp32; elements past d are `fill`
template <bool VEC>
__device__ __forceinline__ void load8(const void* row, bool is_bf16, int64_t d, int v, int T, int tid,
                                      float (&o)[8], float fill = 0.0f) {
  if (VEC) {
    const int64_t e = slot_elem<true>(v, 0, T, tid);
    if (e >= d) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = fill;
    } else if (is_bf16) {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + e);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[2 * i] = __uint_as_float(u[i] << 16);
        o[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    } else {
      const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(row) + e);
      const f32x4 a = p[0], b = p[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i] = a[i];
        o[4 + i] = b[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t e = slot_elem<false>(v, i, T, tid);
      if (e >= d) o[i] = fill;
      else if (is_bf16) o[i] = bf16_to_f32(static_cast<const uint16_t*>(row)[e]);
      else o[i] = static_cast<const float*>(row)[e];
    }
  }
}

// 8 fp32 values to slot v of the row at `row`, rounded once when it is bf16
// (streaming stores)
template <bool VEC>
__device__ __forceinline__ void store8(void* row, bool is_bf16, int64_t d, int v, int T, int tid,
                                       const float (&o)[8]) {
  if (VEC) {
    const int64_t e = slot_elem<true>(v, 0, T, tid);
    if (e >= d) return;
    if (is_bf16) {
      const u32x4 w = {pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7])};
      __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(row) + e));
    } else {
      f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(row) + e);
      __builtin_nontemporal_store((f32x4){o[0], o[1], o[2], o[3]}, p);
      __builtin_nontemporal_store((f32x4){o[4], o[5], o[6], o[7]}, p + 1);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t e = slot_elem<false>(v, i, T, tid);
      if (e >= d) continue;
      if (is_bf16) static_cast<uint16_t*>(row)[e] = to_bf16(o[i]);
      else static_cast<float*>(row)[e] = o[i];
    }
  }
}

// Slot v of a row that is read or written once (VEC), through a resource over
// the row: slots past its end read as zeros and are not written, without a
// branch.  Streaming accesses; the loads are raw, so that a caller issues them
// a row ahead of their use and decodes them then.
struct RawSlot {
  u32x4 a, b;  // b: the second half of an fp32 slot
};
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void* row, bool is_bf16, int64_t d) {
  return out_rsrc(reinterpret_cast<float*>(const_cast<void*>(row)), d * (is_bf16 ? 2 : 4));
}
__device__ __forceinline__ void load_raw(const void* row, bool is_bf16, int64_t d, int v, int T, int tid, RawSlot& o) {
  const __amdgpu_buffer_rsrc_t r = row_rsrc(row, is_bf16, d);
  const uint32_t at = (uint32_t)slot_elem<true>(v, 0, T, tid) * (is_bf16 ? 2 : 4);
  o.a = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 2);
  if (!is_bf16) o.b = __builtin_amdgcn_raw_buffer_load_b128(r, at + 16, 0, 2);
}
__device__ __forceinline__ void decode_raw(const RawSlot& r, bool is_bf16, float (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (is_bf16) {
      o[2 * i] = __uint_as_float(r.a[i] << 16);
      o[2 * i + 1] = __uint_as_float(r.a[i] & 0xFFFF0000u);
    } else {
      o[i] = __uint_as_float(r.a[i]);
      o[4 + i] = __uint_as_float(r.b[i]);
    }
  }
}
__device__ __forceinline__ void store_raw(void* row, bool is_bf16, int64_t d, int v, int T, int tid, const float (&o)[8]) {
  const __amdgpu_buffer_rsrc_t r = row_rsrc(row, is_bf16, d);
  const uint32_t at = (uint32_t)slot_elem<true>(v, 0, T, tid) * (is_bf16 ? 2 : 4);
  if (is_bf16) {
    const u32x4 w = {pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7])};
    __builtin_amdgcn_raw_buffer_store_b128(w, r, at, 0, 2);
  } else {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, (f32x4){o[0], o[1], o[2], o[3]}), r, at, 0, 2);
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, (f32x4){o[4], o[5], o[6], o[7]}), r, at + 16, 0, 2);
  }
}

// start of row r of a [.., d] array of bf16 or fp32
__device__ __forceinline__ const void* row_at(const void* p, bool is_bf16, int64_t r, int64_t d) {
  return static_cast<const uint8_t*>(p) + r * d * (is_bf16 ? 2 : 4);
}
__device__ __forceinline__ void* row_at(void* p, bool is_bf16, int64_t r, int64_t d) {
  return static_cast<uint8_t*>(p) + r * d * (is_bf16 ? 2 : 4);
}

// Sum over the 64 lanes of a wave, every lane gets it: a fixed tree (DPP
// within 16-lane rows, then the four rows' sums by readlane).
__device__ __forceinline__ float wave_sum_f32(float v) {
  v += __uint_as_float(dpp_mov<0xB1>(__float_as_uint(v)));   // quad_perm [1,0,3,2]
  v += __uint_as_float(dpp_mov<0x4E>(__float_as_uint(v)));   // quad_perm [2,3,0,1]
  v += __uint_as_float(dpp_mov<0x141>(__float_as_uint(v)));  // row_half_mirror
  v += __uint_as_float(dpp_mov<0x140>(__float_as_uint(v)));  // row_mirror
  const int b = __float_as_uint(v);
  const float s0 = __uint_as_float(__builtin_amdgcn_readlane(b, 0)) + __uint_as_float(__builtin_amdgcn_readlane(b, 16));
  const float s1 = __uint_as_float(__builtin_amdgcn_readlane(b, 32)) + __uint_as_float(__builtin_amdgcn_readlane(b, 48));
  return s0 + s1;
}

// Sums of N values over the W waves of a block (every thread gets them).  The
// caller alternates `slot` between 0 and 1 from one call to the next, so one
// barrier a call suffices: a wave writes a slot again only after the barrier
// of the call between, which every wave has reached with its reads done.
template <int N>
struct BlockSums {
  float w[2][N][16];
};
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], int W, int slot, BlockSums<N>& s) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum_f32(v[i]);
  if (W == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) s.w[slot][i][threadIdx.x >> 6] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = 0.0f;
    for (int k = 0; k < W; ++k) t += s.w[slot][i][k];
    v[i] = t;
  }
}

}  // namespace nvfp4
