// Rows of bf16, fp16 or fp32 values read and written by the row operators (rows.cu, norm.cu).
//
// A block of nt threads covers a row of H values in chunks of 8 values per thread, held as fp32.
// VEC: thread i owns the 8 consecutive values from (c * nt + i) * 8, moved as 16-byte words; it
// needs H a multiple of 8 and every row to start on a 16-byte boundary. Otherwise thread i owns
// the values (8 * c + e) * nt + i (e = 0..7): single values, neighbouring threads on neighbouring
// addresses, any H and any stride. Values past H read as 0 and are not written.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

template <typename T> struct RowType;
template <> struct RowType<__nv_bfloat16> {
  static __device__ __forceinline__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};
template <> struct RowType<__half> {
  static __device__ __forceinline__ float to(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from(float v) { return __float2half_rn(v); }
};
template <> struct RowType<float> {
  static __device__ __forceinline__ float to(float v) { return v; }
  static __device__ __forceinline__ float from(float v) { return v; }
};

template <typename T> struct alignas(16) Raw8 { T v[8]; };

// Index of value e of chunk c of thread tid.
template <bool VEC>
__device__ __forceinline__ int col_of(int c, int e, int nt, int tid) {
  return VEC ? (c * nt + tid) * 8 + e : (c * 8 + e) * nt + tid;
}

template <bool VEC, typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T* row, int c, int nt, int tid, int H) {
  Raw8<T> r;
  if (VEC) {
    const int n0 = col_of<true>(c, 0, nt, tid);
    uint4* q = reinterpret_cast<uint4*>(&r);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      q[i] = n0 < H ? reinterpret_cast<const uint4*>(row + n0)[i] : make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int n = col_of<false>(c, e, nt, tid);
      r.v[e] = n < H ? row[n] : RowType<T>::from(0.f);
    }
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void to_float(const Raw8<T>& r, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = RowType<T>::to(r.v[e]);
}

template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* row, int c, int nt, int tid, int H, float (&f)[8]) {
  to_float(load_raw<VEC>(row, c, nt, tid, H), f);
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* row, int c, int nt, int tid, int H, const float (&f)[8]) {
  Raw8<T> r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r.v[e] = RowType<T>::from(f[e]);
  if (VEC) {
    const int n0 = col_of<true>(c, 0, nt, tid);
    if (n0 >= H) return;
    const uint4* q = reinterpret_cast<const uint4*>(&r);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(row + n0)[i] = q[i];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int n = col_of<false>(c, e, nt, tid);
      if (n < H) row[n] = r.v[e];
    }
  }
}

// N sums over the block, every thread gets them, in an order fixed by the block size. One barrier
// per call: `buf` (32 * N floats of shared memory) must not be the buffer of the call before.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (nw == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i * 32 + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < nw ? buf[i * 32 + lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// out = sum over j of w[j] * rows[inv[j]] (chunk c of a token), in j order; a choice whose inv is
// outside [0, P) adds nothing. The places and weights of a batch of choices are read before the
// first of their rows, and the rows before the first is used, so that one token waits for memory
// twice and not twice per choice (2048 tokens, 8 choices, H = 2048: 44 us when each row waited for
// its own place).
template <bool VEC, typename T>
__device__ __forceinline__ void weighted_rows(const T* rows, int64_t ld, const int32_t* inv, const float* wts, int k,
                                              int P, int c, int nt, int tid, int H, float (&out)[8]) {
  constexpr int B = sizeof(T) == 2 ? 8 : 4;   // choices in flight: 128 bytes per thread
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = 0.f;
  for (int j0 = 0; j0 < k; j0 += B) {
    Raw8<T> r[B];
    float w[B];
    int p[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const bool in = j0 + b < k;
      p[b] = in ? inv[j0 + b] : -1;
      w[b] = in && wts ? wts[j0 + b] : 1.f;
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const bool on = (unsigned)p[b] < (unsigned)P;
      // a choice left out reads nothing (H = 0) and counts with weight 0 on zeros
      w[b] = on ? w[b] : 0.f;
      r[b] = load_raw<VEC>(rows + (int64_t)(on ? p[b] : 0) * ld, c, nt, tid, on ? H : 0);
    }
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = fmaf(w[b], RowType<T>::to(r[b].v[e]), out[e]);
  }
}

// ---- host side ----
inline size_t dtype_size(int dtype) {
  return dtype == MOE_DTYPE_F32 ? 4 : dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F16 ? 2 : 0;
}
// Whether rows of `stride` elements from `p` all start on a 16-byte boundary (null: nothing to move).
inline bool rows16(const void* p, int64_t stride, size_t size) {
  return !p || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(stride * (int64_t)size)) & 15) == 0;
}
// Threads of a block that covers H values in chunks of 8, at most `most`.
inline int row_threads(int H, int most) {
  const int t = (ceil_div(H, 8) + 31) / 32 * 32;
  return t < most ? t : most;
}

}  // namespace moe
