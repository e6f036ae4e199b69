// Rows of bf16, fp16 or fp32 values read and written by the row operators (rows.cu, norm.cu).
//
// A block of nt threads covers a row of H values in chunks of 8 values per thread, held as fp32. NT, a
// template argument of everything below, is 0 for rows of 16-byte words: thread i owns the 8
// consecutive values from (c * nt + i) * 8; it needs H a multiple of 8 and every row to start on a
// 16-byte boundary. Otherwise NT is nt itself, and thread i owns the values (8 * c + e) * NT + i
// (e = 0..7): single values, neighbouring threads on neighbouring addresses, any H and any stride. (As a
// constant it makes the addresses of a row's values offsets of one pointer: 2 to 4 instructions per
// value read, not 20.) Values past H read as 0 and are not written.
//
// Times in the comments of these files rank two forms of a kernel against each other, most of them on inputs
// that repeat from pass to pass, so that inputs below some 100 MB were in L2.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

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
template <int NT>
__device__ __forceinline__ int col_of(int c, int e, int nt, int tid) {
  return NT == 0 ? (c * nt + tid) * 8 + e : (c * 8 + e) * NT + tid;
}

template <int NT, typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T* row, int c, int nt, int tid, int H) {
  Raw8<T> r;
  if (NT == 0) {
    const int n0 = col_of<0>(c, 0, nt, tid);
    uint4* q = reinterpret_cast<uint4*>(&r);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      q[i] = n0 < H ? reinterpret_cast<const uint4*>(row + n0)[i] : make_uint4(0, 0, 0, 0);
  } else {
    const T* p = row + (c * 8 * NT + tid);
    if ((c * 8 + 8) * NT <= H) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e] = p[e * NT];
    } else {
      const int left = H - c * 8 * NT - tid;
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e] = e * NT < left ? p[e * NT] : RowType<T>::from(0.f);
    }
  }
  return r;
}

// Two fp32 values in one 64-bit register pair: the sm_100 packed forms do both in one instruction.
// The row kernels with long arithmetic per value are bound by issued instructions, which these halve;
// each half rounds as the scalar operation does.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 halves(F2 p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p.v));
  return r;
}
__device__ __forceinline__ float sum_of(F2 p) {
  const float2 h = halves(p);
  return h.x + h.y;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

__device__ __forceinline__ void to_pairs(const Raw8<__nv_bfloat16>& r, F2 (&f)[4]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void to_pairs(const Raw8<__half>& r, F2 (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2(__half2float(r.v[2 * i]), __half2float(r.v[2 * i + 1]));
}
__device__ __forceinline__ void to_pairs(const Raw8<float>& r, F2 (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2(r.v[2 * i], r.v[2 * i + 1]);
}
__device__ __forceinline__ void from_pairs(const F2 (&f)[4], Raw8<__nv_bfloat16>& r) {
  __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __float22bfloat162_rn(halves(f[i]));
}
__device__ __forceinline__ void from_pairs(const F2 (&f)[4], Raw8<__half>& r) {
  __half2* o = reinterpret_cast<__half2*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __float22half2_rn(halves(f[i]));
}
__device__ __forceinline__ void from_pairs(const F2 (&f)[4], Raw8<float>& r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 h = halves(f[i]);
    r.v[2 * i] = h.x;
    r.v[2 * i + 1] = h.y;
  }
}

// The eight values as pairs: of packed words, or value by value.
template <int NT, typename T>
__device__ __forceinline__ void raw_pairs(const Raw8<T>& r, F2 (&f)[4]) {
  if (NT == 0) {
    to_pairs(r, f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(RowType<T>::to(r.v[2 * i]), RowType<T>::to(r.v[2 * i + 1]));
  }
}

template <int NT, typename T>
__device__ __forceinline__ void load8(const T* row, int c, int nt, int tid, int H, F2 (&f)[4]) {
  raw_pairs<NT>(load_raw<NT>(row, c, nt, tid, H), f);
}

template <typename T>
__device__ __forceinline__ void store_raw(T* row, int n0, int H, const Raw8<T>& r) {
  if (n0 >= H) return;
  const uint4* q = reinterpret_cast<const uint4*>(&r);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(row + n0)[i] = q[i];
}

template <int NT, typename T>
__device__ __forceinline__ void store8(T* row, int c, int nt, int tid, int H, const F2 (&f)[4]) {
  if (NT == 0) {
    Raw8<T> r;
    from_pairs(f, r);
    store_raw(row, col_of<0>(c, 0, nt, tid), H, r);
  } else {
    T* p = row + (c * 8 * NT + tid);
    const int left = (c * 8 + 8) * NT <= H ? 8 * NT : H - c * 8 * NT - tid;
    if (left == 8 * NT) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = halves(f[i]);
        p[2 * i * NT] = RowType<T>::from(v.x);
        p[(2 * i + 1) * NT] = RowType<T>::from(v.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = halves(f[i]);
        if (2 * i * NT < left) p[2 * i * NT] = RowType<T>::from(v.x);
        if ((2 * i + 1) * NT < left) p[(2 * i + 1) * NT] = RowType<T>::from(v.y);
      }
    }
  }
}

// N sums over the block (N = 1 to 8), every thread gets them, in an order fixed by the
// block size. The lanes of a warp share the values out between them as they add (half of the values
// to each half-warp, and so on), so 4 sums cost 6 exchanges and not 20. One barrier per call: `buf`
// (32 * M floats of shared memory) must not be the buffer of the call before.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* buf) {
  constexpr int M = N <= 2 ? N : N <= 4 ? 4 : 8;    // zeros beside three, five, six or seven
  constexpr int L = M == 8 ? 3 : M == 4 ? 2 : M == 2 ? 1 : 0, G = 32 >> L;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  float x[M];
#pragma unroll
  for (int i = 0; i < M; ++i) x[i] = i < N ? v[i] : 0.f;
#pragma unroll
  for (int l = 0; l < L; ++l) {
    const int m = M >> (l + 1), off = 16 >> l;
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < m; ++i) {
      const float keep = up ? x[i + m] : x[i], send = up ? x[i] : x[i + m];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
#pragma unroll
  for (int o = G >> 1; o > 0; o >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
  if (nw > 1) {     // lane's value: lane / G
    const int mine = lane & (G - 1);
    float* row = buf + (lane / G) * 32;
    if (mine == 0) row[warp] = x[0];
    __syncthreads();
    float y[M];
#pragma unroll
    for (int i = 0; i < M; ++i) y[i] = mine + i * G < nw ? row[mine + i * G] : 0.f;
#pragma unroll
    for (int m = M >> 1; m > 0; m >>= 1)
#pragma unroll
      for (int i = 0; i < m; ++i) y[i] += y[i + m];
    x[0] = y[0];
#pragma unroll
    for (int o = G >> 1; o > 0; o >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
  }
  if (M == 1) {
    v[0] = x[0];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, x[0], i * G);
  }
}

// out[c] = sum over j of w[j] * rows[inv[j]] (chunks c0 to c0 + NC - 1 of a token), in j order; a choice
// whose inv is outside [0, P) adds nothing. The places and weights of B choices are read before the
// first of their rows, and the rows before the first is used, so that one token waits for memory
// twice and not twice per choice (2048 tokens, 8 choices, H = 2048: 44 us when each row waited for
// its own place).
template <int B, int NC, int NT, typename T>
__device__ __forceinline__ void weighted_rows(const T* rows, int64_t ld, const int32_t* inv, const float* wts, int k,
                                              int P, int c0, int nt, int tid, int H, F2 (&out)[NC][4]) {
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) out[c][e] = f2(0.f, 0.f);
  for (int j0 = 0; j0 < k; j0 += B) {
    Raw8<T> r[B][NC];
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
      const T* row = rows + (int64_t)(on ? p[b] : 0) * ld;
#pragma unroll
      for (int c = 0; c < NC; ++c) r[b][c] = load_raw<NT>(row, c0 + c, nt, tid, on ? H : 0);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (j0 + b >= k) break;
      const F2 w2 = f2(w[b], w[b]);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        F2 v[4];
        raw_pairs<NT>(r[b][c], v);
#pragma unroll
        for (int e = 0; e < 4; ++e) out[c][e] = fma2(w2, v[e], out[c][e]);
      }
    }
  }
}

// ---- host side ----
// Parts of at most `per` that n >= 0 things take; n + per need not fit an int (2^31 - 1 tokens are allowed).
inline int parts_of(int n, int per) { return n / per + (n % per != 0); }
// moe_dispatch without its checks; `size` bytes per value, strides in values (rows.cu). Also the grouped
// layer path's first step.
int launch_dispatch(const void* x, int64_t ldx, size_t size, const int32_t* idx, int T, int H, int E, int k,
                    int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, void* xp, int64_t ldp,
                    cudaStream_t s);
inline size_t dtype_size(int dtype) {
  return dtype == MOE_DTYPE_F32 ? 4 : dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F16 ? 2 : 0;
}
// Whether rows of `stride` elements from `p` all start on a 16-byte boundary (null: nothing to move).
inline bool rows16(const void* p, int64_t stride, size_t size) {
  return !p || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(stride * (int64_t)size)) & 15) == 0;
}
// Calls f(integral constant) for the block size of single values, among those given (ascending), whose
// one chunk covers H, or else the last.
template <int N, int... Rest, typename F>
auto by_width(int H, F f) {
  if constexpr (sizeof...(Rest) == 0) {
    return f(std::integral_constant<int, N>());
  } else {
    return H <= 8 * N ? f(std::integral_constant<int, N>()) : by_width<Rest...>(H, f);
  }
}
// Threads of a block that covers H values in chunks of 8, at most `most`.
inline int row_threads(int H, int most) {
  const int t = (parts_of(H, 8) + 31) / 32 * 32;
  return t < most ? t : most;
}

}  // namespace moe
