// The ring form of the norms' gradient and its launch, included by one file per row type.
#pragma once

#include <atomic>
#include <type_traits>

#include "norm_back.cuh"

namespace moe {

namespace {

// The gradient for rows whose tensors fit a ring of stages in shared memory: each thread copies its part
// of the next rows (cp.async) while it works on this one, so the loads of several rows stay in flight
// across the two block-wide sums of a row. Of rows of 16-byte words a thread only reads what it copied
// itself: the ring needs no barrier. The weights and the per-channel gate stay in registers. T = 8192,
// H = 4096, bf16, gate per value, next norm: 88 us, and 234 with loads at the top of each row, when a row's
// loads waited for the sums of the row before.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The first n bytes of the 16, zeros behind them.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

template <typename T>
__device__ __forceinline__ void ring_load(const unsigned char* s, int nt, F2 (&f)[4]) {
  Raw8<T> r;
  uint4* q = reinterpret_cast<uint4*>(&r);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) q[i] = *reinterpret_cast<const uint4*>(s + (size_t)i * nt * 16);
  to_pairs(r, f);
}

// Word i of a thread holds the 16 / sizeof(T) columns from here: neighbouring threads on neighbouring
// words (the two words of eight fp32 values next to each other cost twice the requests: 209 us
// against 142 at T = 8192, H = 4096).
template <typename T>
__device__ __forceinline__ int word_col(int i, int nt, int tid) {
  return (i * nt + tid) * (16 / (int)sizeof(T));
}

template <typename T>
__device__ __forceinline__ void store_pairs(void* base, int64_t ld, int64_t t, int nt, int tid, int H,
                                            const F2 (&f)[4]) {
  Raw8<T> r;
  from_pairs(f, r);
  T* row = static_cast<T*>(base) + t * ld;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    const int n = word_col<T>(i, nt, tid);
    if (n < H) *reinterpret_cast<uint4*>(row + n) = reinterpret_cast<const uint4*>(&r)[i];
  }
}

// A weight or gate vector at the thread's columns; past H what r held before.
template <typename T>
__device__ __forceinline__ void load_words(const void* base, int nt, int tid, int H, Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    const int n = word_col<T>(i, nt, tid);
    if (n < H) reinterpret_cast<uint4*>(&r)[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(base) + n);
  }
}

// Rows on any boundary (NT > 0): the block copies the 16-byte granules that cover a row, and its threads
// read single values from where the row starts in them; a barrier per row stands between the copies
// and the reads, and between the reads and the slot's next copies. T = 4877, H = 3384, bf16 with odd
// strides: 167 us with loads at the top of each row. Of a granule nothing outside the tensor's first and
// last byte is read.
template <typename T, int MAXT, int NT, bool HAS_Y, bool NORM_Y, bool NEXT, int GATE>
__global__ void __launch_bounds__(MAXT, ring_blocks(MAXT, HAS_Y))
    norm_backward_ring_kernel(const BackArgs a, int stages, int stage_bytes) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float buf[2][32 * 8];
  int flip = 0;
  constexpr int W = (int)sizeof(T) / 2;              // 16-byte words per thread and tensor
  const int nt = NT ? NT : blockDim.x, tid = threadIdx.x, H = a.H;
  constexpr bool full = GATE == MOE_GATE_FULL;
  const bool has_d = HAS_Y || a.dho;                 // only the norm before a block may have no other gradient
  const int region = NT ? value_region(H, (int)sizeof(T)) : nt * 16 * W;
  // where each tensor's words lie in a stage
  const int at_y = has_d ? region : 0, at_h = at_y + (HAS_Y ? region : 0), at_x = at_h + (NEXT ? region : 0),
            at_g = at_x + (NEXT ? region : 0);
  unsigned char* own = NT ? ring : ring + tid * 16;
  if constexpr (NT == 0) {      // words past H are zeros and stay so
    for (int o = 0; o < stages * stage_bytes; o += region)
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (word_col<T>(i, nt, tid) >= H) *reinterpret_cast<uint4*>(own + o + i * nt * 16) = make_uint4(0, 0, 0, 0);
  }
  const uint32_t own_s = (uint32_t)__cvta_generic_to_shared(own);
  auto words = [&](uint32_t dst, const void* base, int64_t ld, int64_t t) {
    const T* src = static_cast<const T*>(base) + t * ld;
    if constexpr (NT == 0) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int n = word_col<T>(i, nt, tid);
        if (n < H) copy16(dst + i * nt * 16, src + n);
      }
    } else {
      const char* lo = static_cast<const char*>(base);
      const char* hi = reinterpret_cast<const char*>(static_cast<const T*>(base) + (a.T - 1) * ld + H);
      const int off = (int)(reinterpret_cast<uintptr_t>(src) & 15), bytes = off + H * (int)sizeof(T);
      const char* first = reinterpret_cast<const char*>(src) - off;
      for (int g = tid * 16; g < bytes; g += NT * 16) {
        if (first + g >= lo) {
          copy16(dst + g, first + g, (int)min((int64_t)16, (int64_t)(hi - (first + g))));
        } else {                 // the tensor starts inside this granule
          for (int i = off; i < 16 && i < bytes; i += (int)sizeof(T))
            *reinterpret_cast<T*>(ring + (dst - own_s) + g + i) = *reinterpret_cast<const T*>(first + g + i);
        }
      }
    }
  };
  // a row's values from its slot
  auto take = [&](const unsigned char* s, int at, const void* base, int64_t ld, int64_t t, F2(&f)[4]) {
    if constexpr (NT == 0) {
      ring_load<T>(s + at, nt, f);
    } else {
      const int off = (int)(reinterpret_cast<uintptr_t>(static_cast<const T*>(base) + t * ld) & 15);
      load8<NT>(reinterpret_cast<const T*>(s + at + off), 0, nt, tid, H, f);
    }
  };
  auto put = [&](void* base, int64_t ld, int64_t t, const F2(&f)[4]) {
    if constexpr (NT == 0) store_pairs<T>(base, ld, t, nt, tid, H, f);
    else store8<NT>(static_cast<T*>(base) + t * ld, 0, nt, tid, H, f);
  };
  auto vector = [&](const void* base, Raw8<T>& r) {
    if constexpr (NT == 0) load_words<T>(base, nt, tid, H, r);
    else r = load_raw<NT>(static_cast<const T*>(base), 0, nt, tid, H);
  };
  auto issue = [&](int64_t t, int stage) {
    if (t < a.T) {
      const uint32_t d = own_s + stage * stage_bytes;
      if (has_d) words(d, a.dho, a.lddho, t);
      if (HAS_Y) words(d + at_y, a.y, a.ldy, t);
      if (NEXT) {
        words(d + at_h, a.ho, a.ldho, t);
        words(d + at_x, a.dx, a.lddx, t);
      }
      if (full) words(d + at_g, a.gate, a.ldg, t);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  pdl_begin();
  for (int i = 0; i < stages - 1; ++i) issue((int64_t)blockIdx.x + (int64_t)i * gridDim.x, i);
  const float inv_h = 1.f / (float)H;
  // ones where there is no weight (also past H, where everything else is 0)
  Raw8<T> w, wn, gc;
#pragma unroll
  for (int e = 0; e < 8; ++e) w.v[e] = wn.v[e] = gc.v[e] = RowType<T>::from(1.f);
  if (NORM_Y && a.w) vector(a.w, w);
  if (NEXT && a.w_next) vector(a.w_next, wn);
  if (GATE == MOE_GATE_CHANNEL) vector(a.gate, gc);
  F2 sw[4], sg[4], sn[4];
  const F2 zero = f2(0.f, 0.f), alpha = f2(a.alpha, a.alpha);
#pragma unroll
  for (int e = 0; e < 4; ++e) sw[e] = sg[e] = sn[e] = zero;
  // Where a row has first sums (h'^2, w' dx h', y^2) and second ones that wait for them (w du n, d u), the
  // first are taken a row ahead, together with the second of the row before: one block-wide sum per
  // row. T = 8192, H = 4096, bf16, next norm: 71 us against 79 with one after the other; but with a gate
  // per value, whose rows and gradient are traffic enough, 96 against 87.
  constexpr int kFirst = (NEXT ? 2 : 0) + (NORM_Y ? 1 : 0);
  constexpr int kSecond = (NORM_Y ? 1 : 0) + (GATE == MOE_GATE_TOKEN ? 1 : 0);
  constexpr int kBoth = kFirst + kSecond > 0 ? kFirst + kSecond : 1;
  constexpr bool kAhead = kFirst > 0 && kSecond > 0 && !full && NT == 0;
  auto first_sums = [&](const unsigned char* s, int64_t t, float* out, F2(&h)[4], F2(&x)[4], F2(&y)[4]) {
    if (NEXT) {
      F2 v[4], p0 = zero, p1 = zero;
      take(s, at_h, a.ho, a.ldho, t, h);
      take(s, at_x, a.dx, a.lddx, t, x);
      raw_pairs<NT>(wn, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p0 = fma2(h[e], h[e], p0);
        p1 = fma2(mul2(v[e], x[e]), h[e], p1);
      }
      out[0] = sum_of(p0);
      out[1] = sum_of(p1);
    }
    if (NORM_Y) {
      F2 p2 = zero;
      take(s, at_y, a.y, a.ldy, t, y);
#pragma unroll
      for (int e = 0; e < 4; ++e) p2 = fma2(y[e], y[e], p2);
      out[NEXT ? 2 : 0] = sum_of(p2);
    }
  };
  auto wait_for = [](int left) {       // until at most this many rows are under way
    if (left >= 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (left == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (left == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
  };
  float s[kBoth];
#pragma unroll
  for (int i = 0; i < kBoth; ++i) s[i] = 0.f;
  auto join = [&](auto from, auto count) {       // block-wide: `count` of the sums, from `from` on
    constexpr int F = decltype(from)::value, N = decltype(count)::value;
    if constexpr (N > 0) {
      float part[N];
#pragma unroll
      for (int i = 0; i < N; ++i) part[i] = s[F + i];
      block_sums<N>(part, buf[flip]);
#pragma unroll
      for (int i = 0; i < N; ++i) s[F + i] = part[i];
      flip ^= 1;
    }
  };
  F2 h[4], x[4], y[4];
  if (kAhead) {
    wait_for(stages - 2);
    first_sums(own, blockIdx.x, s, h, x, y);
    join(std::integral_constant<int, 0>(), std::integral_constant<int, kFirst>());
  }
  int stage = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    if (NT > 0) {      // this row is here for every thread, and every thread is done with the slot before
      wait_for(stages - 2);
      __syncthreads();
    }
    issue(t + (int64_t)(stages - 1) * gridDim.x, stage == 0 ? stages - 1 : stage - 1);
    if (NT == 0) wait_for(kAhead ? stages - 2 : stages - 1);      // this row is here, the next where it is needed
    const unsigned char* s0 = own + (size_t)stage * stage_bytes;
    stage = stage + 1 == stages ? 0 : stage + 1;
    const unsigned char* s1 = own + (size_t)stage * stage_bytes;
    F2 d[4], v[4];
    if (!kAhead && kFirst > 0) {
      first_sums(s0, t, s, h, x, y);
      join(std::integral_constant<int, 0>(), std::integral_constant<int, kFirst>());
    }
    if (has_d) {
      take(s0, 0, a.dho, a.lddho, t, d);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = zero;
    }
    if (NEXT) {
      const float r = rsqrtf(s[0] * inv_h + a.eps);
      const float m = -(s[NEXT ? 1 : 0] * inv_h * r);  // -mean(w' dx n), n = h' r
      const F2 r2 = f2(r, r), m2 = f2(m, m);
      if (kAhead) {
        take(s0, at_h, a.ho, a.ldho, t, h);
        take(s0, at_x, a.dx, a.lddx, t, x);
      }
      raw_pairs<NT>(wn, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const F2 n = mul2(h[e], r2);
        d[e] = fma2(r2, fma2(n, m2, mul2(v[e], x[e])), d[e]);
        sn[e] = fma2(x[e], n, sn[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = mul2(alpha, d[e]);
    put(a.dh, a.lddh, t, v);
    const float q = NORM_Y ? rsqrtf(s[NORM_Y && NEXT ? 2 : 0] * inv_h + a.eps) : 1.f;
    const F2 q2 = f2(q, q);
    if constexpr (HAS_Y) {
      F2 g[4], u[4], z0 = zero, z1 = zero;           // sum w du n, sum d u
      if (kAhead || !NORM_Y) take(s0, at_y, a.y, a.ldy, t, y);
      if (full) {
        take(s0, at_g, a.gate, a.ldg, t, g);
      } else if (GATE == MOE_GATE_TOKEN) {
        const float k = static_cast<const float*>(a.gate)[t];
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = f2(k, k);
      } else {
        raw_pairs<NT>(gc, g);
      }
      raw_pairs<NT>(w, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[e] = mul2(y[e], q2);
        u[e] = mul2(d[e], mul2(y[e], v[e]));         // d u
        d[e] = mul2(d[e], g[e]);                     // du
      }
      if (full) {
        if (a.dgate) put(a.dgate, a.lddg, t, u);
      } else if (GATE == MOE_GATE_CHANNEL) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sg[e] = add2(sg[e], u[e]);
      } else if (GATE == MOE_GATE_TOKEN) {
#pragma unroll
        for (int e = 0; e < 4; ++e) z1 = add2(z1, u[e]);
        s[kFirst + kSecond - 1] = sum_of(z1);
      }
      if (NORM_Y) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sw[e] = fma2(d[e], y[e], sw[e]);
          d[e] = mul2(d[e], v[e]);
          z0 = fma2(d[e], y[e], z0);
        }
        s[kFirst] = sum_of(z0);
      }
    }
    F2 ny[4];
    if (kAhead) first_sums(s1, t, s, h, x, ny);   // past the last row the ring holds an older one, not used
    if (kAhead) join(std::integral_constant<int, 0>(), std::integral_constant<int, kBoth>());
    else if (kSecond > 0) join(std::integral_constant<int, kFirst>(), std::integral_constant<int, kSecond>());
    if constexpr (HAS_Y) {
      if (GATE == MOE_GATE_TOKEN && a.dgate && tid == 0) static_cast<float*>(a.dgate)[t] = s[kFirst + kSecond - 1];
      if (NORM_Y) {
        const float m = -(s[kFirst] * inv_h);
        const F2 m2 = f2(m, m);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = mul2(q2, fma2(y[e], m2, d[e]));
      }
      put(a.dy, a.lddy, t, d);
    }
  }
  auto leave = [&](float* out, int i, const F2(&p)[4]) {
    if (!out) return;
    float* row = gridDim.x == 1 ? out : a.part + ((int64_t)blockIdx.x * kSums + i) * a.part_ld;
    if constexpr (NT > 0) return store8<NT>(row, 0, nt, tid, H, p);
    Raw8<float> r;
    from_pairs(p, r);
    const bool words = (reinterpret_cast<uintptr_t>(row) & 15) == 0;      // a caller's vector may lie anywhere
#pragma unroll
    for (int j = 0; j < 2; ++j) {                    // four columns at a time
      const int n = word_col<T>(W == 1 ? 0 : j, nt, tid) + (W == 1 ? 4 * j : 0);
      if (n >= H) continue;
      if (words) {
        *reinterpret_cast<float4*>(row + n) = make_float4(r.v[4 * j], r.v[4 * j + 1], r.v[4 * j + 2], r.v[4 * j + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) row[n + e] = r.v[4 * j + e];
      }
    }
  };
  leave(a.dw, 0, sw);
  leave(GATE == MOE_GATE_CHANNEL ? static_cast<float*>(a.dgate) : nullptr, 1, sg);
  leave(a.dw_next, 2, sn);
}

// What a call has is a template argument: with the branches taken at run time a thread issued 550
// instructions per row of 8 values, without them 368 (108.9 against 89.7 us at T = 8192, H = 4096).
template <typename T, int MAXT, int NT, bool HAS_Y, bool NORM_Y, bool NEXT, int GATE>
int launch_one(const BackArgs& a, int blocks, int nt, int stages, int stage_bytes, cudaStream_t s) {
  auto kern = norm_backward_ring_kernel<T, MAXT, NT, HAS_Y, NORM_Y, NEXT, GATE>;
  // the shared-memory limit is a property of the kernel on a device: set on its first launch there
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  if (int rc = check_cuda(cudaGetDevice(&dev), "norm_backward_ring_kernel: device")) return rc;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    if (int rc = check_cuda(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes),
                            "norm_backward_ring_kernel: shared memory"))
      return rc;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  return check_cuda(launch_pdl(kern, dim3(blocks), dim3(nt), (size_t)stages * stage_bytes, s, a, stages, stage_bytes),
                    "norm_backward_ring_kernel");
}

template <typename T, int MAXT, int NT, bool NORM_Y, bool NEXT>
int by_gate(const BackArgs& a, int blocks, int nt, int stages, int stage_bytes, cudaStream_t s) {
  switch (a.gate_mode) {
    case MOE_GATE_CHANNEL:
      return launch_one<T, MAXT, NT, true, NORM_Y, NEXT, MOE_GATE_CHANNEL>(a, blocks, nt, stages, stage_bytes, s);
    case MOE_GATE_TOKEN:
      return launch_one<T, MAXT, NT, true, NORM_Y, NEXT, MOE_GATE_TOKEN>(a, blocks, nt, stages, stage_bytes, s);
    case MOE_GATE_FULL:
      return launch_one<T, MAXT, NT, true, NORM_Y, NEXT, MOE_GATE_FULL>(a, blocks, nt, stages, stage_bytes, s);
    default:
      return launch_one<T, MAXT, NT, true, NORM_Y, NEXT, MOE_GATE_NONE>(a, blocks, nt, stages, stage_bytes, s);
  }
}

template <typename T, int MAXT, int NT>
int by_flags(const BackArgs& a, int blocks, int nt, int stages, int stage_bytes, cudaStream_t s) {
  if (!a.has_y)
    return launch_one<T, MAXT, NT, false, false, true, MOE_GATE_NONE>(a, blocks, nt, stages, stage_bytes, s);
  if (a.norm_y)
    return a.next ? by_gate<T, MAXT, NT, true, true>(a, blocks, nt, stages, stage_bytes, s)
                  : by_gate<T, MAXT, NT, true, false>(a, blocks, nt, stages, stage_bytes, s);
  return a.next ? by_gate<T, MAXT, NT, false, true>(a, blocks, nt, stages, stage_bytes, s)
                : by_gate<T, MAXT, NT, false, false>(a, blocks, nt, stages, stage_bytes, s);
}

}  // namespace

template <typename T>
int launch_norm_ring(const BackArgs& a, int blocks, int nt, bool words, int stages, int stage_bytes, cudaStream_t s) {
  if (words)
    return nt <= 256 ? by_flags<T, 256, 0>(a, blocks, nt, stages, stage_bytes, s)
                     : by_flags<T, kRingThreads, 0>(a, blocks, nt, stages, stage_bytes, s);
  if (nt == 128) return by_flags<T, 256, 128>(a, blocks, nt, stages, stage_bytes, s);
  return nt == 256 ? by_flags<T, 256, 256>(a, blocks, nt, stages, stage_bytes, s)
                   : by_flags<T, kRingThreads, kRingThreads>(a, blocks, nt, stages, stage_bytes, s);
}

}  // namespace moe
