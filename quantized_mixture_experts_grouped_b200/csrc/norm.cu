// Norms before and after a block, fused with the block's gate, the scaled residual and the next
// block's norm; and their gradients. The block here is the MoE layer of "Every Expert Counts:
// ExactMoE for Memory-Efficient W4A16 Inference" (Abstract): the residual stream around it stays
// in 16 bits, every statistic and sum is fp32.
//
//   pre   x = rms(h) w                        rms(v) = v r(v),  r(v) = (mean(v^2) + eps)^(-1/2)
//   post  u = rms(y) w (or y);  h' = alpha h + g u;  x' = rms(h') w'
//   Gradient of rms(v) w towards v, applied to d, with n = rms(v):  r (w d - n mean(w d n)).
//
// All of it moves each row once and does some 10 to 25 flops per value: bound by HBM traffic for
// large batches, by the latency of one launch for small ones. A block holds its rows in registers
// (8 or 16 values per thread) between its loads and its stores, so no row is read twice.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "norm_back.cuh"

namespace moe {

namespace {

constexpr int kMaxNormH = 16384;

struct PostArgs {
  const void *y, *h, *w, *gate, *w_next;
  void *h_out, *x_next, *y_out;
  int64_t ldy, ldh, ldg, ldho, ldx, ldyo;
  const int32_t* inv;                // fused combine: y = sum_j wts * yp[inv]
  const float* wts;
  int k, P, T, H, gate_mode;
  bool norm_y, next;
  float alpha, eps;
};

// The value of one weight or gate vector at this thread's columns (ones where there is none).
template <int NT, typename T>
__device__ __forceinline__ void weight8(const void* w, int c, int nt, int tid, int H, F2 (&f)[4]) {
  if (w) {
    load8<NT>(static_cast<const T*>(w), c, nt, tid, H, f);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = f2(1.f, 1.f);
  }
}

// The gate of token t at this thread's columns.
template <int NT, typename T>
__device__ __forceinline__ void gate8(const void* g, int mode, int64_t ld, int64_t t, int c, int nt, int tid, int H,
                                      F2 (&f)[4]) {
  if (mode == MOE_GATE_CHANNEL || mode == MOE_GATE_FULL) {
    load8<NT>(static_cast<const T*>(g) + (mode == MOE_GATE_FULL ? t * ld : 0), c, nt, tid, H, f);
  } else {
    const float v = mode == MOE_GATE_TOKEN ? static_cast<const float*>(g)[t] : 1.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = f2(v, v);
  }
}

// The sum of the squares of a thread's values.
template <int NC>
__device__ __forceinline__ float squares(const F2 (&v)[NC][4]) {
  F2 s = f2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fma2(v[c][e], v[c][e], s);
  return sum_of(s);
}

// A block of the forward kernels has blockDim.y rows of blockDim.x threads: narrow rows share a block,
// so that it has 256 threads (8192 rows of 512 values took 8.9 us with a block each). Rows past the
// last read as zeros and write nothing.
constexpr int kBlockRows = 8;

template <typename T, int NT, int NC, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_pre_kernel(const T* __restrict__ h, int64_t ldh, const T* __restrict__ w,
                                                        float eps, int rows, int H, T* __restrict__ x, int64_t ldx) {
  __shared__ float buf[kBlockRows][32];
  pdl_begin();
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int nt = NT ? NT : blockDim.x, tid = threadIdx.x, live = t < rows ? H : 0;
  F2 v[NC][4], w8[NC][4];
#pragma unroll
  for (int c = 0; c < NC; ++c) load8<NT>(h + t * ldh, c, nt, tid, live, v[c]);
#pragma unroll
  for (int c = 0; c < NC; ++c) weight8<NT, T>(w, c, nt, tid, H, w8[c]);
  float ss[1] = {squares(v)};
  block_sums<1>(ss, buf[threadIdx.y]);
  const float r = rsqrtf(ss[0] / H + eps);
  const F2 r2 = f2(r, r);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[c][e] = mul2(mul2(v[c][e], r2), w8[c][e]);
    store8<NT>(x + t * ldx, c, nt, tid, live, v[c]);
  }
}

// YT: type of the rows y comes from (fused: y is the combine of its token's rows). h_out may be h:
// a thread reads its values of the row before it writes them, and no other thread reads them.
// FUSED: the choices read at a time, 0 for rows that are y itself. Eight blocks per SM cost the form of
// words with one chunk 4 to 8 bytes of spill per thread, four the fused forms of single values 44 to 152.
template <typename T, typename YT, int FUSED, int NT, int NC, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? (NC == 2 || NT > 0 ? 4 : FUSED ? 1 : 8) : 1)
    norm_post_kernel(const PostArgs a) {
  __shared__ float buf[2][kBlockRows][32];
  pdl_begin();
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int nt = NT ? NT : blockDim.x, tid = threadIdx.x, H = a.H, live = t < a.T ? H : 0;
  F2 h[NC][4], y[NC][4], f[4];
  float s[1];
  const T* hrow = static_cast<const T*>(a.h) + t * a.ldh;
#pragma unroll
  for (int c = 0; c < NC; ++c) load8<NT>(hrow, c, nt, tid, live, h[c]);
  if constexpr (FUSED > 0) {
    weighted_rows<FUSED, NC, NT>(static_cast<const YT*>(a.y), a.ldy, a.inv + t * a.k, a.wts + t * a.k, live ? a.k : 0,
                                  a.P, 0, nt, tid, H, y);
    if (a.y_out) {
#pragma unroll
      for (int c = 0; c < NC; ++c) store8<NT>(static_cast<T*>(a.y_out) + t * a.ldyo, c, nt, tid, live, y[c]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c) load8<NT>(static_cast<const YT*>(a.y) + t * a.ldy, c, nt, tid, live, y[c]);
  }
  if (a.norm_y) {
    s[0] = squares(y);
    block_sums<1>(s, buf[0][threadIdx.y]);
    const float q = rsqrtf(s[0] / H + a.eps);
    const F2 q2 = f2(q, q);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      weight8<NT, T>(a.w, c, nt, tid, H, f);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[c][e] = mul2(mul2(y[c][e], q2), f[e]);
    }
  }
  const F2 alpha = f2(a.alpha, a.alpha);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    gate8<NT, T>(a.gate, a.gate_mode, a.ldg, live ? t : 0, c, nt, tid, H, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[c][e] = fma2(alpha, h[c][e], mul2(f[e], y[c][e]));
    store8<NT>(static_cast<T*>(a.h_out) + t * a.ldho, c, nt, tid, live, h[c]);
  }
  if (!a.next) return;
  s[0] = squares(h);
  block_sums<1>(s, buf[1][threadIdx.y]);
  const float r = rsqrtf(s[0] / H + a.eps);
  const F2 r2 = f2(r, r);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    weight8<NT, T>(a.w_next, c, nt, tid, H, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[c][e] = mul2(mul2(h[c][e], r2), f[e]);
    store8<NT>(static_cast<T*>(a.x_next) + t * a.ldx, c, nt, tid, live, h[c]);
  }
}

// The gradient for rows too wide for the ring (norm_ring.cuh; above 4096 values). One block takes rows
// blockIdx.x, + gridDim.x, ...; every thread keeps the same columns, so the sums over the tokens stay
// with it and leave once per block, as partial sums that norm_sums_kernel adds in block order (no atomics:
// bit-identical run to run). 1024 threads leave 64 registers for three such sums, four tensors and the
// row's values: every form spills, 296 to 460 bytes per thread with one chunk (up to 8192 values), 800 to
// 1472 with two, and a row's loads wait for the sums of the row before. Right, not fast: T = 4096, bf16, both
// norms: 208 us at H = 7168 and 1240 at 16384, where the bytes take 54 and 123.
template <typename T, int NT, int NC>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const BackArgs a) {
  __shared__ float buf[2][32 * 4];
  int flip = 0;                    // the buffer of the next block-wide sums: never the one of the last
  pdl_begin();
  const int nt = NT ? NT : blockDim.x, tid = threadIdx.x, H = a.H;
  const float inv_h = 1.f / (float)H;
  const F2 zero = f2(0.f, 0.f), alpha = f2(a.alpha, a.alpha);
  F2 sw[NC][4], sg[NC][4], sn[NC][4];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) sw[c][e] = sg[c][e] = sn[c][e] = zero;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    F2 d[NC][4], y[NC][4], h[NC][4], x[NC][4], f[4];
    F2 p0 = zero, p1 = zero, p2 = zero;     // sum h'^2, sum w' dx h', sum y^2
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int e = 0; e < 4; ++e) d[c][e] = zero;
      if (a.dho) load8<NT>(static_cast<const T*>(a.dho) + t * a.lddho, c, nt, tid, H, d[c]);
      if (a.has_y) load8<NT>(static_cast<const T*>(a.y) + t * a.ldy, c, nt, tid, H, y[c]);
      if (a.next) {
        load8<NT>(static_cast<const T*>(a.ho) + t * a.ldho, c, nt, tid, H, h[c]);
        load8<NT>(static_cast<const T*>(a.dx) + t * a.lddx, c, nt, tid, H, x[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (a.next) {
        weight8<NT, T>(a.w_next, c, nt, tid, H, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p0 = fma2(h[c][e], h[c][e], p0);
          p1 = fma2(mul2(f[e], x[c][e]), h[c][e], p1);
        }
      }
      if (a.norm_y) {
#pragma unroll
        for (int e = 0; e < 4; ++e) p2 = fma2(y[c][e], y[c][e], p2);
      }
    }
    float s[3] = {sum_of(p0), sum_of(p1), sum_of(p2)};
    if (a.next || a.norm_y) {
      block_sums<3>(s, buf[flip]);
      flip ^= 1;
    }
    if (a.next) {
      const float r = rsqrtf(s[0] * inv_h + a.eps);
      const float m = -(s[1] * inv_h * r);           // -mean(w' dx n), n = h' r
      const F2 r2 = f2(r, r), m2 = f2(m, m);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        weight8<NT, T>(a.w_next, c, nt, tid, H, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const F2 n = mul2(h[c][e], r2);
          d[c][e] = fma2(r2, fma2(n, m2, mul2(f[e], x[c][e])), d[c][e]);
          sn[c][e] = fma2(x[c][e], n, sn[c][e]);
        }
      }
    }
    // dh = alpha d
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = mul2(alpha, d[c][e]);
      store8<NT>(static_cast<T*>(a.dh) + t * a.lddh, c, nt, tid, H, f);
    }
    if (!a.has_y) continue;
    const float q = a.norm_y ? rsqrtf(s[2] * inv_h + a.eps) : 1.f;
    const F2 q2 = f2(q, q);
    F2 z0 = zero, z1 = zero;                         // sum w du n, sum d u
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      F2 g[4], u[4];
      weight8<NT, T>(a.norm_y ? a.w : nullptr, c, nt, tid, H, f);
      gate8<NT, T>(a.gate, a.gate_mode, a.ldg, t, c, nt, tid, H, g);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[c][e] = mul2(y[c][e], q2);
        u[e] = mul2(d[c][e], mul2(y[c][e], f[e]));   // d u
        z1 = add2(z1, u[e]);
        d[c][e] = mul2(d[c][e], g[e]);               // du
        if (a.gate_mode == MOE_GATE_CHANNEL) sg[c][e] = add2(sg[c][e], u[e]);
        if (a.norm_y) sw[c][e] = fma2(d[c][e], y[c][e], sw[c][e]);
        d[c][e] = mul2(d[c][e], f[e]);
        z0 = fma2(d[c][e], y[c][e], z0);
      }
      if (a.gate_mode == MOE_GATE_FULL && a.dgate)
        store8<NT>(static_cast<T*>(a.dgate) + t * a.lddg, c, nt, tid, H, u);
    }
    float z[2] = {sum_of(z0), sum_of(z1)};
    if (a.norm_y || a.gate_mode == MOE_GATE_TOKEN) {
      block_sums<2>(z, buf[flip]);
      flip ^= 1;
    }
    if (a.gate_mode == MOE_GATE_TOKEN && a.dgate && tid == 0) static_cast<float*>(a.dgate)[t] = z[1];
    const float m = a.norm_y ? -(z[0] * inv_h) : 0.f;
    const F2 m2 = f2(m, m);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (a.norm_y) {
#pragma unroll
        for (int e = 0; e < 4; ++e) d[c][e] = mul2(q2, fma2(y[c][e], m2, d[c][e]));
      }
      store8<NT>(static_cast<T*>(a.dy) + t * a.lddy, c, nt, tid, H, d[c]);
    }
  }
  float* out[kSums] = {a.dw, a.gate_mode == MOE_GATE_CHANNEL ? static_cast<float*>(a.dgate) : nullptr, a.dw_next};
#pragma unroll
  for (int i = 0; i < kSums; ++i) {
    if (!out[i]) continue;
    float* o = gridDim.x == 1 ? out[i] : a.part + ((int64_t)blockIdx.x * kSums + i) * a.part_ld;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      Raw8<float> v;
      from_pairs(i == 0 ? sw[c] : i == 1 ? sg[c] : sn[c], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int n = col_of<NT>(c, e, nt, tid);
        if (n < H) o[n] = v.v[e];
      }
    }
  }
}

// Adds the blocks' partial sums: a block has 4 * L columns (L lanes of 16 bytes) by 1024 / L runs, run i
// taking the blocks i, i + runs, ... in order; then the runs are added in a fixed tree. A run is at most
// five blocks long (one turn of loads): with 19 after one another the sums of 592 blocks took 4.5 us.
struct Sums {
  float* out[kSums];               // the sums asked for, and which of the partial sums each is
  int which[kSums];
};
template <int L>
__global__ void __launch_bounds__(1024) norm_sums_kernel(const float* __restrict__ part, int blocks, int H, int ld,
                                                         const Sums s) {
  constexpr int kCols = 4 * L, kRuns = 1024 / L;
  __shared__ float sum[32][kCols + 1];
  pdl_begin();
  float* out = s.out[blockIdx.y];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, run = threadIdx.x / L;
  const int n = blockIdx.x * kCols + (lane & (L - 1)) * 4;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (n < H) {
    const float* p = part + (int64_t)s.which[blockIdx.y] * ld + n;
#pragma unroll 5
    for (int b = run; b < blocks; b += kRuns) {
      const float4 x = *reinterpret_cast<const float4*>(p + (int64_t)b * kSums * ld);
      v[0] += x.x;
      v[1] += x.y;
      v[2] += x.z;
      v[3] += x.w;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (lane < L) sum[warp][lane * 4 + i] = v[i];
  }
  __syncthreads();
  if (warp >= kCols) return;
  float total = sum[lane][warp];       // warp w adds column w of the 32 warps
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int col = blockIdx.x * kCols + warp;
  if (lane == 0 && col < H) out[col] = total;
}

// ---- host side ----

// Threads and chunks per thread for rows of H values, and rows of a block.
struct Shape {
  int nt, nc, ny;
};
// Backward: one row at a time, one chunk up to 8192 values (`words`: rows of 16-byte words; single values
// take one of the block sizes that are built).
Shape shape_of(int H, bool words) {
  if (!words) {
    const int nt = H <= 1024 ? 128 : H <= 2048 ? 256 : H <= 4096 ? 512 : 1024;
    return {nt, H <= 8 * nt ? 1 : 2, 1};
  }
  const int nt = row_threads(H, 1024);
  if (H <= 8 * nt) return {nt, 1, 1};
  return {row_threads(parts_of(H, 2), 1024), 2, 1};
}
// Forward, up to 4096 values: 256 threads, with two chunks per thread (half as many exchanges per row,
// twice the loads in flight per thread: T = 2048, H = 2048, bf16, post with next norm 6.2 us against
// 7.1), but one up to 256 rows of 2048 values, where a row's own latency counts (2.2 against 2.4 at
// T = 1); up to 256 wider rows take one chunk in more threads too, as any do from 4097 on. Single values:
// two chunks from 1025 on.
Shape shape_forward(int rows, int H, bool words) {
  if (!words) {
    const int nc = H <= 1024 ? 1 : 2, nt = H <= 256 ? 32 : H <= 2048 ? 128 : H <= 4096 ? 256 : 1024;
    return {nt, nc, nt > 256 ? 1 : 256 / nt};
  }
  if (H > 4096 || (H > 2048 && rows <= 256)) return shape_of(H, true);
  const int nc = H <= 256 || (H <= 2048 && rows <= 256) ? 1 : 2, nt = row_threads(parts_of(H, nc), 256);
  return {nt, nc, 256 / nt < kBlockRows ? 256 / nt : kBlockRows};
}
// Calls f(threads, chunks) as integral constants for the forward shape of single values.
template <typename F>
auto by_values(const Shape& sh, F f) {
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  if (sh.nt == 32) return f(std::integral_constant<int, 32>(), One());
  if (sh.nt == 128 && sh.nc == 1) return f(std::integral_constant<int, 128>(), One());
  if (sh.nt == 128) return f(std::integral_constant<int, 128>(), Two());
  if (sh.nt == 256) return f(std::integral_constant<int, 256>(), Two());
  return f(std::integral_constant<int, 1024>(), Two());
}

// Calls f(typed null pointer) for the row type.
template <typename F>
int by_type(int dtype, F f) {
  if (dtype == MOE_DTYPE_BF16) return f((__nv_bfloat16*)nullptr);
  if (dtype == MOE_DTYPE_F16) return f((__half*)nullptr);
  return f((float*)nullptr);
}

int norm_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = 148;
  }
  return n;
}

// Blocks of the backward kernel: what the SMs hold at a time, and no more than these, so that the
// workspace's size does not depend on the device.
int most_blocks(int H) { return 148 * ring_blocks(row_threads(H, 1024), false); }
int back_blocks(int T, int H, int per_sm) {
  const int b = norm_sms() * per_sm, most = most_blocks(H);
  return T < b ? T : b < most ? b : most;
}
int part_stride(int H) { return (H + 3) / 4 * 4; }
size_t norm_ws(int T, int H) {
  const size_t most = most_blocks(H), b = (size_t)T < most ? (T > 0 ? T : 1) : most;
  return align_up(b * kSums * part_stride(H) * sizeof(float), 256);
}

int check_norm(const char* me, int T, int H, int dtype, float eps) {
  if (T < 0 || H < 1) return fail(MOE_ERR_ARG, "%s: bad sizes T=%d H=%d", me, T, H);
  if (H > kMaxNormH) return fail(MOE_ERR_SHAPE, "%s: H=%d exceeds %d", me, H, kMaxNormH);
  if (!dtype_size(dtype)) return fail(MOE_ERR_ARG, "%s: unknown type %d", me, dtype);
  if (!(eps > 0.f) || eps > 1e30f) return fail(MOE_ERR_ARG, "%s: eps must be positive and finite", me);
  return MOE_OK;
}

// Rows that are written lie apart; rows only read may repeat (stride 0).
int check_ld(const char* me, const char* name, const void* p, int64_t ld, int T, int H, bool written) {
  if (p && (ld < 0 || (written && T > 1 && ld < H)))
    return fail(MOE_ERR_ARG, "%s: row stride %lld of %s (H=%d)", me, (long long)ld, name, H);
  return MOE_OK;
}

int check_gate(const char* me, const void* gate, int mode, int T) {
  if (mode < MOE_GATE_NONE || mode > MOE_GATE_FULL) return fail(MOE_ERR_ARG, "%s: unknown gate mode %d", me, mode);
  if (T > 0 && (mode != MOE_GATE_NONE) != (gate != nullptr))
    return fail(MOE_ERR_ARG, "%s: gate pointer and gate mode %d do not go together", me, mode);
  return MOE_OK;
}

// Whether an output shares its start with one of the others.
bool shares(const void* out, std::initializer_list<const void*> others) {
  return out && std::find(others.begin(), others.end(), out) != others.end();
}

bool gate16(const void* gate, int mode, int64_t ld, size_t z) {
  if (mode == MOE_GATE_CHANNEL) return rows16(gate, 0, z);
  return mode != MOE_GATE_FULL || rows16(gate, ld, z);
}

template <typename T, typename YT, bool FUSED>
int launch_post(const PostArgs& a, int rows, bool vec, cudaStream_t s) {
  const Shape sh = shape_forward(rows, a.H, vec);
  // choices read at a time: eight with one chunk per thread, for few tokens; two with two chunks, which
  // leaves room for four blocks per SM (T = 2048, k = 8, H = 2048, bf16, on one input, partly in L2: 17.2 us,
  // with four at a time in two blocks 22.3, and moe_combine and moe_norm_post one after the other 20.3; on
  // inputs that change 22.0 against 23.1 one after the other)
  constexpr int F8 = FUSED ? 8 : 0, F4 = FUSED ? 4 : 0, F2_ = FUSED ? 2 : 0;
  auto words = [&]() {
    if (sh.nt * sh.ny <= 256)
      return sh.nc == 1 ? norm_post_kernel<T, YT, F8, 0, 1, 256> : norm_post_kernel<T, YT, F2_, 0, 2, 256>;
    return sh.nc == 1 ? norm_post_kernel<T, YT, F4, 0, 1, 1024> : norm_post_kernel<T, YT, F2_, 0, 2, 1024>;
  };
  auto values = [](auto n, auto c) {
    constexpr int N = decltype(n)::value, C = decltype(c)::value;
    return norm_post_kernel<T, YT, C == 1 ? F4 : F2_, N, C, N <= 256 ? 256 : N>;
  };
  auto kern = vec ? words() : by_values(sh, values);
  note_launch();
  return check_cuda(launch_pdl(kern, dim3(parts_of(rows, sh.ny)), dim3(sh.nt, sh.ny), 0, s, a), "norm_post_kernel");
}

// Checks common to moe_norm_post and moe_combine_norm_post; *vec receives whether rows move as words.
int check_post(const char* me, const PostArgs& a, int T, int H, int dtype, int flags, bool* vec) {
  if (int rc = check_norm(me, T, H, dtype, a.eps)) return rc;
  if (flags & ~(MOE_NORM_Y | MOE_NORM_NEXT)) return fail(MOE_ERR_ARG, "%s: unknown flags %d", me, flags);
  if (int rc = check_gate(me, a.gate, a.gate_mode, T)) return rc;
  if (T > 0 && (!a.y || !a.h || !a.h_out || (a.next && !a.x_next))) return fail(MOE_ERR_ARG, "%s: null pointer", me);
  if (T > 0 && ((a.h_out == a.h && a.ldho != a.ldh) || a.h_out == a.y ||
                (a.next && (a.x_next == a.h_out || a.x_next == a.h || a.x_next == a.y))))
    return fail(MOE_ERR_ARG, "%s: outputs overlap", me);
  // every row reads the vectors; of a gate per value a row reads its own values before it writes them
  const bool full = a.gate_mode == MOE_GATE_FULL;
  const void* x = a.next ? a.x_next : nullptr;
  if (T > 0 && (shares(a.h_out, {a.w, a.w_next}) || shares(x, {a.w, a.w_next}) ||
                (shares(a.h_out, {a.gate}) && !(full && a.ldho == a.ldg)) ||
                (shares(x, {a.gate}) && !(full && a.ldx == a.ldg))))
    return fail(MOE_ERR_ARG, "%s: an output overlaps a weight or the gate", me);
  const size_t z = dtype_size(dtype);
  if (int rc = check_ld(me, "h", a.h, a.ldh, T, H, false)) return rc;
  if (int rc = check_ld(me, "h_out", a.h_out, a.ldho, T, H, true)) return rc;
  if (a.next)
    if (int rc = check_ld(me, "x_next", a.x_next, a.ldx, T, H, true)) return rc;
  if (a.gate_mode == MOE_GATE_FULL)
    if (int rc = check_ld(me, "gate", a.gate, a.ldg, T, H, false)) return rc;
  *vec = H % 8 == 0 && rows16(a.h, a.ldh, z) && rows16(a.h_out, a.ldho, z) && (!a.norm_y || rows16(a.w, 0, z)) &&
         (!a.next || (rows16(a.w_next, 0, z) && rows16(a.x_next, a.ldx, z))) && gate16(a.gate, a.gate_mode, a.ldg, z);
  return MOE_OK;
}

// The kernel for rows too wide for the ring.
template <typename T>
auto back_kernel(const Shape& sh, bool words) {
  if (words) return sh.nc == 2 ? norm_backward_kernel<T, 0, 2> : norm_backward_kernel<T, 0, 1>;
  return sh.nc == 2 ? norm_backward_kernel<T, 1024, 2> : norm_backward_kernel<T, 1024, 1>;
}

int launch_back(const char* me, BackArgs& a, int dtype, bool vec, void* ws, size_t ws_bytes, cudaStream_t s) {
  const bool channel = a.gate_mode == MOE_GATE_CHANNEL;
  float* sums[kSums] = {a.dw, channel ? static_cast<float*>(a.dgate) : nullptr, a.dw_next};
  const bool any = sums[0] || sums[1] || sums[2];
  if (a.T == 0) {    // the sums over no tokens
    for (float* p : sums)
      if (p)
        if (int rc = check_cuda(cudaMemsetAsync(p, 0, sizeof(float) * a.H, s), me)) return rc;
    return MOE_OK;
  }
  const Shape sh = shape_of(a.H, vec);
  // the ring wants three stages (two rows ahead) and takes up to four; fewer blocks share an SM where
  // that needs their shared memory. Two always fit: five fp32 tensors of 4096 values are 80 KB.
  const int tensors = (a.dho ? 1 : 0) + (a.has_y ? 1 : 0) + (a.next ? 2 : 0) + (a.gate_mode == MOE_GATE_FULL ? 1 : 0);
  const int size = (int)dtype_size(dtype), stage_bytes = tensors * (vec ? sh.nt * 8 * size : value_region(a.H, size));
  int per_sm = ring_blocks(sh.nt, a.has_y);
  while (per_sm > 1 && kRingBytes / per_sm / stage_bytes < 3) per_sm /= 2;
  if (per_sm < 1) per_sm = 1;
  const int fit = kRingBytes / per_sm / stage_bytes;
  const int stages = fit < kRingStages ? fit : kRingStages;
  const bool use_ring = sh.nc == 1 && sh.nt <= kRingThreads && stages >= 2;
  // With sums over the tokens a block is worth its partial sums from two rows on, and eight blocks per
  // SM are enough (H = 2048, T = 512: 6.7 us against 8.2 with a row each; H = 1024, T = 1000: 6.7 against
  // 9.7); one or two rows, or up to four narrow ones of words, take one block and no second launch (two rows of
  // 2048: 2.9 us against 3.7; four of 512: 3.3 against 3.4, and 3.7 against 5.1 where the host's time for
  // the launches counts).
  int blocks = back_blocks(a.T, a.H, any && per_sm > 8 ? 8 : per_sm);
  const bool one = a.T <= 2 || (vec && a.T <= 4 && a.T * a.H <= 6144);
  if (any) blocks = one ? 1 : std::min(blocks, std::max(norm_sms(), parts_of(a.T, 2)));
  a.part_ld = part_stride(a.H);
  if (any) {                       // asked for whether or not this call's size uses it
    const size_t need = norm_ws(a.T, a.H);
    if (!ws || ws_bytes < need)
      return fail(MOE_ERR_ARG, "%s: workspace of %zu bytes is smaller than the %zu needed", me, ws ? ws_bytes : 0,
                  need);
    if (reinterpret_cast<uintptr_t>(ws) & 255) return fail(MOE_ERR_ARG, "%s: workspace must be 256-byte aligned", me);
    a.part = static_cast<float*>(ws);
  }
  note_launch();
  int rc = by_type(dtype, [&](auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    if (use_ring) return launch_norm_ring<T>(a, blocks, sh.nt, vec, stages, stage_bytes, s);
    return check_cuda(launch_pdl(back_kernel<T>(sh, vec), dim3(blocks), dim3(sh.nt), 0, s, a), "norm_backward_kernel");
  });
  if (rc || !any || blocks == 1) return rc;
  Sums asked{};
  int n = 0;
  for (int i = 0; i < kSums; ++i) {
    if (!sums[i]) continue;
    asked.out[n] = sums[i];
    asked.which[n++] = i;
  }
  const bool many = blocks > 5 * 128;
  note_launch();
  return check_cuda(launch_pdl(many ? norm_sums_kernel<2> : norm_sums_kernel<8>, dim3(parts_of(a.H, many ? 8 : 32), n),
                               dim3(1024), 0, s, (const float*)a.part, blocks, a.H, a.part_ld, asked),
                    "norm_sums_kernel");
}

}  // namespace

}  // namespace moe

using namespace moe;

MOE_API int moe_norm_workspace_bytes(int T, int H, size_t* bytes) {
  if (!bytes || T < 0 || H < 1) return fail(MOE_ERR_ARG, "moe_norm_workspace_bytes: bad arguments");
  if (H > kMaxNormH) return fail(MOE_ERR_SHAPE, "moe_norm_workspace_bytes: H=%d exceeds %d", H, kMaxNormH);
  *bytes = norm_ws(T, H);
  return MOE_OK;
}

MOE_API int moe_norm_pre(const void* h, int64_t h_stride, int dtype, const void* w, float eps, int T, int H, void* x,
                         int64_t x_stride, moe_stream_t stream) {
  const char* me = "moe_norm_pre";
  if (int rc = check_norm(me, T, H, dtype, eps)) return rc;
  if (T > 0 && (!h || !x)) return fail(MOE_ERR_ARG, "%s: null pointer", me);
  if (T > 0 && (x == h || x == w)) return fail(MOE_ERR_ARG, "%s: x overlaps an input", me);
  if (int rc = check_ld(me, "h", h, h_stride, T, H, false)) return rc;
  if (int rc = check_ld(me, "x", x, x_stride, T, H, true)) return rc;
  if (T == 0) return MOE_OK;
  const size_t z = dtype_size(dtype);
  const bool vec = H % 8 == 0 && rows16(h, h_stride, z) && rows16(x, x_stride, z) && rows16(w, 0, z);
  const Shape sh = shape_forward(T, H, vec);
  note_launch();
  return by_type(dtype, [&](auto* p) {
    using T_ = std::remove_pointer_t<decltype(p)>;
    auto words = [&]() {
      if (sh.nt * sh.ny <= 256) return sh.nc == 1 ? norm_pre_kernel<T_, 0, 1, 256> : norm_pre_kernel<T_, 0, 2, 256>;
      return sh.nc == 1 ? norm_pre_kernel<T_, 0, 1, 1024> : norm_pre_kernel<T_, 0, 2, 1024>;
    };
    auto values = [](auto n, auto c) {
      constexpr int N = decltype(n)::value;
      return norm_pre_kernel<T_, N, decltype(c)::value, N <= 256 ? 256 : N>;
    };
    auto kern = vec ? words() : by_values(sh, values);
    return check_cuda(launch_pdl(kern, dim3(parts_of(T, sh.ny)), dim3(sh.nt, sh.ny), 0,
                                 reinterpret_cast<cudaStream_t>(stream), static_cast<const T_*>(h), h_stride,
                                 static_cast<const T_*>(w), eps, T, H, static_cast<T_*>(x), x_stride),
                      "norm_pre_kernel");
  });
}

MOE_API int moe_norm_pre_backward(const void* dx, int64_t dx_stride, const void* h, int64_t h_stride, int dtype,
                                  const void* w, float eps, int T, int H, const void* dres, int64_t dres_stride,
                                  void* dh, int64_t dh_stride, float* dw, void* workspace, size_t workspace_bytes,
                                  moe_stream_t stream) {
  const char* me = "moe_norm_pre_backward";
  if (int rc = check_norm(me, T, H, dtype, eps)) return rc;
  if (T > 0 && (!dx || !h || !dh)) return fail(MOE_ERR_ARG, "%s: null pointer", me);
  if (T > 0 && (dh == dx || dh == h || dh == w || (dh == dres && dh_stride != dres_stride)))
    return fail(MOE_ERR_ARG, "%s: dh overlaps an input", me);
  if (int rc = check_ld(me, "dx", dx, dx_stride, T, H, false)) return rc;
  if (int rc = check_ld(me, "h", h, h_stride, T, H, false)) return rc;
  if (int rc = check_ld(me, "dres", dres, dres_stride, T, H, false)) return rc;
  if (int rc = check_ld(me, "dh", dh, dh_stride, T, H, true)) return rc;
  const size_t z = dtype_size(dtype);
  const bool vec = H % 8 == 0 && rows16(dx, dx_stride, z) && rows16(h, h_stride, z) && rows16(dres, dres_stride, z) &&
                   rows16(dh, dh_stride, z) && rows16(w, 0, z);
  BackArgs a{};
  a.dho = dres; a.lddho = dres_stride; a.ho = h; a.ldho = h_stride; a.dx = dx; a.lddx = dx_stride;
  a.w_next = w; a.dh = dh; a.lddh = dh_stride; a.dw_next = dw;
  a.T = T; a.H = H; a.gate_mode = MOE_GATE_NONE; a.next = true; a.alpha = 1.f; a.eps = eps;
  return launch_back(me, a, dtype, vec, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

MOE_API int moe_norm_post(const void* y, int64_t y_stride, const void* h, int64_t h_stride, int dtype, const void* w,
                          const void* gate, int64_t gate_stride, int gate_mode, float alpha, float eps, int T, int H,
                          int flags, void* h_out, int64_t h_out_stride, const void* w_next, void* x_next,
                          int64_t x_next_stride, moe_stream_t stream) {
  const char* me = "moe_norm_post";
  PostArgs a{};
  a.y = y; a.ldy = y_stride; a.h = h; a.ldh = h_stride; a.w = w; a.gate = gate; a.ldg = gate_stride;
  a.gate_mode = gate_mode; a.alpha = alpha; a.eps = eps; a.T = T; a.H = H;
  a.norm_y = (flags & MOE_NORM_Y) != 0; a.next = (flags & MOE_NORM_NEXT) != 0;
  a.h_out = h_out; a.ldho = h_out_stride; a.w_next = w_next; a.x_next = x_next; a.ldx = x_next_stride;
  bool vec = false;
  if (int rc = check_post(me, a, T, H, dtype, flags, &vec)) return rc;
  if (int rc = check_ld(me, "y", y, y_stride, T, H, false)) return rc;
  if (T == 0) return MOE_OK;
  vec = vec && rows16(y, y_stride, dtype_size(dtype));
  return by_type(dtype, [&](auto* p) {
    using T_ = std::remove_pointer_t<decltype(p)>;
    return launch_post<T_, T_, false>(a, T, vec, reinterpret_cast<cudaStream_t>(stream));
  });
}

MOE_API int moe_combine_norm_post(const void* yp, int64_t yp_stride, int yp_dtype, const int32_t* inv,
                                  const float* wts, int k, const void* h, int64_t h_stride, int dtype, const void* w,
                                  const void* gate, int64_t gate_stride, int gate_mode, float alpha, float eps, int T,
                                  int H, int flags, void* h_out, int64_t h_out_stride, const void* w_next,
                                  void* x_next, int64_t x_next_stride, void* y_out, int64_t y_out_stride,
                                  moe_stream_t stream) {
  const char* me = "moe_combine_norm_post";
  PostArgs a{};
  a.y = yp; a.ldy = yp_stride; a.h = h; a.ldh = h_stride; a.w = w; a.gate = gate; a.ldg = gate_stride;
  a.gate_mode = gate_mode; a.alpha = alpha; a.eps = eps; a.T = T; a.H = H;
  a.norm_y = (flags & MOE_NORM_Y) != 0; a.next = (flags & MOE_NORM_NEXT) != 0;
  a.h_out = h_out; a.ldho = h_out_stride; a.w_next = w_next; a.x_next = x_next; a.ldx = x_next_stride;
  a.y_out = y_out; a.ldyo = y_out_stride; a.inv = inv; a.wts = wts; a.k = k;
  if (k < 1) return fail(MOE_ERR_ARG, "%s: k=%d", me, k);
  bool vec = false;
  if (int rc = check_post(me, a, T, H, dtype, flags, &vec)) return rc;
  if ((int64_t)T * k > INT32_MAX) return fail(MOE_ERR_SHAPE, "%s: T*k exceeds 2^31-1", me);
  a.P = T * k;
  if (!dtype_size(yp_dtype) || (yp_dtype != dtype && yp_dtype != MOE_DTYPE_F32))
    return fail(MOE_ERR_ARG, "%s: rows of type %d with results of type %d", me, yp_dtype, dtype);
  if (T > 0 && (!inv || !wts)) return fail(MOE_ERR_ARG, "%s: null pointer", me);
  if (shares(y_out, {yp, h, h_out, x_next, w, gate, w_next}))     // written before the gate and the weights are read
    return fail(MOE_ERR_ARG, "%s: y_out overlaps another tensor", me);
  if (int rc = check_ld(me, "yp", yp, yp_stride, T, H, false)) return rc;
  if (int rc = check_ld(me, "y_out", y_out, y_out_stride, T, H, true)) return rc;
  if (T == 0) return MOE_OK;
  vec = vec && rows16(yp, yp_stride, dtype_size(yp_dtype)) && rows16(y_out, y_out_stride, dtype_size(dtype));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return by_type(dtype, [&](auto* p) {
    using T_ = std::remove_pointer_t<decltype(p)>;
    return yp_dtype == dtype ? launch_post<T_, T_, true>(a, T, vec, s) : launch_post<T_, float, true>(a, T, vec, s);
  });
}

MOE_API int moe_norm_post_backward(const void* dh_out, int64_t dh_out_stride, const void* y, int64_t y_stride,
                                   int dtype, const void* w, const void* gate, int64_t gate_stride, int gate_mode,
                                   float alpha, float eps, int T, int H, int flags, const void* h_out,
                                   int64_t h_out_stride, const void* w_next, const void* dx_next,
                                   int64_t dx_next_stride, void* dh, int64_t dh_stride, void* dy, int64_t dy_stride,
                                   float* dw, void* dgate, int64_t dgate_stride, float* dw_next, void* workspace,
                                   size_t workspace_bytes, moe_stream_t stream) {
  const char* me = "moe_norm_post_backward";
  if (int rc = check_norm(me, T, H, dtype, eps)) return rc;
  if (flags & ~(MOE_NORM_Y | MOE_NORM_NEXT)) return fail(MOE_ERR_ARG, "%s: unknown flags %d", me, flags);
  if (int rc = check_gate(me, gate, gate_mode, T)) return rc;
  const bool norm_y = flags & MOE_NORM_Y, next = flags & MOE_NORM_NEXT;
  if (T > 0 && (!dh_out || !y || !dh || !dy || (next && (!h_out || !dx_next))))
    return fail(MOE_ERR_ARG, "%s: null pointer", me);
  if ((dw && !norm_y) || (dw_next && !next) || (dgate && gate_mode == MOE_GATE_NONE))
    return fail(MOE_ERR_ARG, "%s: gradient asked of something that the call does not have", me);
  const bool full = gate_mode == MOE_GATE_FULL;
  if (T > 0 && ((dh == dh_out && dh_stride != dh_out_stride) || dh == y || dh == dy || dy == dh_out || dy == y ||
                (next && (dh == h_out || dh == dx_next || dy == h_out || dy == dx_next)) ||
                (full && (dh == gate || dy == gate)) ||
                (full && dgate && (dgate == dh || dgate == dy || dgate == gate || dgate == y || dgate == dh_out ||
                                   (next && (dgate == h_out || dgate == dx_next))))))
    return fail(MOE_ERR_ARG, "%s: an output overlaps another tensor", me);
  if (T > 0 && (shares(dh, {w, gate, w_next}) || shares(dy, {w, gate, w_next}) || shares(dgate, {w, w_next})))
    return fail(MOE_ERR_ARG, "%s: an output overlaps a weight or the gate", me);
  if (shares(dw, {dw_next, dgate}) || shares(dw_next, {dgate}))
    return fail(MOE_ERR_ARG, "%s: two gradients share a buffer", me);
  if (int rc = check_ld(me, "dh_out", dh_out, dh_out_stride, T, H, false)) return rc;
  if (int rc = check_ld(me, "y", y, y_stride, T, H, false)) return rc;
  if (int rc = check_ld(me, "dh", dh, dh_stride, T, H, true)) return rc;
  if (int rc = check_ld(me, "dy", dy, dy_stride, T, H, true)) return rc;
  if (next) {
    if (int rc = check_ld(me, "h_out", h_out, h_out_stride, T, H, false)) return rc;
    if (int rc = check_ld(me, "dx_next", dx_next, dx_next_stride, T, H, false)) return rc;
  }
  if (full) {
    if (int rc = check_ld(me, "gate", gate, gate_stride, T, H, false)) return rc;
    if (int rc = check_ld(me, "dgate", dgate, dgate_stride, T, H, true)) return rc;
  }
  const size_t z = dtype_size(dtype);
  const bool vec = H % 8 == 0 && rows16(dh_out, dh_out_stride, z) && rows16(y, y_stride, z) &&
                   rows16(dh, dh_stride, z) && rows16(dy, dy_stride, z) && (!norm_y || rows16(w, 0, z)) &&
                   (!next || (rows16(h_out, h_out_stride, z) && rows16(dx_next, dx_next_stride, z) &&
                              rows16(w_next, 0, z))) &&
                   gate16(gate, gate_mode, gate_stride, z) && (!full || rows16(dgate, dgate_stride, z));
  BackArgs a{};
  a.dho = dh_out; a.lddho = dh_out_stride; a.y = y; a.ldy = y_stride; a.ho = h_out; a.ldho = h_out_stride;
  a.dx = dx_next; a.lddx = dx_next_stride; a.w = w; a.gate = gate; a.ldg = gate_stride; a.w_next = w_next;
  a.dh = dh; a.lddh = dh_stride; a.dy = dy; a.lddy = dy_stride; a.dgate = dgate; a.lddg = dgate_stride;
  a.dw = dw; a.dw_next = dw_next; a.T = T; a.H = H; a.gate_mode = gate_mode;
  a.has_y = true; a.norm_y = norm_y; a.next = next; a.alpha = alpha; a.eps = eps;
  return launch_back(me, a, dtype, vec, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}
