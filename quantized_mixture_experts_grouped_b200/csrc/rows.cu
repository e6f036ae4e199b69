// Token rows sorted by expert and back, with the router's weights, and their gradients (the steps
// around the experts' products of "Every Expert Counts: ExactMoE for Memory-Efficient W4A16
// Inference", Abstract: all selected experts run through fused grouped kernels).
//
//   sort      pair p = t*k+j of expert e goes to place offsets[e] + #{p' < p : e' = e}
//   dispatch  xp[place] = x[t]                    gradient: dx[t] = sum_j dxp[inv[t][j]]
//   combine   out[t] = sum_j w[t][j] yp[inv[t][j]]
//             gradient: dyp[inv[t][j]] = w[t][j] dout[t],  dw[t][j] = <dout[t], yp[inv[t][j]]>
//   router    w = softmax over the k chosen logits, so dlogit[idx_j] = w_j (dw_j - sum_i w_i dw_i)
//
// All of it is bound by HBM traffic (large batches) or by the latency of a launch (small ones), so
// every row is read once and written once, and each operator is one launch, the sort of a large
// batch one more. Sums are fp32 in a fixed order; each result is rounded once, to its own type.
#include <cooperative_groups.h>

#include <type_traits>

#include "rows.cuh"

namespace moe {

namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------------------------- sort

constexpr int kSortThreads = 1024;
constexpr int kSortCluster = 8;

// Turns the warps' counts per expert into the counts of the warps before each, and total[e] into
// their sum: eight neighbouring lanes share an expert, four warps each. All 32 warps call it.
__device__ __forceinline__ void prefix_warps(int32_t (*wcount)[kMaxExperts], int E, int32_t* total) {
  for (int i = threadIdx.x; i < (E + 3) / 4 * 32; i += kSortThreads) {
    const int e = i >> 3, part = i & 7;
    int c[4], sum = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      c[w] = e < E ? wcount[part * 4 + w][e] : 0;
      sum += c[w];
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o, 8);
      if (part >= o) run += v;
    }
    if (e < E && part == 7) total[e] = run;
    run -= sum;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (e < E) wcount[part * 4 + w][e] = run;
      run += c[w];
    }
  }
}

// Inclusive prefix of v over the block's first kMaxExperts threads (0 from the others); the caller
// has a barrier between this and the next use of wsum.
__device__ __forceinline__ int prefix_experts(int v, int32_t* wsum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (threadIdx.x < kMaxExperts && lane == 31) wsum[warp] = v;
  __syncthreads();
  if (threadIdx.x < kMaxExperts)
    for (int w = 0; w < warp; ++w) v += wsum[w];
  return v;
}

// Stable counting sort of the P pairs by expert in ONE launch: a cluster of blocks, each with a
// contiguous run of pairs, each warp with a contiguous part of the block's run. A warp counts its
// pairs per expert (warp match, so equal ids cost one add), the block prefixes its warps' counts,
// the cluster exchanges the blocks' counts through distributed shared memory, and the warps walk
// their pairs once more to place them. Integer counts: the result does not depend on timing.
__global__ void __launch_bounds__(kSortThreads) sort_pairs_kernel(const int32_t* __restrict__ idx, int P, int E,
                                                                  int32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ perm,
                                                                  int32_t* __restrict__ inv) {
  __shared__ int32_t wcount[kSortThreads / 32][kMaxExperts];
  __shared__ int32_t total[kMaxExperts];
  __shared__ int32_t first[kMaxExperts];
  __shared__ int32_t wsum[kMaxExperts / 32];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int nw = kSortThreads / 32;
  const int per_block = (int)(((int64_t)P + kSortCluster - 1) / kSortCluster);
  const int per_warp = (per_block + 32 * nw - 1) / (32 * nw) * 32;
  const int64_t b0 = (int64_t)rank * per_block, b1 = min(b0 + per_block, (int64_t)P);
  const int64_t w0 = b0 + (int64_t)warp * per_warp, w1 = min(w0 + per_warp, b1);
  for (int e = lane; e < E; e += 32) wcount[warp][e] = 0;
  pdl_begin();
  __syncwarp();
  for (int64_t p0 = w0; p0 < w1; p0 += 32) {
    int e = p0 + lane < w1 ? idx[p0 + lane] : -1;
    if ((unsigned)e >= (unsigned)E) e = -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && (same & ((1u << lane) - 1u)) == 0) wcount[warp][e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  prefix_warps(wcount, E, total);
  cluster.sync();
  // each block: pairs of expert e in the blocks before it, and in all of them
  int all = 0, before = 0;
  const int e0 = threadIdx.x;
  if (e0 < E) {
    int c[kSortCluster];
#pragma unroll
    for (int r = 0; r < kSortCluster; ++r) c[r] = *cluster.map_shared_rank(&total[e0], r);
#pragma unroll
    for (int r = 0; r < kSortCluster; ++r) {
      if (r < rank) before += c[r];
      all += c[r];
    }
  }
  cg::cluster_group::arrival_token done = cluster.barrier_arrive();   // the others' counts are read
  const int incl = prefix_experts(all, wsum);
  if (e0 < E) {
    first[e0] = incl - all + before;
    if (rank == 0) {
      counts[e0] = all;
      offsets[e0] = incl - all;
      if (e0 == E - 1) offsets[E] = incl;
    }
  }
  __syncthreads();
  for (int64_t p0 = w0; p0 < w1; p0 += 32) {
    const int64_t p = p0 + lane;
    int e = p < w1 ? idx[p] : -1;
    if ((unsigned)e >= (unsigned)E) e = -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int lower = __popc(same & ((1u << lane) - 1u));
    int place = -1;
    if (e >= 0) place = first[e] + wcount[warp][e] + lower;
    __syncwarp();
    if (e >= 0 && lower == 0) wcount[warp][e] += __popc(same);
    __syncwarp();
    if (p < w1) inv[p] = place;
    if (place >= 0) perm[place] = (int32_t)p;
  }
  cluster.barrier_wait(std::move(done));   // no block leaves while another reads its counts
}

// ------------------------------------------------------------------------------------- dispatch

constexpr int kRowThreads = 256;
constexpr int kSmallPairs = 2048;

// One token's row to its choices' places; U is the unit moved (16 bytes where the rows allow it).
template <typename U>
__device__ __forceinline__ void copy_row(const U* __restrict__ src, U* xp, int64_t ldp, const int32_t* place, int k,
                                         int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const U v = src[i];
    for (int j = 0; j < k; ++j) {
      const int p = place[j];
      if (p >= 0) xp[(int64_t)p * ldp + i] = v;
    }
  }
}

// 16-bit values on any boundary: a thread takes the values c - 1, c, c + 1 (c even) and writes whole
// 32-bit words, the pair (c, c + 1) where the place starts on one and (c - 1, c) where it does not (a
// value at a time: 26 us against 12 for 2048 tokens of 8 choices in words).
template <>
__device__ __forceinline__ void copy_row<uint16_t>(const uint16_t* __restrict__ src, uint16_t* xp, int64_t ldp,
                                                   const int32_t* place, int k, int n) {
  for (int c = 2 * threadIdx.x; c <= n; c += 2 * blockDim.x) {
    const uint32_t before = c > 0 ? src[c - 1] : 0, here = c < n ? src[c] : 0, after = c + 1 < n ? src[c + 1] : 0;
    const uint32_t even = here | after << 16, odd = before | here << 16;
    for (int j = 0; j < k; ++j) {
      const int p = place[j];
      if (p < 0) continue;
      uint16_t* dst = xp + (int64_t)p * ldp + c;
      if ((reinterpret_cast<uintptr_t>(dst) & 3) == 0) {
        if (c + 1 < n) *reinterpret_cast<uint32_t*>(dst) = even;
        else if (c < n) *dst = (uint16_t)here;
      } else if (c > 0 && c < n) {
        *reinterpret_cast<uint32_t*>(dst - 1) = odd;
      } else if (c == 0) {
        *dst = (uint16_t)here;
      } else {
        dst[-1] = (uint16_t)before;
      }
    }
  }
}

template <typename U>
__global__ void __launch_bounds__(kRowThreads) copy_rows_kernel(const U* __restrict__ x, int64_t ldx,
                                                                const int32_t* __restrict__ inv, int k, int n, U* xp,
                                                                int64_t ldp) {
  pdl_begin();
  const int64_t t = blockIdx.x;
  copy_row(x + t * ldx, xp, ldp, inv + t * k, k, n);
}

// Sort and copy in one launch for few pairs: block t finds its own k places by counting the pairs
// that go before each of them (every block reads all P ids; P * k comparisons per block), then
// copies its row. One more block writes the counts and offsets.
template <typename U>
__global__ void __launch_bounds__(kRowThreads) dispatch_small_kernel(const U* __restrict__ x, int64_t ldx,
                                                                     const int32_t* __restrict__ idx, int T, int E,
                                                                     int k, int n, int32_t* __restrict__ counts,
                                                                     int32_t* __restrict__ offsets,
                                                                     int32_t* __restrict__ perm,
                                                                     int32_t* __restrict__ inv, U* xp, int64_t ldp) {
  __shared__ int32_t es[kSmallPairs];
  __shared__ int32_t place[kSmallPairs];
  __shared__ int32_t wsum[kMaxExperts / 32];
  const int P = T * k, t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  pdl_begin();
  for (int p = threadIdx.x; p < P; p += blockDim.x) {
    const int e = idx[p];
    es[p] = (unsigned)e < (unsigned)E ? e : INT32_MAX;
  }
  if (t == T) {
    for (int e = threadIdx.x; e < kMaxExperts; e += blockDim.x) place[e] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < P; p += blockDim.x)
      if (es[p] < E) atomicAdd(&place[es[p]], 1);
    __syncthreads();
    const int e = threadIdx.x;   // 256 threads, at most 256 experts
    const int c = place[e], incl = prefix_experts(c, wsum);
    if (e < E) {
      counts[e] = c;
      offsets[e] = incl - c;
      if (e == E - 1) offsets[E] = incl;
    }
    return;
  }
  __syncthreads();
  for (int j = warp; j < k; j += nw) {
    const int mine = t * k + j, e = es[mine];
    int lower = 0;
    for (int p = lane; p < P; p += 32) lower += es[p] < e || (es[p] == e && p < mine);
    lower = __reduce_add_sync(0xffffffffu, lower);
    if (lane == 0) {
      place[j] = e < E ? lower : -1;
      inv[mine] = place[j];
      if (e < E) perm[lower] = mine;
    }
  }
  __syncthreads();
  copy_row(x + (int64_t)t * ldx, xp, ldp, place, k, n);
}

template <typename U>
int dispatch_units(const void* x, int64_t ldx, const int32_t* idx, int T, int E, int k, int n, int32_t* counts,
                   int32_t* offsets, int32_t* perm, int32_t* inv, void* xp, int64_t ldp, cudaStream_t s) {
  const U* xs = static_cast<const U*>(x);
  U* xd = static_cast<U*>(xp);
  const int64_t P = (int64_t)T * k;
  if (T > 0 && P <= kSmallPairs) {
    note_launch();
    return check_cuda(launch_pdl(dispatch_small_kernel<U>, dim3(T + 1), dim3(kRowThreads), 0, s, xs, ldx, idx, T, E, k,
                                 n, counts, offsets, perm, inv, xd, ldp),
                      "dispatch_small_kernel");
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kSortCluster);
  cfg.blockDim = dim3(kSortThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kSortCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  note_launch();
  if (int rc = check_cuda(cudaLaunchKernelEx(&cfg, sort_pairs_kernel, idx, (int)P, E, counts, offsets, perm, inv),
                          "sort_pairs_kernel"))
    return rc;
  if (T == 0) return MOE_OK;
  note_launch();
  return check_cuda(launch_pdl(copy_rows_kernel<U>, dim3(T), dim3(kRowThreads), 0, s, xs, ldx, (const int32_t*)inv, k,
                               n, xd, ldp),
                    "copy_rows_kernel");
}

// ------------------------------------------------------------------------------------- combine

template <typename YT, typename OT, int NT, int B, int NC>
__global__ void __launch_bounds__(kRowThreads, NC == 2 || (NT == 0 && sizeof(YT) == 2) || (NT > 0 && B == 4) ? 4 : 1)
    combine_rows_kernel(const YT* __restrict__ yp, int64_t ldy, const int32_t* __restrict__ inv,
                        const float* __restrict__ wts, int T, int k, int P, int H, OT* __restrict__ out, int64_t ldo) {
  pdl_begin();
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= T) return;
  F2 v[NC][4];
  weighted_rows<B, NC, NT>(yp, ldy, inv + t * k, wts ? wts + t * k : nullptr, k, P, blockIdx.y * NC, blockDim.x,
                            threadIdx.x, H, v);
#pragma unroll
  for (int c = 0; c < NC; ++c) store8<NT>(out + t * ldo, blockIdx.y * NC + c, blockDim.x, threadIdx.x, H, v[c]);
}

// Gradient of combine: one block per token. dout's row stays in registers while the token's rows
// pass by: each is read once (its dot product with dout) and its gradient row written once. The
// dot products of up to kDots choices are reduced together at the end of the row.
constexpr int kDots = 8;
constexpr int kFewPairs = 1024;

template <typename YT, typename OT>
__global__ void __launch_bounds__(kRowThreads, 4)
    combine_backward_kernel(const OT* __restrict__ dout, int64_t ldo, const YT* __restrict__ yp, int64_t ldy,
                            const int32_t* __restrict__ inv, const float* __restrict__ wts, int k, int P, int H,
                            YT* __restrict__ dyp, int64_t lddy, float* __restrict__ dwts) {
  __shared__ float buf[2][32 * kDots];
  pdl_begin();
  const int64_t t = blockIdx.x;
  const int nt = blockDim.x, tid = threadIdx.x;
  const int chunks = (H + 8 * nt - 1) / (8 * nt);
  const int32_t* it = inv + t * k;
  const float* wt = wts + t * k;
  int flip = 0;
  for (int j0 = 0; j0 < k; j0 += kDots, flip ^= 1) {
    float w[kDots];
    int pos[kDots];
#pragma unroll
    for (int b = 0; b < kDots; ++b) {
      const bool in = j0 + b < k;
      pos[b] = in ? it[j0 + b] : -1;
      w[b] = in ? wt[j0 + b] : 0.f;
    }
#pragma unroll
    for (int b = 0; b < kDots; ++b)
      if ((unsigned)pos[b] >= (unsigned)P) pos[b] = -1;
    F2 part[kDots];
#pragma unroll
    for (int b = 0; b < kDots; ++b) part[b] = f2(0.f, 0.f);
    for (int c = 0; c < chunks; ++c) {
      F2 d[4];
      load8<0>(dout + t * ldo, c, nt, tid, H, d);
      // four choices' words at a time and four blocks per SM: T = 2048, k = 8, H = 2048 took 54 us for
      // this and moe_dispatch_backward with eight and three, 49 with four and five (spills), 44 like this
      // (fp32 rows spill 24 bytes)
      constexpr int B = 4;
#pragma unroll
      for (int b0 = 0; b0 < kDots; b0 += B) {
        if (j0 + b0 >= k) break;
        Raw8<YT> r[B];
        if (dwts) {
#pragma unroll
          for (int b = 0; b < B; ++b) {
            const bool on = pos[b0 + b] >= 0;
            r[b] = load_raw<0>(yp + (int64_t)(on ? pos[b0 + b] : 0) * ldy, c, nt, tid, on ? H : 0);
          }
        }
        if (dyp) {          // does not wait for yp's rows
#pragma unroll
          for (int b = 0; b < B; ++b) {
            if (j0 + b0 + b >= k) break;
            const F2 w2 = f2(w[b0 + b], w[b0 + b]);
            F2 g[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) g[e] = mul2(w2, d[e]);
            const bool on = pos[b0 + b] >= 0;
            store8<0>(dyp + (int64_t)(on ? pos[b0 + b] : 0) * lddy, c, nt, tid, on ? H : 0, g);
          }
        }
        if (dwts) {
#pragma unroll
          for (int b = 0; b < B; ++b) {
            if (j0 + b0 + b >= k) break;
            F2 v[4];
            raw_pairs<0>(r[b], v);
#pragma unroll
            for (int e = 0; e < 4; ++e) part[b0 + b] = fma2(d[e], v[e], part[b0 + b]);
          }
        }
      }
    }
    if (dwts) {
      float dot[kDots];
#pragma unroll
      for (int b = 0; b < kDots; ++b) dot[b] = sum_of(part[b]);
      block_sums<kDots>(dot, buf[flip]);
#pragma unroll
      for (int b = 0; b < kDots; ++b)
        if (tid == b && j0 + b < k) dwts[t * k + j0 + b] = pos[b] >= 0 ? dot[b] : 0.f;
    }
  }
}

// The same with a block per token and group of G choices: groups do not wait for one another, and dout's
// row, read once per group, comes from L2 after the first. Which form a call takes, with the microseconds
// of groups of 1 / 2 / 4 / 8 and of a block per token (bf16 rows, H = 2048 unless it says otherwise; inputs
// that change from pass to pass):
//   up to 1024 pairs, where latency counts, one choice: T = 1, k = 8: 1.6 against 2.8 per token; 512 pairs:
//     3.1 against 4.8; 1024: 3.9 against 5.2; 2048: 6.3 each
//   one choice, and two of words wider than 1024, one: T = 8192, k = 2: 36 / 39 / 40 / 70 against 50
//   single values, bound by their loads and stores, of which a group shares dout's, four (two of two):
//     T = 2048, k = 8: 49 / 42 / 37 / 42; H = 1031: 39 / 35 / 29 / 35; T = 4096, H = 255: 34 / 18 / 13 / 12
//   two narrow choices of words, two: T = 8192, H = 512: 17 / 12 / 12 / 17 against 14
//   fp32 words from 512 values on, two: T = 2048, k = 8: 51 / 45 / 47 / 51 against 54; k = 4: 27 / 25 / 27 /
//     29 against 31; T = 4096, k = 8, H = 512: 34 / 24 / 25 / 26 against 29; below, H = 256: 34 / 17 / 14 / 14
//     against 18, H = 128: 34 / 17 / 11 / 10 against 8.9
//   other words, a block per token: T = 2048, k = 8: 35 / 37 / 32 / 44 against 27; k = 4: 19 / 20 / 19 / 28
//     against 18; k = 3: 15 / 18 / 16 / 24 against 16
template <typename YT, typename OT, int NT, int G>
__global__ void __launch_bounds__(kRowThreads)
    combine_group_backward_kernel(const OT* __restrict__ dout, int64_t ldo, const YT* __restrict__ yp, int64_t ldy,
                                 const int32_t* __restrict__ inv, const float* __restrict__ wts, int k, int P, int H,
                                 YT* __restrict__ dyp, int64_t lddy, float* __restrict__ dwts) {
  __shared__ float buf[32 * G];
  pdl_begin();
  const int groups = (k + G - 1) / G;
  const int nt = NT ? NT : blockDim.x, tid = threadIdx.x;
  const int t = blockIdx.x / groups, j0 = (blockIdx.x - t * groups) * G;
  const int64_t first = (int64_t)t * k + j0;
  int pos[G];
  float w[G];
  bool any = false;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const bool in = j0 + g < k;
    pos[g] = in ? inv[first + g] : -1;
    w[g] = in ? wts[first + g] : 0.f;
    if ((unsigned)pos[g] >= (unsigned)P) pos[g] = -1;
    any |= pos[g] >= 0;
  }
  if (!any) {
    if (dwts && tid < G && j0 + tid < k) dwts[first + tid] = 0.f;
    return;
  }
  const OT* drow = dout + (int64_t)t * ldo;
  const int chunks = (H + 8 * nt - 1) / (8 * nt);
  F2 part[G];
#pragma unroll
  for (int g = 0; g < G; ++g) part[g] = f2(0.f, 0.f);
#pragma unroll 2
  for (int c = 0; c < chunks; ++c) {
    F2 d[4];
    load8<NT>(drow, c, nt, tid, H, d);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (pos[g] < 0) continue;
      if (dwts) {
        F2 v[4];
        load8<NT>(yp + (int64_t)pos[g] * ldy, c, nt, tid, H, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) part[g] = fma2(d[e], v[e], part[g]);
      }
      if (dyp) {
        F2 o[4];
        const F2 w2 = f2(w[g], w[g]);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = mul2(w2, d[e]);
        store8<NT>(dyp + (int64_t)pos[g] * lddy, c, nt, tid, H, o);
      }
    }
  }
  if (!dwts) return;
  float dot[G];
#pragma unroll
  for (int g = 0; g < G; ++g) dot[g] = sum_of(part[g]);
  block_sums<G>(dot, buf);
#pragma unroll
  for (int g = 0; g < G; ++g)
    if (tid == g && j0 + g < k) dwts[first + g] = pos[g] >= 0 ? dot[g] : 0.f;
}

// ------------------------------------------------------------------------------------- router

constexpr int kRouterWarps = 8;

// One warp per token: lane j holds choice j. The row of E gradients is put together in shared memory
// (zeros, then the chosen ones; a repeated id adds up in choice order) and written whole, as 16-byte
// words with VEC. Several tokens per warp (8 lanes each for k = 8) were no faster at 16384 tokens of
// 256 experts (5.5 us against 5.1) and slower at 64 (2.3 against 1.7).
template <typename LT, bool VEC>
__global__ void __launch_bounds__(32 * kRouterWarps) route_backward_kernel(const int32_t* __restrict__ idx,
                                                                           const float* __restrict__ wts,
                                                                           const float* __restrict__ dwts, int T,
                                                                           int E, int k, LT* __restrict__ dlogits,
                                                                           int64_t ldl) {
  __shared__ __align__(16) float rows[kRouterWarps][kMaxExperts];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* row = rows[warp];
  for (int e = lane; e < E; e += 32) row[e] = 0.f;
  pdl_begin();
  const int64_t t = (int64_t)blockIdx.x * kRouterWarps + warp;
  if (t >= T) return;
  const int32_t* it = idx + t * k;
  const float *wt = wts + t * k, *dt = dwts + t * k;
  // the first 32 choices in one turn of loads
  const int e0 = lane < k ? it[lane] : -1;
  const float w0 = lane < k ? wt[lane] : 0.f, d0 = lane < k ? dt[lane] : 0.f;
  float mean = w0 * d0;
  for (int j = lane + 32; j < k; j += 32) mean = fmaf(wt[j], dt[j], mean);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
  __syncwarp();
  for (int jb = 0; jb < k; jb += 32) {
    const int j = jb + lane;
    int e = jb == 0 ? e0 : j < k ? it[j] : -1;
    if ((unsigned)e >= (unsigned)E) e = -1;
    const float g = e < 0 ? 0.f : jb == 0 ? w0 * (d0 - mean) : wt[j] * (dt[j] - mean);
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int turn = e >= 0 ? __popc(same & ((1u << lane) - 1u)) : 0;
    const int turns = __reduce_max_sync(0xffffffffu, turn);
    for (int i = 0; i <= turns; ++i) {
      if (e >= 0 && turn == i) row[e] += g;
      __syncwarp();
    }
  }
  LT* out = dlogits + t * ldl;
  if (VEC) {
    for (int e = lane * 8; e < E; e += 256) {
      float v[8];
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(row + e);
      *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(row + e + 4);
      Raw8<LT> r;
#pragma unroll
      for (int c = 0; c < 8; ++c) r.v[c] = RowType<LT>::from(v[c]);
      store_raw(out, e, E, r);
    }
  } else {
    for (int e = lane; e < E; e += 32) out[e] = RowType<LT>::from(row[e]);
  }
}

// ---- host side ----

// Calls f(typed null pointer, typed null pointer) for the (rows, out) types that are built: equal
// types, or fp32 rows with 16-bit results.
template <typename F>
int by_types(int y, int o, F f) {
  using B = __nv_bfloat16;
  using Hf = __half;
  if (y == MOE_DTYPE_BF16 && o == MOE_DTYPE_BF16) return f((B*)nullptr, (B*)nullptr);
  if (y == MOE_DTYPE_F16 && o == MOE_DTYPE_F16) return f((Hf*)nullptr, (Hf*)nullptr);
  if (y == MOE_DTYPE_F32 && o == MOE_DTYPE_F32) return f((float*)nullptr, (float*)nullptr);
  if (y == MOE_DTYPE_F32 && o == MOE_DTYPE_BF16) return f((float*)nullptr, (B*)nullptr);
  if (y == MOE_DTYPE_F32 && o == MOE_DTYPE_F16) return f((float*)nullptr, (Hf*)nullptr);
  return fail(MOE_ERR_ARG, "unsupported types: rows %d with results %d", y, o);
}

// Threads of a block for rows moved value by value, as by_width<32, 128, 256> chooses.
int value_threads(int H) { return H <= 256 ? 32 : H <= 1024 ? 128 : kRowThreads; }

int launch_combine_rows(const void* yp, int64_t ldy, int ydt, const int32_t* inv, const float* wts, int T, int H, int k,
                        void* out, int64_t ldo, int odt, cudaStream_t s) {
  if (T == 0) return MOE_OK;
  const bool vec = H % 8 == 0 && rows16(yp, ldy, dtype_size(ydt)) && rows16(out, ldo, dtype_size(odt));
  // Words: two chunks per thread of two choices at a time (four in 16 bits), in four blocks per SM; one
  // chunk of eight for more choices in 16 bits (T = 2048, k = 8, H = 2048 with sort and copy: 34.4 us
  // against 35.5 with two chunks of four and 37.3 of two), and in fp32 for so few tokens that a token's
  // own latency counts (T = 2048: 18 us against 16 with two chunks of two; T = 1: 1.7 against 4.2).
  // Single values: one chunk of four, of eight for few tokens. Narrow rows share a block.
  const bool wide = ydt == MOE_DTYPE_F32;
  const bool eight = vec && k > 4 && (!wide || T <= 256), two = vec && !eight && H > 256;
  const int nt = vec ? row_threads(parts_of(H, two ? 2 : 1), kRowThreads) : value_threads(H), ny = kRowThreads / nt;
  // a launch has at most 65535 blocks along the columns: wider rows take one launch per such slice
  const int cols = 8 * nt * (two ? 2 : 1), slice = 65535 * cols;
  return by_types(ydt, odt, [&](auto* y, auto* o) {
    using YT = std::remove_pointer_t<decltype(y)>;
    using OT = std::remove_pointer_t<decltype(o)>;
    auto values = [](auto n) { return combine_rows_kernel<YT, OT, decltype(n)::value, 4, 1>; };
    auto few = [](auto n) { return combine_rows_kernel<YT, OT, decltype(n)::value, 8, 1>; };
    auto kern = !vec    ? (k > 4 && T <= 256 ? by_width<32, 128, 256>(H, few) : by_width<32, 128, 256>(H, values))
                : eight ? combine_rows_kernel<YT, OT, 0, 8, 1>
                : !two  ? combine_rows_kernel<YT, OT, 0, 4, 1>
                : k <= 2 ? combine_rows_kernel<YT, OT, 0, 2, 2>
                         : combine_rows_kernel<YT, OT, 0, sizeof(YT) == 2 ? 4 : 2, 2>;
    int rc = MOE_OK;
    for (int64_t c0 = 0; c0 < H && rc == MOE_OK; c0 += slice) {
      const int h = H - c0 < slice ? (int)(H - c0) : slice;
      note_launch();
      rc = check_cuda(launch_pdl(kern, dim3(parts_of(T, ny), parts_of(h, cols)), dim3(nt, ny), 0, s,
                                 static_cast<const YT*>(yp) + c0, ldy, inv, wts, T, k, T * k, h,
                                 static_cast<OT*>(out) + c0, ldo),
                      "combine_rows_kernel");
    }
    return rc;
  });
}

int check_rows(const char* what, int T, int H, int k) {
  if (T < 0 || H < 1 || k < 1) return fail(MOE_ERR_ARG, "%s: bad sizes T=%d H=%d k=%d", what, T, H, k);
  if ((int64_t)T * k > INT32_MAX) return fail(MOE_ERR_SHAPE, "%s: T*k exceeds 2^31-1", what);
  if (H > 1 << 30) return fail(MOE_ERR_SHAPE, "%s: H=%d exceeds 2^30", what, H);   // column numbers are ints
  return MOE_OK;
}

// Strides count elements. Rows that are written lie apart; rows only read may repeat (stride 0).
int check_stride(const char* what, const char* name, int64_t stride, int64_t rows, int H, bool written) {
  if (stride < 0 || (written && rows > 1 && stride < H))
    return fail(MOE_ERR_ARG, "%s: row stride %lld of %s (H=%d)", what, (long long)stride, name, H);
  return MOE_OK;
}

int check_dtype(const char* what, int dtype) {
  return dtype_size(dtype) ? MOE_OK : fail(MOE_ERR_ARG, "%s: unknown type %d", what, dtype);
}

}  // namespace

int launch_dispatch(const void* x, int64_t ldx, size_t size, const int32_t* idx, int T, int H, int E, int k,
                    int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, void* xp, int64_t ldp,
                    cudaStream_t s) {
  if (H * size % 16 == 0 && rows16(x, ldx, size) && rows16(xp, ldp, size)) {
    const int per = 16 / (int)size;
    return dispatch_units<uint4>(x, ldx / per, idx, T, E, k, H / per, counts, offsets, perm, inv, xp, ldp / per, s);
  }
  if (size == 4) return dispatch_units<uint32_t>(x, ldx, idx, T, E, k, H, counts, offsets, perm, inv, xp, ldp, s);
  return dispatch_units<uint16_t>(x, ldx, idx, T, E, k, H, counts, offsets, perm, inv, xp, ldp, s);
}

}  // namespace moe

using namespace moe;

MOE_API int moe_dispatch(const void* x, int64_t x_stride, int dtype, const int32_t* idx, int T, int H, int E, int k,
                         int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, void* xp, int64_t xp_stride,
                         moe_stream_t stream) {
  const char* me = "moe_dispatch";
  if (int rc = check_rows(me, T, H, k)) return rc;
  if (int rc = check_dtype(me, dtype)) return rc;
  if (E < 1) return fail(MOE_ERR_ARG, "%s: E=%d", me, E);
  if (E > kMaxExperts) return fail(MOE_ERR_SHAPE, "%s: E=%d exceeds %d", me, E, kMaxExperts);
  if (!counts || !offsets || (T > 0 && (!x || !idx || !perm || !inv || !xp)))
    return fail(MOE_ERR_ARG, "%s: null pointer", me);
  if (T > 0 && x == xp) return fail(MOE_ERR_ARG, "%s: xp overlaps x", me);
  const void* ints[] = {counts, offsets, perm, inv, idx};      // an empty batch has only the first two
  for (int i = 0, n = T > 0 ? 5 : 2; i < n; ++i)
    for (int j = 0; j < i; ++j)
      if (ints[i] == ints[j]) return fail(MOE_ERR_ARG, "%s: idx and the index outputs overlap", me);
  if (int rc = check_stride(me, "x", x_stride, T, H, false)) return rc;
  if (int rc = check_stride(me, "xp", xp_stride, (int64_t)T * k, H, true)) return rc;
  return launch_dispatch(x, x_stride, dtype_size(dtype), idx, T, H, E, k, counts, offsets, perm, inv, xp, xp_stride,
                         reinterpret_cast<cudaStream_t>(stream));
}

MOE_API int moe_dispatch_backward(const void* dxp, int64_t dxp_stride, int dtype, const int32_t* inv, int T, int H,
                                  int k, void* dx, int64_t dx_stride, moe_stream_t stream) {
  const char* me = "moe_dispatch_backward";
  if (int rc = check_rows(me, T, H, k)) return rc;
  if (int rc = check_dtype(me, dtype)) return rc;
  if (T > 0 && (!dxp || !inv || !dx)) return fail(MOE_ERR_ARG, "%s: null pointer", me);
  if (T > 0 && dx == dxp) return fail(MOE_ERR_ARG, "%s: dx overlaps dxp", me);
  if (int rc = check_stride(me, "dxp", dxp_stride, (int64_t)T * k, H, false)) return rc;
  if (int rc = check_stride(me, "dx", dx_stride, T, H, true)) return rc;
  return launch_combine_rows(dxp, dxp_stride, dtype, inv, nullptr, T, H, k, dx, dx_stride, dtype,
                             reinterpret_cast<cudaStream_t>(stream));
}

MOE_API int moe_combine(const void* yp, int64_t yp_stride, int yp_dtype, const int32_t* inv, const float* wts, int T,
                        int H, int k, void* out, int64_t out_stride, int out_dtype, moe_stream_t stream) {
  const char* me = "moe_combine";
  if (int rc = check_rows(me, T, H, k)) return rc;
  if (int rc = check_dtype(me, yp_dtype)) return rc;
  if (int rc = check_dtype(me, out_dtype)) return rc;
  if (yp_dtype != out_dtype && yp_dtype != MOE_DTYPE_F32)
    return fail(MOE_ERR_ARG, "%s: rows of type %d with results of type %d", me, yp_dtype, out_dtype);
  if (T > 0 && (!yp || !inv || !wts || !out)) return fail(MOE_ERR_ARG, "%s: null pointer", me);
  if (T > 0 && out == yp) return fail(MOE_ERR_ARG, "%s: out overlaps yp", me);
  if (int rc = check_stride(me, "yp", yp_stride, (int64_t)T * k, H, false)) return rc;
  if (int rc = check_stride(me, "out", out_stride, T, H, true)) return rc;
  return launch_combine_rows(yp, yp_stride, yp_dtype, inv, wts, T, H, k, out, out_stride, out_dtype,
                             reinterpret_cast<cudaStream_t>(stream));
}

MOE_API int moe_combine_backward(const void* dout, int64_t dout_stride, int dout_dtype, const void* yp,
                                 int64_t yp_stride, int yp_dtype, const int32_t* inv, const float* wts, int T, int H,
                                 int k, void* dyp, int64_t dyp_stride, float* dwts, moe_stream_t stream) {
  const char* me = "moe_combine_backward";
  if (int rc = check_rows(me, T, H, k)) return rc;
  if (int rc = check_dtype(me, yp_dtype)) return rc;
  if (int rc = check_dtype(me, dout_dtype)) return rc;
  if (yp_dtype != dout_dtype && yp_dtype != MOE_DTYPE_F32)
    return fail(MOE_ERR_ARG, "%s: rows of type %d with results of type %d", me, yp_dtype, dout_dtype);
  if (T > 0 && !dyp && !dwts) return fail(MOE_ERR_ARG, "%s: dyp and dwts are both null", me);
  if (T > 0 && (!dout || !inv || !wts || (dwts && !yp))) return fail(MOE_ERR_ARG, "%s: null pointer", me);
  if (dyp && (dyp == yp || dyp == dout)) return fail(MOE_ERR_ARG, "%s: dyp overlaps an input", me);
  if (int rc = check_stride(me, "dout", dout_stride, T, H, false)) return rc;
  if (int rc = check_stride(me, "yp", yp_stride, (int64_t)T * k, H, false)) return rc;
  if (int rc = check_stride(me, "dyp", dyp_stride, dyp ? (int64_t)T * k : 0, H, true)) return rc;
  if (T == 0) return MOE_OK;
  const size_t ys = dtype_size(yp_dtype);
  const bool vec = H % 8 == 0 && rows16(dout, dout_stride, dtype_size(dout_dtype)) &&
                   (!dwts || rows16(yp, yp_stride, ys)) && rows16(dyp, dyp_stride, ys);
  note_launch();
  return by_types(yp_dtype, dout_dtype, [&](auto* y, auto* o) {
    using YT = std::remove_pointer_t<decltype(y)>;
    using OT = std::remove_pointer_t<decltype(o)>;
    // choices in a group (0: a block per token); measured at combine_group_backward_kernel
    const int G = T * k <= kFewPairs || k == 1 || (vec && k == 2 && H > 1024) ? 1
                  : !vec                                                   ? (k == 2 ? 2 : 4)
                  : k == 2 || (sizeof(YT) == 4 && H >= 512)                ? 2 : 0;
    auto form = [&](auto g) {
      constexpr int N = decltype(g)::value;
      auto by_nt = [](auto n) { return combine_group_backward_kernel<YT, OT, decltype(n)::value, N>; };
      if constexpr (N < 4)      // groups of four are for single values alone
        if (vec) return by_nt(std::integral_constant<int, 0>());
      return by_width<32, 128, 256>(H, by_nt);
    };
    auto kern = G == 0   ? combine_backward_kernel<YT, OT>
                : G == 1 ? form(std::integral_constant<int, 1>())
                : G == 2 ? form(std::integral_constant<int, 2>())
                         : form(std::integral_constant<int, 4>());
    const dim3 grid(G ? T * parts_of(k, G) : T), block(vec ? row_threads(H, kRowThreads) : value_threads(H));
    return check_cuda(launch_pdl(kern, grid, block, 0, reinterpret_cast<cudaStream_t>(stream),
                                 static_cast<const OT*>(dout), dout_stride, static_cast<const YT*>(yp), yp_stride, inv,
                                 wts, k, T * k, H, static_cast<YT*>(dyp), dyp_stride, dwts),
                      "combine_backward_kernel");
  });
}

MOE_API int moe_route_topk_backward(const int32_t* idx, const float* wts, const float* dwts, int T, int E, int k,
                                    void* dlogits, int64_t dlogits_stride, int dtype, moe_stream_t stream) {
  const char* me = "moe_route_topk_backward";
  if (T < 0 || k < 1 || k > E) return fail(MOE_ERR_ARG, "%s: bad sizes T=%d E=%d k=%d", me, T, E, k);
  if (E > kMaxExperts) return fail(MOE_ERR_SHAPE, "%s: E=%d exceeds %d", me, E, kMaxExperts);
  if ((int64_t)T * k > INT32_MAX) return fail(MOE_ERR_SHAPE, "%s: T*k exceeds 2^31-1", me);
  if (int rc = check_dtype(me, dtype)) return rc;
  if (T > 0 && (!idx || !wts || !dwts || !dlogits)) return fail(MOE_ERR_ARG, "%s: null pointer", me);
  if (int rc = check_stride(me, "dlogits", dlogits_stride, T, E, true)) return rc;
  if (T == 0) return MOE_OK;
  note_launch();
  return by_types(dtype, dtype, [&](auto* l, auto*) {
    using LT = std::remove_pointer_t<decltype(l)>;
    const bool vec = E % 8 == 0 && rows16(dlogits, dlogits_stride, sizeof(LT));
    auto kern = vec ? route_backward_kernel<LT, true> : route_backward_kernel<LT, false>;
    return check_cuda(launch_pdl(kern, dim3(parts_of(T, kRouterWarps)), dim3(32 * kRouterWarps), 0,
                                 reinterpret_cast<cudaStream_t>(stream), idx, wts, dwts, T, E, k,
                                 static_cast<LT*>(dlogits), dlogits_stride),
                      "route_backward_kernel");
  });
}
