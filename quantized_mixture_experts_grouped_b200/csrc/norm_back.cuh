// The gradient of the norms around a block (see norm.cu for the formulas): its arguments, and the launch of
// the ring form, for rows of up to 4096 values.
#pragma once

#include "rows.cuh"

namespace moe {

constexpr int kSums = 3;                  // column sums of the backward pass: dw, dgate, dw_next
constexpr int kRingStages = 4;            // five were slower (96 us against 100 at T = 8192, H = 4096)
constexpr int kRingBytes = 224 * 1024 - 4096;        // of an SM's 228 KB, for all its blocks
constexpr int kRingThreads = 512;         // most threads of a block of the ring kernel

struct BackArgs {
  const void *dho, *y, *ho, *dx, *w, *gate, *w_next;   // dho may be null (no residual gradient)
  void *dh, *dy, *dgate;
  float *dw, *dw_next, *part;      // part: fp32 [blocks][kSums][part_ld], used with more than one block
  int64_t lddho, ldy, ldho, lddx, ldg, lddh, lddy, lddg;
  int T, H, part_ld, gate_mode;
  bool has_y, norm_y, next;        // has_y false: the gradient of the norm before a block
  float alpha, eps;
};

// Blocks of the ring kernel that share an SM by their registers (64 a thread before a block, 128 after
// one), 16 at most.
constexpr int ring_blocks(int threads, bool has_y) {
  return (has_y ? 512 : 1024) / threads < 16 ? (has_y ? 512 : 1024) / threads : 16;
}

// Bytes of a stage for one tensor's row moved value by value: the 16-byte granules that cover it wherever
// it starts.
__host__ __device__ constexpr int value_region(int H, int size) { return (H * size + 31) / 16 * 16; }

// Launches the ring kernel for rows of type T (one file per type, so that they compile side by side);
// words: rows of 16-byte words, else value by value with nt 128, 256 or kRingThreads.
template <typename T>
int launch_norm_ring(const BackArgs& a, int blocks, int nt, bool words, int stages, int stage_bytes, cudaStream_t s);

}  // namespace moe
