// What the kernels over many tensors share (adamw.cu, grad_norm.cu): tables of
// tensors in kernel parameters and the walk over their chunks.
//
// A launch takes a table of up to CAP tensors by value, so that a captured
// graph holds all of it and nothing on the device has to be kept for it. The
// tensors are cut into chunks of kOptimChunk elements, numbered through; a CTA
// takes chunk after chunk, 16 consecutive elements a thread.
#pragma once

#include "fp8_block.cuh"

namespace taco {

constexpr int kOptimThreads = 256;
constexpr int64_t kOptimChunk = kOptimThreads * 16;

// Tensor of chunk c: the last one whose first chunk is at most c. `t` is the
// tensor of an earlier chunk of the same CTA, and mostly c's too.
template <typename Table>
__device__ __forceinline__ int tensor_of(const Table& table, uint32_t c, int t) {
  int hi = table.count;
  if (t + 1 == hi || c < table.t[t + 1].first) return t;
  int lo = t + 1;   // first[lo] <= c
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (table.t[mid].first <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

}  // namespace taco
