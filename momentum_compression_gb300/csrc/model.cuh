// Argument blocks and launchers of the model-side operators (dropout,
// relative position bias, attention).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "keep.cuh"
#include "ob.h"

namespace ob {

struct DropoutArgs {
  const void* x;
  const void* residual;  // or null
  void* y;
  uint64_t ldx, ldr, ldy, rows, cols;  // one row where every array is contiguous
  uint64_t n;                          // rows * cols
  uint64_t magic;                      // ceil(2^64 / cols)
  int small;                           // n < 2^32: rows by `magic`
  Keep keep;
};

struct RelposArgs {
  ob_relpos rp;
  const void* table;
  int table_type;
  int H;
  int64_t Lq, Lk, q_offset;
  void* out;
  int64_t stride_h, stride_l;
};

struct RelposBwdArgs {
  ob_relpos rp;
  const void* dout;
  int64_t N, Lq, Lk, q_offset;
  int64_t stride_n, stride_h, stride_l;
  int H;
  int n_per;        // entries of N a block adds
  int64_t strips;   // of columns
  int64_t blocks_t; // blocks a head: tiles x entries
  int blocks_n;
  float* partial;   // [H][blocks][num_buckets]
  void* dtable;
  int table_type;
};

cudaError_t launch_dropout(const DropoutArgs& a, int type, cudaStream_t s);
cudaError_t launch_relpos_bias(const RelposArgs& a, int out_type, cudaStream_t s);
// The most blocks a head that the gradient of these sizes may take.
int64_t relpos_bwd_blocks(const RelposBwdArgs& a);
cudaError_t launch_relpos_bias_bwd(const RelposBwdArgs& a, int out_type, cudaStream_t s);

// Sums partial[h][0..parts)[b] in a fixed order into dtable[b][h].
cudaError_t launch_bucket_sums(const float* partial, int parts, int H, int num_buckets,
                               void* dtable, int type, cudaStream_t s);

#ifdef __CUDACC__
// Launches a kernel that may start while the one before it on the stream still
// runs (its launch and prologue overlap that one's end): it calls grid_wait()
// before it touches anything the others write or read, and the one before
// calls grid_release() when the next may start.
template <typename... P, typename... A>
inline cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                                 cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Buckets.  `first` is ob_relpos.first of a side, staged in shared memory.
// ---------------------------------------------------------------------------

// The largest b with first[b] <= n (first[0] = 0).
__device__ __forceinline__ int side_bucket(const int* first, int side, int n) {
  int lo = 0, hi = side;  // first[lo] <= n, and first[hi] > n or hi = side
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= n)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int bucket_of(const int* first, int side, int two_sided, int64_t d) {
  const int64_t n64 = d > 0 ? (two_sided ? d : 0) : -d;
  const int n = n64 < (1 << 24) ? (int)n64 : (1 << 24);  // past every max_distance
  return side_bucket(first, side, n) + (two_sided && d > 0 ? side : 0);
}

// Distances of bucket b that lie in [dmin, dmax]: [lo, hi), empty if lo >= hi.
__device__ __forceinline__ void bucket_range(const int* first, int side, int two_sided, int b,
                                             int64_t dmin, int64_t dmax, int64_t* lo,
                                             int64_t* hi) {
  const bool right = b >= side;
  const int s = right ? b - side : b;
  const int64_t n0 = first[s];
  const int64_t n1 = s + 1 < side ? first[s + 1] : INT64_MAX / 2;  // n in [n0, n1)
  if (right) {
    *lo = n0 > 1 ? n0 : 1;
    *hi = n1;
  } else {
    *lo = 1 - n1;
    *hi = n0 == 0 && n1 > 0 && !two_sided ? INT64_MAX / 2 : 1 - n0;
  }
  if (*lo < dmin) *lo = dmin;
  if (*hi > dmax + 1) *hi = dmax + 1;
}
#endif

}  // namespace ob
