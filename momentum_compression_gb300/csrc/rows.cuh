// Rows as layer norm's kernels take them: eight columns to a thread at a time, packed as
// in memory, unpacked to fp32 two columns a register; sums over a block.
#pragma once

#include <type_traits>

#include "elem.cuh"
#include "layers.cuh"
#include "model.cuh"
#include "ob_internal.cuh"
#include "tc.cuh"

namespace ob {
namespace {

constexpr int kSms = 152;
constexpr int kWide = 512;  // threads of a block that walks over its row

// Sum over the block's threads, in every thread.  `buf`: 33 floats.
__device__ __forceinline__ float block_sum(float v, float* buf) {
  v = warp_butterfly_sum(v);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  __syncthreads();
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  return warp_butterfly_sum(lane < warps ? buf[lane] : 0.0f);
}

// ---------------------------------------------------------------------------
// Rows in registers.  A thread has CH chunks of eight columns: consecutive ones
// where everything lies on 16 bytes (LIES 1; 2: and the chunks are the row exactly),
// else (0) every `threads`-th, so that narrow accesses of a warp still lie side by side.
// The arithmetic takes two columns an instruction.
// ---------------------------------------------------------------------------

template <int LIES>
__device__ __forceinline__ int column(int c, int j, int t, int threads) {
  return LIES ? (c * threads + t) * 8 + j : (c * 8 + j) * threads + t;
}

__device__ __forceinline__ uint64_t twice(float x) { return pair(x, x); }

template <typename T>
__device__ __forceinline__ uint64_t unpack_pair(uint32_t w);
template <>
__device__ __forceinline__ uint64_t unpack_pair<__nv_bfloat16>(uint32_t w) {
  return pair(w << 16, w & 0xffff0000u);
}
template <>
__device__ __forceinline__ uint64_t unpack_pair<__half>(uint32_t w) {
  const float2 f = unpack2<__half>(w);
  return pair(f.x, f.y);
}

// Chunk c as it lies in memory; what is past the row is 0.
template <typename T, int LIES>
struct Chunk {
  static constexpr int kWords = sizeof(T) / 2;
  uint4 raw[kWords];
  __device__ __forceinline__ void load(const T* row, int c, int t, int threads, int cols) {
    if constexpr (LIES > 0) {
      const int at = column<1>(c, 0, t, threads);
      if (LIES == 1)
#pragma unroll
        for (int i = 0; i < kWords; ++i) raw[i] = make_uint4(0, 0, 0, 0);
      if (LIES == 2 || at < cols) {
        const uint4* p = reinterpret_cast<const uint4*>(row + at);
#pragma unroll
        for (int i = 0; i < kWords; ++i) raw[i] = p[i];
      }
    } else {
      T v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = column<0>(c, j, t, threads);
        v[j] = from_f32<T>(0.0f);
        if (at < cols) v[j] = row[at];
      }
      memcpy(raw, v, sizeof raw);
    }
  }
  // Pairs of columns in fp32.
  __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
    if constexpr (sizeof(T) == 4) {
      v[0] = pair(raw[0].x, raw[0].y);
      v[1] = pair(raw[0].z, raw[0].w);
      v[2] = pair(raw[1].x, raw[1].y);
      v[3] = pair(raw[1].z, raw[1].w);
    } else {
      v[0] = unpack_pair<T>(raw[0].x);
      v[1] = unpack_pair<T>(raw[0].y);
      v[2] = unpack_pair<T>(raw[0].z);
      v[3] = unpack_pair<T>(raw[0].w);
    }
  }
  __device__ __forceinline__ void put(const uint64_t (&v)[4]) {
    float f[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) unpair(v[k], &f[2 * k], &f[2 * k + 1]);
    if constexpr (sizeof(T) == 4)
      memcpy(raw, f, 32);
    else
      raw[0] = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                          pack2<T>(f[6], f[7]));
  }
  __device__ __forceinline__ void store(T* row, int c, int t, int threads, int cols) const {
    if constexpr (LIES > 0) {
      const int at = column<1>(c, 0, t, threads);
      if (LIES == 2 || at < cols) {
        uint4* p = reinterpret_cast<uint4*>(row + at);
#pragma unroll
        for (int i = 0; i < kWords; ++i) p[i] = raw[i];
      }
    } else {
      T v[8];
      memcpy(v, raw, sizeof raw);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = column<0>(c, j, t, threads);
        if (at < cols) row[at] = v[j];
      }
    }
  }
};

// f(zero of the type) for a run-time type.
template <typename F>
__device__ __forceinline__ void with_type(int type, F f) {
  if (type == OB_TYPE_F32)
    f(0.0f);
  else if (type == OB_TYPE_BF16)
    f(__nv_bfloat16());
  else
    f(__half());
}

template <typename F>
cudaError_t by_type(int type, F f) {
  if (type == OB_TYPE_F32) return f(0.0f);
  if (type == OB_TYPE_BF16) return f(__nv_bfloat16());
  return f(__half());
}

int row_blocks(uint64_t rows) { return (int)(rows < 65535 ? rows : 65535); }

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace
}  // namespace ob
