// Attention with dropout and the bucketed bias, forward and backward: one
// warp per row, dot products in fp32.
#include <cmath>

#include "attn.cuh"
#include "elem.cuh"

namespace ob {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxD = 128;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <typename T>
__device__ __forceinline__ const T* row(const Heads& t, int b, int i, int h) {
  return static_cast<const T*>(t.data) + b * t.b + i * t.l + h * t.h;
}
template <typename T>
__device__ __forceinline__ T* row_out(const Heads& t, int b, int i, int h) {
  return static_cast<T*>(t.data) + b * t.b + i * t.l + h * t.h;
}

template <typename T>
__device__ __forceinline__ float dot(const float* x, const T* y, int D) {
  float s = 0.0f;
  for (int d = 0; d < D; ++d) s = __fmaf_rn(x[d], to_f32(y[d]), s);
  return s;
}

// Whether the pair's weight is kept.
__device__ __forceinline__ bool pair_kept(const AttnArgs& a, int bh, int i, int j) {
  if (!a.keep.T) return true;
  const uint64_t per_row = (uint64_t)((a.Lk + 7) / 8);
  const uint4 w = keep_words(a.keep, ((uint64_t)bh * a.Lq + i) * per_row + (j >> 3));
  return keep_byte(w, a.keep.T) >> (j & 7) & 1;
}

// dq and the bucket sums of its row, part i of partial[h].
template <typename T>
__global__ void k_dq(const __grid_constant__ AttnArgs a) {
  __shared__ int first[OB_RELPOS_MAX_SIDE];
  __shared__ float qs[kWarps][kMaxD], gs[kWarps][kMaxD];
  __shared__ float by_b[kWarps][2 * OB_RELPOS_MAX_SIDE];
  for (int b = threadIdx.x; b < a.rp.side; b += blockDim.x) first[b] = a.rp.first[b];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int b = lane; b < 2 * OB_RELPOS_MAX_SIDE; b += 32) by_b[warp][b] = 0.0f;
  __syncthreads();
  const int i = blockIdx.x * kWarps + warp, bh = blockIdx.y, b = bh / a.H, h = bh % a.H;
  if (i >= a.Lq) return;
  const int hk = h / (a.H / a.Hkv), n = key_count(a.kv_len, a.Lk, b);
  float delta = 0.0f, acc[4] = {0, 0, 0, 0};
  for (int d = lane; d < a.D; d += 32) {
    qs[warp][d] = to_f32(row<T>(a.q, b, i, h)[d]);
    gs[warp][d] = to_f32(row<T>(a.grad_o, b, i, h)[d]);
    delta = __fmaf_rn(gs[warp][d], to_f32(row<T>(a.o, b, i, h)[d]), delta);
  }
  delta = warp_sum(delta);
  const float lse = a.lse[(size_t)bh * a.Lq + i];
  __syncwarp();
  for (int j0 = 0; j0 < n && lse != -INFINITY; j0 += 32) {
    const int j = j0 + lane;
    float ds = 0.0f;
    int bucket = 0;
    if (j < n && (!a.causal || j <= i + a.q_offset)) {
      float s = dot(qs[warp], row<T>(a.k, b, j, hk), a.D) * a.scale;
      if (a.biased) {
        bucket = bucket_of(first, a.rp.side, a.rp.two_sided, j - i - a.q_offset);
        s += load_as_f32(a.table, (size_t)bucket * a.H + h, a.type);
      }
      const float g = pair_kept(a, bh, i, j)
                          ? a.keep.scale * dot(gs[warp], row<T>(a.v, b, j, hk), a.D) : 0.0f;
      ds = expf(s - lse) * (g - delta);
    }
    for (int k = 0; k < 32 && j0 + k < n; ++k) {
      const float x = __shfl_sync(0xffffffffu, ds, k);
      const int bk = __shfl_sync(0xffffffffu, bucket, k);
      if (x == 0.0f) continue;
      if (lane == 0) by_b[warp][bk] += x;
      const T* kr = row<T>(a.k, b, j0 + k, hk);
      for (int t = 0; t < 4; ++t)
        if (lane + 32 * t < a.D) acc[t] = __fmaf_rn(x, to_f32(kr[lane + 32 * t]), acc[t]);
    }
  }
  for (int t = 0; t < 4; ++t)
    if (lane + 32 * t < a.D)
      row_out<T>(a.dq, b, i, h)[lane + 32 * t] = from_f32<T>(acc[t] * a.scale);
  __syncwarp();
  if (a.dtable)
    for (int k = lane; k < a.rp.num_buckets; k += 32)
      static_cast<float*>(a.workspace)[(((size_t)h * a.B + b) * a.Lq + i) * a.rp.num_buckets + k] =
          by_b[warp][k];
}

// dk and dv of one key: over the heads that share it and their queries.
template <typename T>
__global__ void k_dkv(const __grid_constant__ AttnArgs a) {
  __shared__ int first[OB_RELPOS_MAX_SIDE];
  __shared__ float ks[kWarps][kMaxD], vs[kWarps][kMaxD];
  for (int b = threadIdx.x; b < a.rp.side; b += blockDim.x) first[b] = a.rp.first[b];
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = blockIdx.x * kWarps + warp, b = blockIdx.y / a.Hkv, hk = blockIdx.y % a.Hkv;
  if (j >= a.Lk) return;
  const int group = a.H / a.Hkv, n = key_count(a.kv_len, a.Lk, b);
  float dk[4] = {0, 0, 0, 0}, dv[4] = {0, 0, 0, 0};
  if (j < n) {
    for (int d = lane; d < a.D; d += 32) {
      ks[warp][d] = to_f32(row<T>(a.k, b, j, hk)[d]);
      vs[warp][d] = to_f32(row<T>(a.v, b, j, hk)[d]);
    }
    __syncwarp();
    for (int h = hk * group; h < (hk + 1) * group; ++h) {
      const int bh = b * a.H + h;
      for (int i0 = 0; i0 < a.Lq; i0 += 32) {
        const int i = i0 + lane;
        float ds = 0.0f, z = 0.0f;
        if (i < a.Lq && (!a.causal || j <= i + a.q_offset) &&
            a.lse[(size_t)bh * a.Lq + i] != -INFINITY) {
          const T* g = row<T>(a.grad_o, b, i, h);
          float s = dot(ks[warp], row<T>(a.q, b, i, h), a.D) * a.scale;
          if (a.biased)
            s += load_as_f32(
                a.table,
                (size_t)bucket_of(first, a.rp.side, a.rp.two_sided, j - i - a.q_offset) * a.H + h,
                a.type);
          const float p = expf(s - a.lse[(size_t)bh * a.Lq + i]);
          const bool kept = pair_kept(a, bh, i, j);
          float delta = 0.0f;
          const T* o = row<T>(a.o, b, i, h);
          for (int d = 0; d < a.D; ++d) delta = __fmaf_rn(to_f32(g[d]), to_f32(o[d]), delta);
          z = kept ? p * a.keep.scale : 0.0f;
          ds = p * ((kept ? a.keep.scale * dot(vs[warp], g, a.D) : 0.0f) - delta);
        }
        for (int k = 0; k < 32 && i0 + k < a.Lq; ++k) {
          const float x = __shfl_sync(0xffffffffu, ds, k), y = __shfl_sync(0xffffffffu, z, k);
          const T* q = row<T>(a.q, b, i0 + k, h);
          const T* g = row<T>(a.grad_o, b, i0 + k, h);
          for (int t = 0; t < 4; ++t)
            if (lane + 32 * t < a.D) {
              dk[t] = __fmaf_rn(x, to_f32(q[lane + 32 * t]), dk[t]);
              dv[t] = __fmaf_rn(y, to_f32(g[lane + 32 * t]), dv[t]);
            }
        }
      }
    }
  }
  for (int t = 0; t < 4; ++t)
    if (lane + 32 * t < a.D) {
      row_out<T>(a.dk, b, j, hk)[lane + 32 * t] = from_f32<T>(dk[t] * a.scale);
      row_out<T>(a.dv, b, j, hk)[lane + 32 * t] = from_f32<T>(dv[t]);
    }
}

template <typename T>
cudaError_t bwd(const AttnArgs& a, cudaStream_t s) {
  if (a.B && a.Lq)
    k_dq<T><<<dim3((a.Lq + kWarps - 1) / kWarps, a.B * a.H), 32 * kWarps, 0, s>>>(a);
  if (a.B && a.Lk)
    k_dkv<T><<<dim3((a.Lk + kWarps - 1) / kWarps, a.B * a.Hkv), 32 * kWarps, 0, s>>>(a);
  if (a.dtable) {
    cudaError_t e = launch_bucket_sums(static_cast<const float*>(a.workspace), a.B * a.Lq, a.H,
                                       a.rp.num_buckets, a.dtable, a.type, s);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace

size_t attn_workspace_bytes(const AttnArgs& a) {
  return a.biased ? (size_t)a.B * a.H * a.Lq * a.rp.num_buckets * sizeof(float) : 0;
}

cudaError_t launch_attn_bwd(const AttnArgs& a, cudaStream_t s) {
  return a.type == OB_TYPE_BF16 ? bwd<__nv_bfloat16>(a, s) : bwd<__half>(a, s);
}

}  // namespace ob
