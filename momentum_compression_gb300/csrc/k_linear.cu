// The dense layer: y = act(x w^T + b) + residual and its gradients.
#include "elem.cuh"
#include "layers.cuh"

namespace ob {
namespace {

constexpr float kSqrtHalf = 0.70710678f, kInvSqrt2Pi = 0.39894228f;
constexpr float kTanhA = 0.79788456f, kTanhB = 0.044715f;

__device__ __forceinline__ float act_of(float z, int act) {
  if (act == OB_ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays one
  if (act == OB_ACT_GELU) return 0.5f * z * (1.0f + erff(z * kSqrtHalf));
  if (act == OB_ACT_GELU_TANH)
    return 0.5f * z * (1.0f + tanhf(kTanhA * __fmaf_rn(kTanhB * z * z, z, z)));
  return z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
  if (act == OB_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if (act == OB_ACT_GELU)
    return __fmaf_rn(z * kInvSqrt2Pi, expf(-0.5f * z * z), 0.5f * (1.0f + erff(z * kSqrtHalf)));
  if (act == OB_ACT_GELU_TANH) {
    const float t = tanhf(kTanhA * __fmaf_rn(kTanhB * z * z, z, z));
    return __fmaf_rn(0.5f * z * (1.0f - t * t), kTanhA * __fmaf_rn(3.0f * kTanhB, z * z, 1.0f),
                     0.5f * (1.0f + t));
  }
  return 1.0f;
}

struct Epilogue {
  const void *bias, *residual;
  int64_t ldr;
  void* z;
  int64_t ldz;
  int act;
};

// c[i][j] = sum over k of a(i, k) b(k, j); a(i, k) at a + i * am + k * ak.
template <typename T>
__global__ void __launch_bounds__(256)
    k_product(const T* a, int64_t am, int64_t ak, const T* b, int64_t bk, int64_t bn, T* c,
              int64_t ldc, int64_t M, int64_t N, int64_t K, Epilogue ep) {
  __shared__ float as[16][65], bs[16][65];
  const int64_t i0 = (int64_t)blockIdx.y * 64, j0 = (int64_t)blockIdx.x * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += 16) {
    for (int t = threadIdx.x; t < 64 * 16; t += 256) {
      const int64_t i = i0 + t / 16, k = k0 + t % 16, j = j0 + t % 64, kb = k0 + t / 64;
      as[t % 16][t / 16] = i < M && k < K ? to_f32(a[i * am + k * ak]) : 0.0f;
      bs[t / 64][t % 64] = j < N && kb < K ? to_f32(b[kb * bk + j * bn]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int w = 0; w < 4; ++w)
          acc[u][w] = __fmaf_rn(as[k][ty * 4 + u], bs[k][tx + 16 * w], acc[u][w]);
    __syncthreads();
  }
  for (int u = 0; u < 4; ++u)
    for (int w = 0; w < 4; ++w) {
      const int64_t i = i0 + ty * 4 + u, j = j0 + tx + 16 * w;
      if (i >= M || j >= N) continue;
      float z = acc[u][w];
      if (ep.bias) z += to_f32(static_cast<const T*>(ep.bias)[j]);
      if (ep.z) static_cast<T*>(ep.z)[i * ep.ldz + j] = from_f32<T>(z);
      float y = act_of(z, ep.act);
      if (ep.residual) y += to_f32(static_cast<const T*>(ep.residual)[i * ep.ldr + j]);
      c[i * ldc + j] = from_f32<T>(y);
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
    k_dz(const T* dy, int64_t lddy, const T* z, int64_t ldz, T* dz, int64_t M, int64_t N, int act) {
  const int64_t i = blockIdx.y, j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= N) return;
  for (int64_t r = i; r < M; r += gridDim.y)
    dz[r * N + j] = from_f32<T>(to_f32(dy[r * lddy + j]) * act_slope(to_f32(z[r * ldz + j]), act));
}

template <typename T>
__global__ void __launch_bounds__(1024)
    k_dbias(const T* dy, int64_t lddy, const T* z, int64_t ldz, T* db, int64_t M, int64_t N,
            int act) {
  __shared__ float sum[32][33];
  const int64_t j = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float t = 0.0f;
  if (j < N)
    for (int64_t r = threadIdx.y; r < M; r += 32) {
      const float g = to_f32(dy[r * lddy + j]);
      t += z ? g * act_slope(to_f32(z[r * ldz + j]), act) : g;
    }
  sum[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0 && j < N) {
    t = 0.0f;
    for (int r = 0; r < 32; ++r) t += sum[r][threadIdx.x];
    db[j] = from_f32<T>(t);
  }
}

template <typename T>
void product(const T* a, int64_t am, int64_t ak, const T* b, int64_t bk, int64_t bn, T* c,
             int64_t ldc, int64_t M, int64_t N, int64_t K, const Epilogue& ep, cudaStream_t s) {
  const dim3 grid((unsigned)((N + 63) / 64), (unsigned)((M + 63) / 64));
  k_product<T><<<grid, 256, 0, s>>>(a, am, ak, b, bk, bn, c, ldc, M, N, K, ep);
}

}  // namespace

size_t linear_workspace_bytes(const LinearArgs& a, bool backward) {
  return backward && a.act != OB_ACT_NONE ? (size_t)(a.M * a.N) * 2 : 0;
}

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t s) {
  auto go = [&](auto zero) {
    using T = decltype(zero);
    const Epilogue ep{a.bias, a.residual.data, a.residual.ld, a.z.data, a.z.ld, a.act};
    product<T>(static_cast<const T*>(a.x.data), a.x.ld, 1, static_cast<const T*>(a.w.data),
               a.w_kn ? a.w.ld : 1, a.w_kn ? 1 : a.w.ld, static_cast<T*>(a.y.data), a.y.ld, a.M,
               a.N, a.K, ep, s);
    return cudaGetLastError();
  };
  return a.type == OB_TYPE_BF16 ? go(__nv_bfloat16()) : go(__half());
}

cudaError_t launch_linear_bwd(const LinearArgs& a, cudaStream_t s) {
  auto go = [&](auto zero) {
    using T = decltype(zero);
    const T* dz = static_cast<const T*>(a.dy.data);
    int64_t lddz = a.dy.ld;
    const T* z = a.act != OB_ACT_NONE ? static_cast<const T*>(a.z.data) : nullptr;
    const T* dy = dz;
    if (z && (a.dx.data || a.dw.data) && a.M > 0) {
      T* to = reinterpret_cast<T*>(a.workspace);
      const dim3 grid((unsigned)((a.N + 255) / 256), (unsigned)(a.M < 65535 ? a.M : 65535));
      k_dz<T><<<grid, 256, 0, s>>>(dy, a.dy.ld, z, a.z.ld, to, a.M, a.N, a.act);
      dz = to;
      lddz = a.N;
    }
    const Epilogue none{nullptr, nullptr, 0, nullptr, 0, OB_ACT_NONE};
    const T *x = static_cast<const T*>(a.x.data), *w = static_cast<const T*>(a.w.data);
    if (a.dx.data && a.M > 0)
      product<T>(dz, lddz, 1, w, a.w_kn ? 1 : a.w.ld, a.w_kn ? a.w.ld : 1,
                 static_cast<T*>(a.dx.data), a.dx.ld, a.M, a.K, a.N, none, s);
    if (a.dw.data && a.w_kn)
      product<T>(x, 1, a.x.ld, dz, lddz, 1, static_cast<T*>(a.dw.data), a.dw.ld, a.K, a.N, a.M,
                 none, s);
    else if (a.dw.data)
      product<T>(dz, 1, lddz, x, a.x.ld, 1, static_cast<T*>(a.dw.data), a.dw.ld, a.N, a.K, a.M,
                 none, s);
    if (a.dbias)
      k_dbias<T><<<(unsigned)((a.N + 31) / 32), dim3(32, 32), 0, s>>>(
          dy, a.dy.ld, z, a.z.ld, static_cast<T*>(a.dbias), a.M, a.N, a.act);
    return cudaGetLastError();
  };
  return a.type == OB_TYPE_BF16 ? go(__nv_bfloat16()) : go(__half());
}

}  // namespace ob
