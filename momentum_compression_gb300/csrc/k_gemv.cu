// The dense layer's product for up to eight rows (single tokens): B is read once
// and bounds it; the products are fp32 multiply-adds.
//   B stored [N][K]   a warp a column of the output: its lanes share the sum, 16 bytes
//                     of B's row a lane and step, eight steps on their way at once
//   B stored [K][N]   a lane eight columns; the sum is cut among a block's warps and
//                     among blocks, whose parts a second kernel adds in their order
#include <type_traits>

#include "act.cuh"
#include "elem.cuh"
#include "layers.cuh"
#include "model.cuh"
#include "ob_internal.cuh"
#include "tc.cuh"

namespace ob {
namespace {

constexpr int kGemvThreads = 256, kGemvWarps = kGemvThreads / 32;

struct GemvArgs {
  Mat a, b;
  int64_t N, K;
  int M, per;          // per: steps of the sum of a block ([K][N])
  Epilogue ep;
  float* partial;      // [parts][M][N]
  int parts;
};

template <typename T>
__device__ __forceinline__ void finish(const Epilogue& e, float z, int m, int64_t n) {
  if (e.bias) z += to_f32(static_cast<const T*>(e.bias)[n]);
  if (e.z.data) static_cast<T*>(e.z.data)[m * e.z.ld + n] = from_f32<T>(z);
  float y = 0.0f;
  by_act(e.act, [&](auto act) { y = act_of<decltype(act)::value>(z); });
  if (e.residual.data) y += to_f32(static_cast<const T*>(e.residual.data)[m * e.residual.ld + n]);
  static_cast<T*>(e.out.data)[m * e.out.ld + n] = from_f32<T>(y);
}

template <typename T>
__device__ __forceinline__ void pairs_of(const uint4& u, uint64_t (&v)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack2<T>(w[k]);
    v[k] = pair(f.x, f.y);
  }
}

// R: rows of A, M or the next power of two.
template <typename T, int R>
__global__ void __launch_bounds__(kGemvThreads) k_gemv_nk(const __grid_constant__ GemvArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t n = (int64_t)blockIdx.x * kGemvWarps + (threadIdx.x >> 5);
  if (n >= a.N) return;
  const T* b = static_cast<const T*>(a.b.data) + n * a.b.ld;
  const T* x = static_cast<const T*>(a.a.data);
  const int64_t chunks = a.K / 8;
  uint64_t sum[R];
#pragma unroll
  for (int m = 0; m < R; ++m) sum[m] = 0;
  grid_wait();
  constexpr int kAhead = R < 8 ? 8 : 4;
#pragma unroll 1
  for (int64_t c0 = lane; c0 < chunks; c0 += 32 * kAhead) {
    uint4 w[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (c0 + 32 * u < chunks) w[u] = __ldcs(reinterpret_cast<const uint4*>(b) + c0 + 32 * u);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (c0 + 32 * u >= chunks) break;
      uint64_t wv[4];
      pairs_of<T>(w[u], wv);
#pragma unroll
      for (int m = 0; m < R; ++m) {
        if (m >= a.M) break;
        uint64_t xv[4];
        pairs_of<T>(reinterpret_cast<const uint4*>(x + m * a.a.ld)[c0 + 32 * u], xv);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[m] = fma2(wv[k], xv[k], sum[m]);
      }
    }
  }
  float total[R];
#pragma unroll
  for (int m = 0; m < R; ++m) {
    float lo, hi;
    unpair(sum[m], &lo, &hi);
    total[m] = lo + hi;
  }
  const int64_t k = chunks * 8 + lane;  // the last few
  if (k < a.K)
#pragma unroll
    for (int m = 0; m < R; ++m)
      if (m < a.M) total[m] = __fmaf_rn(to_f32(b[k]), to_f32(x[m * a.a.ld + k]), total[m]);
  float mine = 0.0f;
#pragma unroll
  for (int m = 0; m < R; ++m) {
    const float t = warp_butterfly_sum(total[m]);
    if (lane == m) mine = t;
  }
  if (lane < a.M) finish<T>(a.ep, mine, lane, n);
}

// A block's share of the sum for 256 columns and R rows.
template <typename T, int R>
__global__ void __launch_bounds__(kGemvThreads) k_gemv_kn(const __grid_constant__ GemvArgs a) {
  __shared__ float sums[kGemvWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * 256 + lane * 8;
  const int64_t k0 = (int64_t)blockIdx.y * a.per, k1 = k0 + a.per < a.K ? k0 + a.per : a.K;
  const T *x = static_cast<const T*>(a.a.data), *b = static_cast<const T*>(a.b.data);
  const bool whole = n + 8 <= a.N;
  uint64_t sum[R][4];
#pragma unroll
  for (int m = 0; m < R; ++m)
#pragma unroll
    for (int q = 0; q < 4; ++q) sum[m][q] = 0;
  grid_wait();
  constexpr int kAhead = 8;
#pragma unroll 1
  for (int64_t k = k0 + warp; k < k1; k += kGemvWarps * kAhead) {
    uint4 w[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t row = k + u * kGemvWarps;
      w[u] = make_uint4(0, 0, 0, 0);
      if (row < k1 && whole) {
        w[u] = __ldcs(reinterpret_cast<const uint4*>(b + row * a.b.ld + n));
      } else if (row < k1) {
        T v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = n + j < a.N ? b[row * a.b.ld + n + j] : from_f32<T>(0.0f);
        memcpy(&w[u], v, 16);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t row = k + u * kGemvWarps;
      if (row >= k1) break;
      uint64_t wv[4];
      pairs_of<T>(w[u], wv);
#pragma unroll
      for (int m = 0; m < R; ++m) {
        if (m >= a.M) break;
        const float f = to_f32(x[m * a.a.ld + row]);
        const uint64_t f2 = pair(f, f);
#pragma unroll
        for (int q = 0; q < 4; ++q) sum[m][q] = fma2(wv[q], f2, sum[m][q]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < R; ++m) {
    if (m >= a.M) break;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q)
      unpair(sum[m][q], &sums[warp][lane * 8 + 2 * q], &sums[warp][lane * 8 + 2 * q + 1]);
    __syncthreads();
    const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kGemvWarps; ++w) t += sums[w][threadIdx.x];
    if (col >= a.N) continue;
    if (a.parts > 1)
      a.partial[((int64_t)blockIdx.y * a.M + m) * a.N + col] = t;
    else
      finish<T>(a.ep, t, m, col);
  }
}

template <typename T>
__global__ void __launch_bounds__(128) k_gemv_join(const __grid_constant__ GemvArgs a) {
  const int64_t n = (int64_t)blockIdx.x * 128 + threadIdx.x;
  const int m = blockIdx.y;
  grid_wait();
  if (n >= a.N) return;
  float t = 0.0f;
#pragma unroll 8
  for (int p = 0; p < a.parts; ++p) t += a.partial[((int64_t)p * a.M + m) * a.N + n];
  finish<T>(a.ep, t, m, n);
}

// Parts of the sum, by sizes alone: two blocks an SM, 32 steps a warp's lane at least.
int gemv_parts(int64_t N, int64_t K) {
  const int64_t columns = (N + 255) / 256, want = 2 * 152 / columns, most = (K + 255) / 256;
  return (int)(want < 1 ? 1 : most < 1 ? 1 : want < most ? want : most);
}

template <typename T, int R>
cudaError_t go(const Gemm& g, cudaStream_t s) {
  GemvArgs a{};
  a.a = g.a;
  a.b = g.b;
  a.N = g.N;
  a.K = g.K;
  a.M = (int)g.M;
  a.ep = g.ep;
  a.partial = g.partial;
  a.parts = 1;
  if (!g.b_mn)
    return launch_behind(k_gemv_nk<T, R>, dim3((unsigned)((g.N + kGemvWarps - 1) / kGemvWarps)),
                         dim3(kGemvThreads), 0, s, a);
  a.parts = gemv_parts(g.N, g.K);
  a.per = (int)((g.K + a.parts - 1) / a.parts);
  const cudaError_t e = launch_behind(k_gemv_kn<T, R>, dim3((unsigned)((g.N + 255) / 256), a.parts),
                                      dim3(kGemvThreads), 0, s, a);
  if (e != cudaSuccess || a.parts == 1) return e;
  return launch_behind(k_gemv_join<T>, dim3((unsigned)((g.N + 127) / 128), a.M), dim3(128), 0, s, a);
}

}  // namespace

size_t gemv_partial_bytes(int64_t M, int64_t N, int64_t K) {
  const int parts = gemv_parts(N, K);
  return parts > 1 ? (size_t)parts * M * N * sizeof(float) : 0;
}

cudaError_t launch_gemv(const Gemm& g, cudaStream_t s) {
  auto by_rows = [&](auto zero) {
    using T = decltype(zero);
    return g.M == 1 ? go<T, 1>(g, s) : g.M == 2 ? go<T, 2>(g, s) : g.M <= 4 ? go<T, 4>(g, s) : go<T, 8>(g, s);
  };
  return g.ep.type == OB_TYPE_BF16 ? by_rows(__nv_bfloat16()) : by_rows(__half());
}

}  // namespace ob
