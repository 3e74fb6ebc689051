// The dense layer's product for up to eight rows (single tokens): B is read once
// and bounds it; the products are fp32 multiply-adds.
//   B stored [N][K]   a warp a column of the output, or two, for which A is staged in
//                     shared memory: its lanes share the sum, 16 bytes of a row of B a
//                     lane and step, eight of them on their way at once
//   B stored [K][N]   a lane eight columns; the sum is cut among a block's warps and
//                     among blocks, whose parts a second kernel adds in their order
// One row of 2048 by [8192][2048] bf16 takes 9 us (33.5 MB at 3.7 TB/s: half of it the
// launch and the ramp of one wave), four rows 12, eight 18 (the multiply-adds and what
// unpacks their operands); [K][N] 10 and 18.  From nine rows on the matrix unit is quicker.
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

// R: rows of A, M or the next power of two; C: columns of a warp.  From four rows on those
// of A are staged, as many steps as are on their way.
template <typename T, int R, int C>
__global__ void __launch_bounds__(kGemvThreads) k_gemv_nk(const __grid_constant__ GemvArgs a) {
  constexpr int kAhead = 8 / C;
  constexpr bool kStage = R > 2;
  __shared__ uint4 xs[kStage ? R : 1][kStage ? 32 * kAhead : 1];
  const int lane = threadIdx.x & 31;
  const int64_t n0 = ((int64_t)blockIdx.x * kGemvWarps + (threadIdx.x >> 5)) * C;
  const T* b = static_cast<const T*>(a.b.data) + n0 * a.b.ld;
  const T* x = static_cast<const T*>(a.a.data);
  const int cols = a.N <= n0 ? 0 : a.N - n0 < C ? (int)(a.N - n0) : C;
  const int64_t chunks = a.K / 8;
  uint64_t sum[R][C];
#pragma unroll
  for (int m = 0; m < R; ++m)
#pragma unroll
    for (int j = 0; j < C; ++j) sum[m][j] = 0;
  grid_wait();
#pragma unroll 1
  for (int64_t c0 = 0; c0 < chunks; c0 += 32 * kAhead) {
    uint4 w[kAhead][C];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int64_t c = c0 + 32 * u + lane;
        w[u][j] = make_uint4(0, 0, 0, 0);
        if (c < chunks && j < cols) w[u][j] = __ldcs(reinterpret_cast<const uint4*>(b + j * a.b.ld) + c);
      }
    if (kStage) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < R * 32 * kAhead / kGemvThreads; ++i) {
        const int m = (i * kGemvThreads + threadIdx.x) / (32 * kAhead);
        const int64_t c = c0 + (i * kGemvThreads + threadIdx.x) % (32 * kAhead);
        xs[m][c - c0] = m < a.M && c < chunks ? reinterpret_cast<const uint4*>(x + m * a.a.ld)[c]
                                              : make_uint4(0, 0, 0, 0);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (c0 + 32 * u >= chunks) break;
      uint64_t wv[C][4];
#pragma unroll
      for (int j = 0; j < C; ++j) pairs_of<T>(w[u][j], wv[j]);
#pragma unroll
      for (int m = 0; m < R; ++m) {
        uint4 r = make_uint4(0, 0, 0, 0);
        if (kStage)
          r = xs[m][32 * u + lane];
        else if (m < a.M && c0 + 32 * u + lane < chunks)
          r = reinterpret_cast<const uint4*>(x + m * a.a.ld)[c0 + 32 * u + lane];
        uint64_t xv[4];
        pairs_of<T>(r, xv);
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) sum[m][j] = fma2(wv[j][k], xv[k], sum[m][j]);
      }
    }
  }
  const int64_t k = chunks * 8 + lane;  // the last few
#pragma unroll
  for (int j = 0; j < C; ++j) {
    if (j >= cols) break;
    float mine = 0.0f;
#pragma unroll
    for (int m = 0; m < R; ++m) {
      if (m >= a.M) break;
      float lo, hi;
      unpair(sum[m][j], &lo, &hi);
      float t = lo + hi;
      if (k < a.K) t = __fmaf_rn(to_f32(b[j * a.b.ld + k]), to_f32(x[m * a.a.ld + k]), t);
      t = warp_butterfly_sum(t);
      if (lane == m) mine = t;
    }
    if (lane < a.M) finish<T>(a.ep, mine, lane, n0 + j);
  }
}

// A block's share of the sum for 256 columns and R rows; what it needs of A is staged in fp32, a
// step's R values side by side.
constexpr int kStaged = 256;  // steps
template <typename T, int R>
__global__ void __launch_bounds__(kGemvThreads) k_gemv_kn(const __grid_constant__ GemvArgs a) {
  __shared__ float sums[kGemvWarps][256];
  __shared__ __align__(16) float xs[kStaged][R];
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
  constexpr int kAhead = R < 8 ? 8 : 4;
#pragma unroll 1
  for (int64_t s0 = k0; s0 < k1; s0 += kStaged) {
    const int steps = k1 - s0 < kStaged ? (int)(k1 - s0) : kStaged;
    __syncthreads();
    for (int i = threadIdx.x; i < R * kStaged; i += kGemvThreads) {
      const int m = i / kStaged, k = i % kStaged;
      xs[k][m] = m < a.M && k < steps ? to_f32(x[m * a.a.ld + s0 + k]) : 0.0f;
    }
    __syncthreads();
#pragma unroll 1
    for (int k = warp; k < steps; k += kGemvWarps * kAhead) {
      uint4 w[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t row = s0 + k + u * kGemvWarps;
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
        const int at = k + u * kGemvWarps;
        if (at >= steps) break;
        uint64_t wv[4];
        pairs_of<T>(w[u], wv);
        float f[R];
        memcpy(f, xs[at], sizeof f);
#pragma unroll
        for (int m = 0; m < R; ++m)
#pragma unroll
          for (int q = 0; q < 4; ++q) sum[m][q] = fma2(wv[q], pair(f[m], f[m]), sum[m][q]);
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
  if (!g.b_mn) {
    constexpr int C = R > 2 ? 2 : 1, kCols = kGemvWarps * C;
    return launch_behind(k_gemv_nk<T, R, C>, dim3((unsigned)((g.N + kCols - 1) / kCols)),
                         dim3(kGemvThreads), 0, s, a);
  }
  a.parts = gemv_parts(g.N, g.K);
  a.per = (int)((g.K + a.parts - 1) / a.parts);
  const cudaError_t e = launch_behind(k_gemv_kn<T, R>, dim3((unsigned)((g.N + 255) / 256), a.parts),
                                      dim3(kGemvThreads), 0, s, a);
  if (e != cudaSuccess || a.parts == 1) return e;
  return launch_behind(k_gemv_join<T>, dim3((unsigned)((g.N + 127) / 128), a.M), dim3(128), 0, s, a);
}

}  // namespace

size_t gemv_partial_bytes(int64_t M, int64_t N, int64_t K, bool b_mn) {
  const int parts = b_mn ? gemv_parts(N, K) : 1;
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
