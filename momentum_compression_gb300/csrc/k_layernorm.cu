// Layer norm over rows, forward and backward.
//   y = (s - mean) rstd w + b,  s = x + residual rounded to the type
//   dx = rstd (h - mean(h) - xhat mean(h xhat)) + dsum,  h = dy w
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
// The variance is that of the centred values (a second pass over the row),
// never a difference of squares.  All sums are fp32.
#include "elem.cuh"
#include "layers.cuh"
#include "model.cuh"
#include "ob_internal.cuh"

namespace ob {
namespace {

constexpr int kWide = 512;       // threads of a block that walks over its row
constexpr int kStrip = 32;       // columns of a block of the weights' gradient
constexpr int kStripRows = 32;

// Sum over the block's threads, in every thread.  `buf`: 33 floats.
__device__ __forceinline__ float block_sum(float v, float* buf) {
  v = warp_butterfly_sum(v);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  __syncthreads();
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  return warp_butterfly_sum(lane < warps ? buf[lane] : 0.0f);
}

// Any width: the row is read again for each pass.
template <typename T>
__global__ void __launch_bounds__(kWide) k_ln_fwd_wide(const LayerNormArgs a) {
  __shared__ float buf[33];
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.ldr : nullptr;
    T* y = static_cast<T*>(a.y) + row * a.ldy;
    T* sum = a.sum ? static_cast<T*>(a.sum) + row * a.lds : nullptr;
    auto value = [&](int c) {
      const float v = to_f32(x[c]);
      return r ? to_f32(from_f32<T>(v + to_f32(r[c]))) : v;
    };
    float total = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += kWide) total += value(c);
    const float mean = block_sum(total, buf) / (float)a.cols;
    float square = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += kWide) {
      const float d = value(c) - mean;
      square = __fmaf_rn(d, d, square);
    }
    const float rstd = 1.0f / sqrtf(block_sum(square, buf) / (float)a.cols + a.eps);
    for (int c = threadIdx.x; c < a.cols; c += kWide) {
      const float v = value(c);
      const float w = a.weight ? load_as_f32(a.weight, c, a.w_type) : 1.0f;
      const float b = a.bias ? load_as_f32(a.bias, c, a.w_type) : 0.0f;
      if (sum) sum[c] = from_f32<T>(v);
      y[c] = from_f32<T>(__fmaf_rn((v - mean) * rstd, w, b));
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kWide) k_ln_dx_wide(const LayerNormBwdArgs a) {
  __shared__ float buf[33];
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const T* ds = a.dsum ? static_cast<const T*>(a.dsum) + row * a.ldds : nullptr;
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += kWide) {
      const float h = to_f32(dy[c]) * (a.weight ? load_as_f32(a.weight, c, a.w_type) : 1.0f);
      s1 += h;
      s2 = __fmaf_rn(h, (to_f32(x[c]) - mean) * rstd, s2);
    }
    const float m1 = block_sum(s1, buf) / (float)a.cols, m2 = block_sum(s2, buf) / (float)a.cols;
    for (int c = threadIdx.x; c < a.cols; c += kWide) {
      const float h = to_f32(dy[c]) * (a.weight ? load_as_f32(a.weight, c, a.w_type) : 1.0f);
      const float xhat = (to_f32(x[c]) - mean) * rstd;
      const float v = rstd * __fmaf_rn(-xhat, m2, h - m1);
      dx[c] = from_f32<T>(ds ? v + to_f32(ds[c]) : v);
    }
  }
}

// Sums of dy xhat and dy over a part of the rows, for 32 columns: into partial[part].
template <typename T>
__global__ void __launch_bounds__(kStrip * kStripRows) k_ln_dw_wide(const LayerNormBwdArgs a) {
  __shared__ float sw[kStripRows][kStrip + 1], sb[kStripRows][kStrip + 1];
  const int c = blockIdx.x * kStrip + threadIdx.x;
  const uint64_t per = (a.rows + a.parts - 1) / a.parts, r0 = blockIdx.y * per;
  const uint64_t r1 = r0 + per < a.rows ? r0 + per : a.rows;
  float w = 0.0f, b = 0.0f;
  if (c < a.cols)
    for (uint64_t r = r0 + threadIdx.y; r < r1; r += kStripRows) {
      const float dy = to_f32(static_cast<const T*>(a.dy)[r * a.lddy + c]);
      const float x = to_f32(static_cast<const T*>(a.x)[r * a.ldx + c]);
      w = __fmaf_rn(dy, (x - a.mean[r]) * a.rstd[r], w);
      b += dy;
    }
  sw[threadIdx.y][threadIdx.x] = w;
  sb[threadIdx.y][threadIdx.x] = b;
  __syncthreads();
  // a warp a column: its 32 rows of sums
  const float tw = warp_butterfly_sum(sw[threadIdx.x][threadIdx.y]);
  const float tb = warp_butterfly_sum(sb[threadIdx.x][threadIdx.y]);
  const int col = blockIdx.x * kStrip + threadIdx.y;
  if (threadIdx.x == 0 && col < a.cols) {
    float* p = a.partial + (size_t)blockIdx.y * 2 * a.cols;
    p[col] = tw;
    p[a.cols + col] = tb;
  }
}

// dweight and dbias from the parts, in a fixed order.
__global__ void __launch_bounds__(256) k_ln_sums(const LayerNormBwdArgs a) {
  grid_wait();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= 2 * a.cols) return;
  void* to = i < a.cols ? a.dweight : a.dbias;
  if (!to) return;
  float t = 0.0f;
  for (int p = 0; p < a.parts; ++p) t += a.partial[(size_t)p * 2 * a.cols + i];
  store_from_f32(to, i < a.cols ? i : i - a.cols, a.w_type, t);
}

template <typename F>
cudaError_t by_type(int type, F f) {
  if (type == OB_TYPE_F32) return f(0.0f);
  if (type == OB_TYPE_BF16) return f(__nv_bfloat16());
  return f(__half());
}

int row_blocks(uint64_t rows) { return (int)(rows < 65535 ? rows : 65535); }

}  // namespace

cudaError_t launch_layernorm_fwd(const LayerNormArgs& a, int type, cudaStream_t s) {
  return by_type(type, [&](auto zero) {
    using T = decltype(zero);
    k_ln_fwd_wide<T><<<row_blocks(a.rows), kWide, 0, s>>>(a);
    return cudaGetLastError();
  });
}

int layernorm_bwd_parts(uint64_t rows, int) {
  return (int)(rows < 64 ? 1 : rows / 64 < 64 ? rows / 64 : 64);
}

cudaError_t launch_layernorm_bwd(const LayerNormBwdArgs& a, int type, cudaStream_t s) {
  return by_type(type, [&](auto zero) {
    using T = decltype(zero);
    if (a.dx) k_ln_dx_wide<T><<<row_blocks(a.rows), kWide, 0, s>>>(a);
    if (a.dweight || a.dbias) {
      const dim3 grid((a.cols + kStrip - 1) / kStrip, a.parts);
      k_ln_dw_wide<T><<<grid, dim3(kStrip, kStripRows), 0, s>>>(a);
      cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      return launch_behind(k_ln_sums, (2 * a.cols + 255) / 256, 256, 0, s, a);
    }
    return cudaGetLastError();
  });
}

}  // namespace ob
