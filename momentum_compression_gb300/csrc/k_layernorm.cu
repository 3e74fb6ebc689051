// Layer norm over rows, the forward pass.
//   y = (s - mean) rstd w + b,  s = x + residual rounded to the type
// The variance is that of the centred values (a second pass over the row),
// never a difference of squares.  All sums are fp32.
//
// HBM bounds it: 65536 x 2048 bf16 90 us (5.95 TB/s); 16384 x 1024 with a residual, whose
// arrays partly stay in L2, 23.5 us.  One row of 2048 takes 2.4 us, the launch.  Rows at odd
// starts are read and written an element at a time: 4099 x 1001 fp16 9.8 us, bound by
// instructions (IPC 2.1 of 4); whole words of global memory shifted into place were
// little quicker (65536 x 1001 bf16: 132 for 144 us, with a residual 232 for 217).  Rows
// wider than the registers hold (16384 columns) are read again for each pass.
#include "rows.cuh"

namespace ob {
namespace {

constexpr int kFwdMost = 512 * 8 * 4;  // columns that a block's registers hold

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

// A row to LANES lanes of a warp (256 threads a block), or to a block (LANES 0).  The row
// stays as it lies in memory, two elements a register, and is unpacked again for each pass.
template <typename T, int CH, int LIES, int LANES>
__global__ void __launch_bounds__(LANES ? 256 : 512, !LANES || CH == 8 ? 2 : 3)
    k_ln_fwd(const __grid_constant__ LayerNormArgs a) {
  __shared__ float buf[33];
  constexpr int kRows = LANES ? 32 / LANES : 1;  // of a warp
  const int threads = LANES ? LANES : blockDim.x, t = threadIdx.x & (LANES ? LANES - 1 : ~0);
  const uint64_t first = LANES ? ((uint64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kRows : blockIdx.x;
  const uint64_t step = LANES ? (uint64_t)gridDim.x * 8 * kRows : gridDim.x;
  auto row_sum = [&](uint64_t v) {
    float lo, hi;
    unpair(v, &lo, &hi);
    if (!LANES) return block_sum(lo + hi, buf);
    float sum = lo + hi;
#pragma unroll
    for (int o = LANES / 2; o >= 1; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
  };
  grid_wait();
  for (uint64_t from = first; from < a.rows; from += step) {
    // lanes without a row go through the last one, and keep nothing
    uint64_t row = from + (kRows > 1 ? (threadIdx.x & 31) / LANES : 0);
    const bool real = kRows == 1 || row < a.rows;
    if (!real) row = a.rows - 1;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    Chunk<T, LIES> in[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) in[c].load(x, c, t, threads, a.cols);
    if (a.residual) {
      const T* r = static_cast<const T*>(a.residual) + row * a.ldr;
      Chunk<T, LIES> k[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) k[c].load(r, c, t, threads, a.cols);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        uint64_t p[4], q[4];
        in[c].get(p);
        k[c].get(q);
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = add2(p[j], q[j]);
        in[c].put(p);  // the sum as it is kept
        if (a.sum && real) in[c].store(static_cast<T*>(a.sum) + row * a.lds, c, t, threads, a.cols);
      }
    }
    uint64_t total = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      uint64_t v[4];
      in[c].get(v);
      total = add2(total, add2(add2(v[0], v[1]), add2(v[2], v[3])));
    }
    const float mean = row_sum(total) / (float)a.cols;
    const uint64_t less = twice(-mean);
    uint64_t square = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (LIES == 1 && column<1>(c, 0, t, threads) >= a.cols) break;
      uint64_t v[4];
      in[c].get(v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = add2(v[j], less);
        if (LIES == 0) {
          float lo, hi;
          unpair(v[j], &lo, &hi);
          v[j] = pair(column<0>(c, 2 * j, t, threads) < a.cols ? lo : 0.0f,
                      column<0>(c, 2 * j + 1, t, threads) < a.cols ? hi : 0.0f);
        }
        square = fma2(v[j], v[j], square);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum(square) / (float)a.cols + a.eps);
    const uint64_t rstd2 = twice(rstd);
    T* y = static_cast<T*>(a.y) + row * a.ldy;
    with_type(a.w_type, [&](auto zero) {
      using W = decltype(zero);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        uint64_t v[4], w[4];
        in[c].get(v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = mul2(add2(v[j], less), rstd2);
        Chunk<W, LIES> k;
        if (a.weight) {
          k.load(static_cast<const W*>(a.weight), c, t, threads, a.cols);
          k.get(w);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], w[j]);
        }
        if (a.bias) {
          k.load(static_cast<const W*>(a.bias), c, t, threads, a.cols);
          k.get(w);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = add2(v[j], w[j]);
        }
        in[c].put(v);
        if (real) in[c].store(y, c, t, threads, a.cols);
      }
    });
    if (t == 0 && real) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

template <typename T, int LIES>
cudaError_t fwd(const LayerNormArgs& a, cudaStream_t s) {
  const int chunks = (a.cols + 7) / 8;
  // A row a warp needs no barrier, a row a block more of them at a time: the latter
  // where the rows alone do not fill the card, or a warp's registers do not last.
  constexpr int kWarpMost = !LIES ? 2 : sizeof(T) == 4 ? 4 : 8;  // chunks of a lane
  if (chunks <= 32 * kWarpMost && (chunks <= 32 || a.rows >= (uint64_t)kSms * 8)) {
    auto go = [&](auto ch, auto lanes) {
      constexpr int CH = decltype(ch)::value, LANES = decltype(lanes)::value;
      const uint64_t per = 256 / LANES, blocks = (a.rows + per - 1) / per;
      const dim3 grid((unsigned)(blocks < (uint64_t)kSms * 32 ? blocks : kSms * 32));
      if (LIES && a.cols == CH * LANES * 8)
        return launch_behind(k_ln_fwd<T, CH, LIES ? 2 : 0, LANES>, grid, dim3(256), 0, s, a);
      return launch_behind(k_ln_fwd<T, CH, LIES, LANES>, grid, dim3(256), 0, s, a);
    };
#define LN_ROWS(CH, LANES) go(std::integral_constant<int, CH>(), std::integral_constant<int, LANES>())
    // Narrow rows share a warp, so that a lane has two or three loads under way: 400000 x
    // 64 bf16 takes 93 us with a warp each, 30 with eight lanes and 22 with four; 200000 x
    // 256 50 and 40, 100000 x 384 42 and 32.  Four loads take longer where rows are few.
    if (chunks <= 8) return LN_ROWS(2, 4);
    if (chunks <= 16) return LN_ROWS(2, 8);
    if (chunks <= 32) return LN_ROWS(2, 16);
    if constexpr (LIES != 0)
      if (chunks <= 48) return LN_ROWS(3, 16);
    if (chunks <= 64) return LN_ROWS(2, 32);
    if constexpr (LIES != 0) {
      if (chunks <= 96) return LN_ROWS(3, 32);
      if (chunks <= 128) return LN_ROWS(4, 32);
      if constexpr (kWarpMost == 8) return LN_ROWS(8, 32);
    }
#undef LN_ROWS
  }
  const int grid = (int)(a.rows < (uint64_t)kSms * 16 ? a.rows : kSms * 16);
  // Chunks a thread: four where there are rows enough (aligned words of a wide row in
  // flight), as few as the row allows where there are not, and where rows lie anywhere:
  // element loads want threads (16384 x 2049 bf16: 191 us with four, 82 with one).
  const bool few = !LIES || a.rows < kSms * 2;
  const int ch = chunks <= (few ? 512 : 128) ? 1 : !LIES && chunks <= 1024 ? 2 : 4;
  const dim3 threads((chunks + 32 * ch - 1) / (32 * ch) * 32);
  if (ch == 1) return launch_behind(k_ln_fwd<T, 1, LIES, 0>, dim3(grid), threads, 0, s, a);
  if constexpr (!LIES)
    if (ch == 2) return launch_behind(k_ln_fwd<T, 2, LIES, 0>, dim3(grid), threads, 0, s, a);
  return launch_behind(k_ln_fwd<T, 4, LIES, 0>, dim3(grid), threads, 0, s, a);
}

}  // namespace

cudaError_t launch_layernorm_fwd(const LayerNormArgs& a, int type, cudaStream_t s) {
  return by_type(type, [&](auto zero) {
    using T = decltype(zero);
    if (a.cols > kFwdMost) {
      k_ln_fwd_wide<T><<<row_blocks(a.rows), kWide, 0, s>>>(a);
      return cudaGetLastError();
    }
    bool vec = a.cols % 8 == 0 && on16(a.weight) && on16(a.bias);
    const void* p[4] = {a.x, a.residual, a.y, a.sum};
    const uint64_t ld[4] = {a.ldx, a.ldr, a.ldy, a.lds};
    for (int i = 0; i < 4; ++i)
      if (p[i]) vec = vec && on16(p[i]) && (a.rows == 1 || ld[i] * sizeof(T) % 16 == 0);
    return vec ? fwd<T, 1>(a, s) : fwd<T, 0>(a, s);
  });
}

}  // namespace ob
