// Layer norm over rows, the backward pass.
//   dx = rstd (h - mean(h) - xhat mean(h xhat)) + dsum,  h = dy w
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
// All sums are fp32.
//
// HBM bounds it: 65536 x 2048 bf16 144 us (5.6 TB/s); 16384 x 1024 with a second gradient,
// whose arrays partly stay in L2, 31.4 us.  Rows at odd starts are written an element at a
// time: 4099 x 1001 fp16 20 us, bound by instructions and the second launch; whole words
// shifted into place took longer (65536 x 1001 bf16: 255 for 167 us).  Rows wider than the
// registers hold (8192 columns) are read again for each pass.
#include "rows.cuh"

namespace ob {
namespace {

__device__ unsigned g_layernorm_error;

constexpr int kStrip = 32;       // columns of a block of the weights' gradient
constexpr int kStripRows = 32;
constexpr int kBwdMost = 512 * 8 * 2;  // columns that a block's registers hold

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

// The sums over LANES lanes of N = 2 R values each lane has, N a power of two up to 8:
// halves of the values change sides first, so that N + log2(LANES / N) - 1 exchanges do.
// Value lane % LANES / (LANES / N) is returned.
template <int N, int LANES>
__device__ __forceinline__ float lane_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int o = LANES / 2;
#pragma unroll
  for (int n = N / 2; n >= 1; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float send = up ? v[k] : v[k + n], keep = up ? v[k + n] : v[k];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  float r = v[0];
#pragma unroll
  for (; o >= 1; o /= 2) r += __shfl_xor_sync(0xffffffffu, r, o);
  return r;
}

// ---------------------------------------------------------------------------
// Backward.  One warp of a block copies rows of x, dy and dsum into shared memory,
// units of G R rows, several ahead; the others, G groups that each share a row's
// columns, the same ones for every row, walk over a unit twice: for the row's two
// sums and the columns' own, and for dx.  So what is under way to an SM does not
// hang on its registers, and rows at any alignment are copied in whole 16-byte
// words.  HBM bounds it.
// ---------------------------------------------------------------------------

// Threads of a block (and a warp for the copies): 256, or 512 for wide rows.
constexpr int kBwdStages = 4;     // at most

struct LnBwdPlan {
  int threads;     // of a group
  int rows;        // of a unit: R for each group
  int stages, arrays;
  uint32_t pitch;  // bytes of a row in shared memory
  bool runs;       // a unit's rows of each array are one run of 16-byte words
};

template <typename T, int kBwdThreads, int CH, int R, int LIES>
__global__ void __launch_bounds__(kBwdThreads + 32, kBwdThreads == 256 ? 2 : 1)
    k_ln_bwd(const __grid_constant__ LayerNormBwdArgs a, const __grid_constant__ LnBwdPlan p) {
  constexpr int N = 2 * R;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float part[2][kBwdThreads / 32][N];
  __shared__ float merge[kBwdThreads * 8];
  __shared__ uint64_t full[kBwdStages], empty[kBwdStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kBwdThreads / 32);
    }
    fence_barrier_init();
  }
  __syncthreads();
  grid_wait();
  const uint64_t units = (a.rows + p.rows - 1) / p.rows;
  const uint32_t array_bytes = p.rows * p.pitch, stage_bytes = array_bytes * p.arrays;
  const char* from[3] = {static_cast<const char*>(a.x), static_cast<const char*>(a.dy),
                         static_cast<const char*>(a.dsum)};
  const uint64_t ld[3] = {a.ldx * sizeof(T), a.lddy * sizeof(T), a.ldds * sizeof(T)};

  if (warp == kBwdThreads / 32) {
    // ----- copies ----------------------------------------------------------
    int st = 0, par = 1;
    uint32_t n = 0;
    bool ok = true;
    for (uint64_t u = blockIdx.x; u < units; u += gridDim.x, ++n) {
      if (n >= (uint32_t)p.stages) ok = warp_wait(&empty[st], par, &g_layernorm_error, kErrWaitEmpty);
      if (!ok) break;
      const uint64_t r0 = u * p.rows;
      const int rows = (int)(a.rows - r0 < (uint64_t)p.rows ? a.rows - r0 : p.rows);
      uint8_t* to = ring + st * stage_bytes;
      const int copies = p.runs ? p.arrays : rows * p.arrays;
      // of copy i: the 16-byte words that hold its bytes
      auto words = [&](int i, const char** src, uint8_t** dst) {
        const int k = p.runs ? i : i % p.arrays, r = p.runs ? 0 : i / p.arrays;
        const char* q = from[k] + (r0 + r) * ld[k];
        const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(q) & 15);
        const uint32_t bytes = (p.runs ? rows : 1) * a.cols * (uint32_t)sizeof(T);
        *src = q - off;
        *dst = to + k * array_bytes + r * p.pitch;
        return (off + bytes + 15) & ~15u;
      };
      const char* src;
      uint8_t* dst;
      uint32_t bytes = 0;
      for (int i = lane; i < copies; i += 32) bytes += words(i, &src, &dst);
      bytes = __reduce_add_sync(0xffffffffu, bytes);
      if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
      __syncwarp();
      for (int i = lane; i < copies; i += 32) {
        const uint32_t size = words(i, &src, &dst);
        bulk_g2s(dst, src, size, &full[st]);
      }
      if (++st == p.stages) st = 0, par ^= 1;
    }
    // What is in flight lands before the block ends, whoever's wait ran out.
    for (uint32_t i = n > (uint32_t)p.stages ? n - p.stages : 0; i < n; ++i)
      mbar_wait(&full[i % p.stages], (i / p.stages) & 1, &g_layernorm_error, kErrDrain);
    return;
  }

  const int threads = p.threads, t = threadIdx.x & (threads - 1), group = threadIdx.x / threads;
  const int groups = kBwdThreads / threads, warps = threads / 32;
  const float inv = 1.0f / (float)a.cols;
  uint64_t w[CH][4], dw[CH][4], db[CH][4];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[c][j] = twice(1.0f);
      dw[c][j] = db[c][j] = 0;
    }
    if (a.weight)
      with_type(a.w_type, [&](auto zero) {
        using W = decltype(zero);
        Chunk<W, LIES> k;
        k.load(static_cast<const W*>(a.weight), c, t, threads, a.cols);
        k.get(w[c]);
      });
  }
  float ahead_mean[R], ahead_rstd[R];  // of the next unit's rows
  auto statistics = [&](uint64_t u) {
    const uint64_t r0 = u * p.rows + (uint64_t)group * R;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      ahead_mean[r] = r0 + r < a.rows ? a.mean[r0 + r] : 0.0f;
      ahead_rstd[r] = r0 + r < a.rows ? a.rstd[r0 + r] : 0.0f;
    }
  };
  statistics(blockIdx.x);
  int st = 0, par = 0, flip = 0;
  for (uint64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const uint64_t r0 = u * p.rows + (uint64_t)group * R;
    const int rows = r0 < a.rows ? (int)(a.rows - r0 < R ? a.rows - r0 : R) : 0;
    float mean[R], rstd[R], sums[N];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = ahead_mean[r];
      rstd[r] = ahead_rstd[r];
      sums[2 * r] = sums[2 * r + 1] = 0.0f;
    }
    statistics(u + gridDim.x);
    const bool ok = warp_wait(&full[st], par, &g_layernorm_error);
    auto row_of = [&](int k, int r) {
      uint32_t at = st * stage_bytes + k * array_bytes + (group * R + r) * p.pitch;
      if (LIES == 0) at += (uint32_t)(reinterpret_cast<uintptr_t>(from[k] + (r0 + r) * ld[k]) & 15);
      return reinterpret_cast<const T*>(ring + at);
    };
    if (ok)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= rows) break;
        const T *xr = row_of(0, r), *gr = row_of(1, r);
        const uint64_t less = twice(-mean[r]), scale = twice(rstd[r]);
        uint64_t s1 = 0, s2 = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          Chunk<T, LIES> x, g;
          x.load(xr, c, t, threads, a.cols);
          g.load(gr, c, t, threads, a.cols);
          uint64_t xv[4], gv[4];
          x.get(xv);
          g.get(gv);
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // a column past the row has no dy
            const uint64_t h = mul2(gv[j], w[c][j]), xhat = mul2(add2(xv[j], less), scale);
            s1 = add2(s1, h);
            s2 = fma2(h, xhat, s2);
            dw[c][j] = fma2(gv[j], xhat, dw[c][j]);
            db[c][j] = add2(db[c][j], gv[j]);
          }
        }
        float lo, hi;
        unpair(s1, &lo, &hi);
        sums[2 * r] = lo + hi;
        unpair(s2, &lo, &hi);
        sums[2 * r + 1] = lo + hi;
      }
    bool fine = ok;
    if (a.dx) {
      float m[N];
      auto within = [&](auto lanes) {  // a group of lanes of one warp
        constexpr int LANES = decltype(lanes)::value;
        const float mine = lane_sums<N, LANES>(sums);
#pragma unroll
        for (int k = 0; k < N; ++k)
          m[k] = __shfl_sync(0xffffffffu, mine, (lane & ~(LANES - 1)) + k * (LANES / N)) * inv;
      };
      if (kBwdThreads == 256 && threads == 8) {
        within(std::integral_constant<int, 8>());
      } else if (kBwdThreads == 256 && threads == 16) {
        within(std::integral_constant<int, 16>());
      } else if (threads == 32) {
        within(std::integral_constant<int, 32>());
      } else {
        const float mine = lane_sums<N, 32>(sums);
        if ((lane & (32 / N - 1)) == 0) part[flip][warp][lane / (32 / N)] = mine;
        fine = !named_sync_or(1 + group, threads, !ok);
#pragma unroll
        for (int k = 0; k < N; ++k) m[k] = 0.0f;
        for (int q = 0; q < warps; ++q)
#pragma unroll
          for (int k = 0; k < N; ++k) m[k] += part[flip][group * warps + q][k];
#pragma unroll
        for (int k = 0; k < N; ++k) m[k] *= inv;
        flip ^= 1;
      }
      if (fine)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (r >= rows) break;
          const T *xr = row_of(0, r), *gr = row_of(1, r), *sr = row_of(2, r);
          T* out = static_cast<T*>(a.dx) + (r0 + r) * a.lddx;
          const uint64_t less = twice(-mean[r]), scale = twice(rstd[r]);
          const uint64_t m1 = twice(-m[2 * r]), m2 = twice(-m[2 * r + 1]);
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            Chunk<T, LIES> x, g;
            x.load(xr, c, t, threads, a.cols);
            g.load(gr, c, t, threads, a.cols);
            uint64_t xv[4], gv[4];
            x.get(xv);
            g.get(gv);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint64_t xhat = mul2(add2(xv[j], less), scale);
              gv[j] = mul2(scale, fma2(xhat, m2, add2(mul2(gv[j], w[c][j]), m1)));
            }
            if (a.dsum) {
              x.load(sr, c, t, threads, a.cols);
              x.get(xv);
#pragma unroll
              for (int j = 0; j < 4; ++j) gv[j] = add2(gv[j], xv[j]);
            }
            g.put(gv);
            g.store(out, c, t, threads, a.cols);
          }
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
    if (!fine) break;
    if (++st == p.stages) st = 0, par ^= 1;
  }
  if (!a.partial) return;
  // the groups' sums in their order
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if (groups > 1) {
        named_sync(15, kBwdThreads);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          unpair(which ? db[c][j] : dw[c][j], &merge[2 * j * kBwdThreads + threadIdx.x],
                 &merge[(2 * j + 1) * kBwdThreads + threadIdx.x]);
        named_sync(15, kBwdThreads);
      }
      if (group) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = column<LIES>(c, j, t, threads);
        if (at >= a.cols) continue;
        float two[2];
        unpair(which ? db[c][j / 2] : dw[c][j / 2], &two[0], &two[1]);
        float v = two[j & 1];
        for (int q = 1; q < groups; ++q) v += merge[j * kBwdThreads + q * threads + t];
        a.partial[((size_t)blockIdx.x * 2 + which) * a.cols + at] = v;
      }
    }
}

// dweight and dbias from the parts, in a fixed order: 32 sums a block, a warp every
// 32nd part.
__global__ void __launch_bounds__(1024) k_ln_sums(const __grid_constant__ LayerNormBwdArgs a) {
  __shared__ float sums[32][32];
  grid_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float t = 0.0f;
  if (i < 2 * a.cols)
#pragma unroll 8
    for (int p = w; p < a.parts; p += 32) t += a.partial[(size_t)p * 2 * a.cols + i];
  sums[w][lane] = t;
  __syncthreads();
  if (w || i >= 2 * a.cols) return;
  t = 0.0f;
#pragma unroll
  for (int k = 0; k < 32; ++k) t += sums[k][lane];
  void* to = i < a.cols ? a.dweight : a.dbias;
  if (to) store_from_f32(to, i < a.cols ? i : i - a.cols, a.w_type, t);
}

// Threads of a block and of a group (a power of two from 8), and chunks a thread.
int block_threads(int cols) { return cols <= 256 * 8 ? 256 : 512; }
int row_chunks(int cols) { return cols <= 512 * 8 ? 1 : 2; }
int group_threads(int cols) {
  int t = 8;
  while (t * 8 * row_chunks(cols) < cols) t *= 2;
  return t;
}

// Bytes of shared memory for the rows: two blocks an SM, or one.
constexpr uint32_t ring_most(int threads) { return threads == 256 ? 104448 : 196608; }

template <typename T, int kBwdThreads, int CH, int R, int LIES>
cudaError_t bwd_launch(const LayerNormBwdArgs& a, cudaStream_t s) {
  LnBwdPlan p{};
  p.threads = group_threads(a.cols);
  p.rows = kBwdThreads / p.threads * R;
  p.arrays = a.dsum ? 3 : 2;
  const uint32_t row = a.cols * (uint32_t)sizeof(T);
  p.pitch = LIES ? row : (row + 30) / 16 * 16;
  p.runs = LIES && a.ldx == (uint64_t)a.cols && a.lddy == a.ldx && (!a.dsum || a.ldds == a.ldx);
  const uint32_t stage = p.rows * p.pitch * p.arrays, most = ring_most(kBwdThreads);
  p.stages = (int)(most / stage < kBwdStages ? most / stage : kBwdStages);
  static PerDeviceOnce once;
  const cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(k_ln_bwd<T, kBwdThreads, CH, R, LIES>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  });
  if (e != cudaSuccess) return e;
  return launch_behind(k_ln_bwd<T, kBwdThreads, CH, R, LIES>, dim3(a.parts), dim3(kBwdThreads + 32),
                       (size_t)(p.stages * stage), s, a, p);
}

template <typename T, int LIES>
cudaError_t bwd(const LayerNormBwdArgs& a, cudaStream_t s) {
  if (a.cols <= 256 * 8) {
    // Four rows of a group share a barrier, where there are units enough for every
    // block and two of them fit; else two.
    const int groups = 256 / group_threads(a.cols);
    const size_t row = LIES ? a.cols * sizeof(T) : a.cols * sizeof(T) + 30;
    const size_t unit = (size_t)groups * 4 * row * (a.dsum ? 3 : 2);
    const bool four = a.rows >= (uint64_t)a.parts * groups * 16 && unit <= ring_most(256) / 2;
    if (LIES && a.cols == group_threads(a.cols) * 8)
      return four ? bwd_launch<T, 256, 1, 4, LIES ? 2 : 0>(a, s)
                  : bwd_launch<T, 256, 1, 2, LIES ? 2 : 0>(a, s);
    return four ? bwd_launch<T, 256, 1, 4, LIES>(a, s) : bwd_launch<T, 256, 1, 2, LIES>(a, s);
  }
  return a.cols <= 512 * 8 ? bwd_launch<T, 512, 1, 1, LIES>(a, s)
                           : bwd_launch<T, 512, 2, 1, LIES>(a, s);
}

}  // namespace

cudaError_t layernorm_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_layernorm_error);
}

int layernorm_bwd_parts(uint64_t rows, int cols) {
  if (cols > kBwdMost) return (int)(rows < 64 ? 1 : rows / 64 < 64 ? rows / 64 : 64);
  // all blocks that run at a time, as far as there are rows for them
  const int threads = block_threads(cols);
  const uint64_t most = threads == 256 ? 2 * kSms : kSms, per = threads / group_threads(cols);
  const uint64_t want = (rows + per - 1) / per;
  return (int)(want < most ? want : most);
}

cudaError_t launch_layernorm_bwd(const LayerNormBwdArgs& b, int type, cudaStream_t s) {
  return by_type(type, [&](auto zero) {
    using T = decltype(zero);
    LayerNormBwdArgs a = b;
    const bool sums = a.dweight || a.dbias;
    if (!sums) a.partial = nullptr;
    cudaError_t e = cudaSuccess;
    if (a.cols > kBwdMost) {
      if (a.dx) k_ln_dx_wide<T><<<row_blocks(a.rows), kWide, 0, s>>>(a);
      if (sums) {
        const dim3 grid((a.cols + kStrip - 1) / kStrip, a.parts);
        k_ln_dw_wide<T><<<grid, dim3(kStrip, kStripRows), 0, s>>>(a);
      }
      e = cudaGetLastError();
    } else {
      bool vec = a.cols % 8 == 0 && on16(a.weight);
      const void* p[4] = {a.x, a.dy, a.dx, a.dsum};
      const uint64_t ld[4] = {a.ldx, a.lddy, a.lddx, a.ldds};
      for (int i = 0; i < 4; ++i)
        if (p[i]) vec = vec && on16(p[i]) && (a.rows == 1 || ld[i] * sizeof(T) % 16 == 0);
      e = vec ? bwd<T, 1>(a, s) : bwd<T, 0>(a, s);
    }
    if (e != cudaSuccess || !sums) return e;
    return launch_behind(k_ln_sums, dim3((2 * a.cols + 31) / 32), dim3(1024), 0, s, a);
  });
}

}  // namespace ob
