// The relative position bias by buckets and its gradient.
//
// The bias depends on the distance d = j - i - q_offset alone, so a tile of R
// rows and C columns holds R + C - 1 different values: the forward kernel
// looks those up once into shared memory and then only writes (bound: HBM
// writes; 16 x 2048 x 2048 bf16 at XXX us).  The gradient adds along diagonals: a lane keeps the running sums
// of its columns' diagonals in registers while it walks down the rows, and
// hands the one that leaves its columns to the next lane, so an element
// costs one load and one addition (bound: HBM reads).
#include "elem.cuh"
#include "model.cuh"

namespace ob {
namespace {

constexpr int kBiasThreads = 256;
constexpr int kBiasRows = 64;

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

// Distances between the outermost buckets up to which the buckets are looked
// up in a map; a wider bias searches its edges for every distance.
constexpr int kMapSpan = 2048;

// Block (column chunk, row strip, head).  VEC: 8 columns a thread in 16-byte
// stores (32 for fp32), one new value a row (the other seven move up); else
// one column a thread and step, any alignment.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kBiasThreads) k_relpos_bias(const __grid_constant__ RelposArgs a) {
  constexpr int kCols = 8 * kBiasThreads;
  __shared__ int first[OB_RELPOS_MAX_SIDE];
  __shared__ T head[2 * OB_RELPOS_MAX_SIDE];
  __shared__ uint8_t map[kMapSpan + 1];
  __shared__ T val[kBiasRows + kCols];
  const int last = a.rp.first[a.rp.side - 1], left = last, right = a.rp.two_sided ? last : 0;
  const bool mapped = left + right <= kMapSpan;
  for (int b = threadIdx.x; b < a.rp.side; b += kBiasThreads) first[b] = a.rp.first[b];
  __syncthreads();
  if (mapped)
    for (int t = threadIdx.x; t <= left + right; t += kBiasThreads)
      map[t] = (uint8_t)bucket_of(first, a.rp.side, a.rp.two_sided, t - left);
  const int64_t c0 = (int64_t)blockIdx.x * kCols;
  const int ncols = (int)min((int64_t)kCols, a.Lk - c0);
  for (int64_t strip = blockIdx.y; strip * kBiasRows < a.Lq; strip += gridDim.y) {
    const int64_t i0 = strip * kBiasRows;
    const int nrows = (int)min((int64_t)kBiasRows, a.Lq - i0);
    for (int h = blockIdx.z; h < a.H; h += gridDim.z) {
      for (int b = threadIdx.x; b < a.rp.num_buckets; b += kBiasThreads)
        head[b] = from_f32<T>(load_as_f32(a.table, (size_t)b * a.H + h, a.table_type));
      __syncthreads();  // and the previous tile's readers are done with val
      // val[t]: distance dmin + t, dmin of the last row and the first column
      const int64_t dmin = c0 - (i0 + nrows - 1) - a.q_offset;
#pragma unroll 4
      for (int t = threadIdx.x; t < nrows + ncols - 1; t += kBiasThreads) {
        const int64_t d = dmin + t;
        val[t] = head[mapped ? map[(int)max((int64_t)-left, min((int64_t)right, d)) + left]
                             : bucket_of(first, a.rp.side, a.rp.two_sided, d)];
      }
      __syncthreads();
      T* out = static_cast<T*>(a.out) + (int64_t)h * a.stride_h + i0 * a.stride_l + c0;
      if (VEC) {
        const int c = 8 * threadIdx.x;
        if (c < ncols) {
          T* p = out + c;
          const T* at = val + (nrows - 1) + c;  // row r: at[-r .. -r + 7]
          T w[8];
#pragma unroll
          for (int i = 0; i < 7; ++i) w[i + 1] = at[i + 1];  // as if of row -1, moved up below
#pragma unroll 8
          for (int r = 0; r < nrows; ++r) {
            if (r) {
#pragma unroll
              for (int i = 7; i > 0; --i) w[i] = w[i - 1];
            }
            w[0] = at[-r];
            uint4 o[sizeof(T) / 2];
            memcpy(o, w, sizeof(o));
#pragma unroll
            for (int i = 0; i < (int)(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = o[i];
            p += a.stride_l;
          }
        }
      } else {
        for (int r = 0; r < nrows; ++r) {
          T* p = out + (int64_t)r * a.stride_l;
          const T* at = val + (nrows - 1 - r);
          for (int c = threadIdx.x; c < ncols; c += kBiasThreads) p[c] = at[c];
        }
      }
    }
  }
}

template <typename T>
cudaError_t launch_bias(const RelposArgs& a, cudaStream_t s) {
  const bool vec = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.Lk % 8 == 0 &&
                   a.stride_h % 8 == 0 && a.stride_l % 8 == 0;
  const int64_t strips = (a.Lq + kBiasRows - 1) / kBiasRows;
  const dim3 grid((unsigned)((a.Lk + 8 * kBiasThreads - 1) / (8 * kBiasThreads)),
                  (unsigned)(strips < 65535 ? strips : 65535),
                  (unsigned)(a.H < 65535 ? a.H : 65535));
  if (vec)
    k_relpos_bias<T, true><<<grid, kBiasThreads, 0, s>>>(a);
  else
    k_relpos_bias<T, false><<<grid, kBiasThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------

constexpr int kGradWarps = 8;
constexpr int kGradRows = 32;  // rows of a block's strip

// V columns a lane: 8 where 16-byte loads are possible (32 bytes for fp32),
// else 1.  A warp takes kGradRows rows of 32 V columns; a block's warps lie
// side by side over warps_c column strips (a power of two, no more than the
// columns fill) and one below the other in the rest, and add n_per entries.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kGradWarps)
    k_relpos_grad(const __grid_constant__ RelposBwdArgs a) {
  constexpr int kWarpCols = 32 * V;
  constexpr int kDist = kGradRows + kWarpCols;  // distances of a warp's tile, and one spare
  __shared__ int first[OB_RELPOS_MAX_SIDE];
  __shared__ float by_d[kGradWarps][kDist];
  __shared__ float by_b[kGradWarps][2 * OB_RELPOS_MAX_SIDE];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int b = threadIdx.x; b < a.rp.side; b += 32 * kGradWarps) first[b] = a.rp.first[b];
  __syncthreads();
  int bl = blockIdx.x;
  const int bn = bl % a.blocks_n;
  bl /= a.blocks_n;
  const int bc = bl % a.blocks_c;
  const int wc = a.warps_c;
  const int64_t i0 = ((int64_t)(bl / a.blocks_c) * (kGradWarps / wc) + warp / wc) * kGradRows;
  const int64_t c0 = ((int64_t)bc * wc + warp % wc) * kWarpCols;
  const int64_t n0 = (int64_t)bn * a.n_per;
  const int h = blockIdx.y;
  const int nn = (int)min((int64_t)a.n_per, a.N - n0);
  const int nrows = (int)min((int64_t)kGradRows, a.Lq - i0);
  const int64_t c = c0 + lane * V;
  const T* p = static_cast<const T*>(a.dout) + n0 * a.stride_n + h * a.stride_h +
               i0 * a.stride_l + c;
  const bool in = c < a.Lk;  // V = 8: Lk % 8 == 0, so all eight or none

  const bool live = c0 < a.Lk && i0 < a.Lq;
  if (live) {
    // acc[k]: the sum so far of the diagonal that column c + k is on in this
    // row.  by_d[t]: diagonal of distance dmin + t, dmin of the last row and
    // column c0; the diagonal of (row r, column c0 + x) is t = nrows - 1 - r + x.
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
    // kBatch rows at a time: their loads are all on the way before the first is
    // added in.
    constexpr int kBatch = V == 8 ? 4 : 8;
    for (int r0 = 0; r0 < nrows; r0 += kBatch) {
      float v[kBatch][V];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][k] = 0.0f;
      const T* q = p + (int64_t)r0 * a.stride_l;
#pragma unroll 2
      for (int n = 0; n < nn; ++n, q += a.stride_n) {
        if constexpr (V == 8) {
          uint4 w[kBatch][sizeof(T) / 2];
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int j = 0; j < (int)(sizeof(T) / 2); ++j)
              w[i][j] = in && r0 + i < nrows
                            ? __ldcs(reinterpret_cast<const uint4*>(q + i * a.stride_l) + j)
                            : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            if constexpr (sizeof(T) == 4) {
              float f[8];
              memcpy(f, w[i], 32);
#pragma unroll
              for (int k = 0; k < 8; ++k) v[i][k] += f[k];
            } else {
              const uint32_t u[4] = {w[i][0].x, w[i][0].y, w[i][0].z, w[i][0].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = unpack2<T>(u[k]);
                v[i][2 * k] += f.x;
                v[i][2 * k + 1] += f.y;
              }
            }
          }
        } else {
          float f[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            f[i] = in && r0 + i < nrows ? to_f32(q[i * a.stride_l]) : 0.0f;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) v[i][0] += f[i];
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = r0 + i;
        if (r >= nrows) break;
        if (r) {  // one row down a diagonal is one column to the right
          const float left = __shfl_up_sync(0xffffffffu, acc[V - 1], 1);
          if (lane == 31) by_d[warp][nrows - r + kWarpCols - 1] = acc[V - 1];
#pragma unroll
          for (int k = V - 1; k > 0; --k) acc[k] = acc[k - 1];
          acc[0] = lane ? left : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += v[i][k];
      }
    }
    // the last row's diagonals, from column c0 on (those of columns past Lk hold
    // sums of earlier rows or 0)
#pragma unroll
    for (int k = 0; k < V; ++k) by_d[warp][lane * V + k] = acc[k];
  }
  __syncwarp();
  // Diagonals to buckets: the distances of a bucket are a range.  All in one
  // bucket (most tiles): the warp adds them up; else a lane a bucket.
  const int64_t dmin = c0 - (i0 + nrows - 1) - a.q_offset, dmax = dmin + nrows + kWarpCols - 2;
  const int b0 = bucket_of(first, a.rp.side, a.rp.two_sided, dmin);
  const bool one = b0 == bucket_of(first, a.rp.side, a.rp.two_sided, dmax);
  float all = 0.0f;
  if (live && one) {
#pragma unroll 4
    for (int t = lane; t <= (int)(dmax - dmin); t += 32) all += by_d[warp][t];
#pragma unroll
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  for (int b = lane; b < a.rp.num_buckets; b += 32) {
    float sum = 0.0f;
    if (live && one) {
      if (b == b0) sum = all;
    } else if (live) {
      int64_t lo, hi;
      bucket_range(first, a.rp.side, a.rp.two_sided, b, dmin, dmax, &lo, &hi);
#pragma unroll 4
      for (int t = (int)(lo - dmin); t < (int)(hi - dmin); ++t) sum += by_d[warp][t];
    }
    by_b[warp][b] = sum;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < a.rp.num_buckets; b += 32 * kGradWarps) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kGradWarps; ++w) sum += by_b[w][b];
    a.partial[((int64_t)h * gridDim.x + blockIdx.x) * a.rp.num_buckets + b] = sum;
  }
}

// One block per head: warp w adds parts w, w + 32, ... of 32 buckets (a lane
// each), then the 32 sums of a bucket are added in order.
__global__ void __launch_bounds__(1024)
    k_bucket_sums(const float* partial, int parts, int H, int nb, void* dtable, int type) {
  __shared__ float s[32][33];
  const int h = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int b0 = 0; b0 < nb; b0 += 32) {
    const int b = b0 + lane;
    float sum = 0.0f;
    if (b < nb) {
#pragma unroll 4
      for (int k = warp; k < parts; k += 32) sum += partial[((int64_t)h * parts + k) * nb + b];
    }
    s[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && b < nb) {
      float t = 0.0f;
      for (int w = 0; w < 32; ++w) t += s[w][lane];
      store_from_f32(dtable, (size_t)b * H + h, type, t);
    }
    __syncthreads();
  }
}

template <typename T>
cudaError_t launch_grad(const RelposBwdArgs& a, bool aligned, cudaStream_t s) {
  const dim3 grid((unsigned)(a.blocks_l * a.blocks_c * a.blocks_n), (unsigned)a.H);
  if (aligned)
    k_relpos_grad<T, 8><<<grid, 32 * kGradWarps, 0, s>>>(a);
  else
    k_relpos_grad<T, 1><<<grid, 32 * kGradWarps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_relpos_bias(const RelposArgs& a, int out_type, cudaStream_t s) {
  if (out_type == OB_TYPE_F32) return launch_bias<float>(a, s);
  if (out_type == OB_TYPE_BF16) return launch_bias<__nv_bfloat16>(a, s);
  return launch_bias<__half>(a, s);
}

void plan_relpos_bwd(RelposBwdArgs& a, bool aligned) {
  const int64_t strips = (a.Lk + (aligned ? 255 : 31)) / (aligned ? 256 : 32);
  a.warps_c = 1;
  while (a.warps_c < kGradWarps && a.warps_c < strips) a.warps_c *= 2;
  const int64_t rows = kGradRows * (kGradWarps / a.warps_c);
  a.blocks_l = (int)((a.Lq + rows - 1) / rows);
  a.blocks_c = (int)((strips + a.warps_c - 1) / a.warps_c);
  // Entries are split over blocks until the card is covered four times (152
  // SMs of eight resident blocks).
  const int64_t tiles = (int64_t)a.blocks_l * a.blocks_c * a.H;
  int64_t split = (4 * 152 + tiles - 1) / tiles;
  if (split > a.N) split = a.N;
  if (split < 1) split = 1;
  a.n_per = (int)((a.N + split - 1) / split);
  a.blocks_n = (int)((a.N + a.n_per - 1) / a.n_per);
}

cudaError_t launch_relpos_bias_bwd(const RelposBwdArgs& a, int out_type, bool aligned,
                                   cudaStream_t s) {
  cudaError_t e = out_type == OB_TYPE_F32    ? launch_grad<float>(a, aligned, s)
                  : out_type == OB_TYPE_BF16 ? launch_grad<__nv_bfloat16>(a, aligned, s)
                                             : launch_grad<__half>(a, aligned, s);
  if (e != cudaSuccess) return e;
  return launch_bucket_sums(a.partial, a.blocks_l * a.blocks_c * a.blocks_n, a.H,
                            a.rp.num_buckets, a.dtable, a.table_type, s);
}

cudaError_t launch_bucket_sums(const float* partial, int parts, int H, int num_buckets,
                               void* dtable, int type, cudaStream_t s) {
  k_bucket_sums<<<(unsigned)H, 1024, 0, s>>>(partial, parts, H, num_buckets, dtable, type);
  return cudaGetLastError();
}

}  // namespace ob
