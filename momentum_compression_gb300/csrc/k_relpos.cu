// The relative position bias by buckets and its gradient.
//
// The bias depends on the distance d = j - i - q_offset alone, so a tile of R
// rows and C columns holds R + C - 1 different values: the forward kernel
// looks those up once into shared memory and then only writes (bound: HBM
// writes; 16 x 2048 x 2048 bf16 in 25.1 us, 5.3 TB/s).  The gradient adds
// along diagonals: a lane keeps the running sums of its columns' diagonals in
// registers while it walks down the rows, and hands the one that leaves its
// columns to the next lane, so an element costs one load and one addition
// (bound: HBM reads; 32 x 12 x 512 x 512 bf16, 201 MB, in 40.5 us alone, 5.0
// TB/s; 42.3 us with the host's call and the second kernel).
#include "elem.cuh"
#include "model.cuh"
#include "ob_internal.cuh"

namespace ob {
namespace {

constexpr int kBiasThreads = 256;
constexpr int kBiasRows = 32;  // of a block: with 64 and half the blocks, 26.7 us

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

// Distances between the outermost buckets up to which the buckets are looked
// up in a map; a wider bias searches its edges for every distance.
constexpr int kMapSpan = 2048;

// Block (column chunk, row strip, head).  VEC: 8 columns a thread in 16-byte
// stores (32 for fp32), one new value a row (the other seven move up); else
// rows at any alignment, their aligned 16 bytes read from the values in two
// words and shifted, the ends one by one.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kBiasThreads)
    k_relpos_bias(const __grid_constant__ RelposArgs a) {
  constexpr int kCols = 8 * kBiasThreads;
  __shared__ int first[OB_RELPOS_MAX_SIDE];
  __shared__ T head[2 * OB_RELPOS_MAX_SIDE];
  __shared__ uint8_t map[kMapSpan + 1];
  constexpr int E = 16 / sizeof(T);
  alignas(16) __shared__ T val[kBiasRows + kCols + 2 * E];
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
        const uint4* words = reinterpret_cast<const uint4*>(val);
        // thread and step: one of the `per` words that a row may touch
        const int per = (ncols + 2 * E - 2) / E;
        const int rows = kBiasThreads / per, rest = kBiasThreads % per;
        int r = threadIdx.x / per, u = threadIdx.x % per;
#pragma unroll 2
        while (r < nrows) {
          T* p = out + (int64_t)r * a.stride_l;
          const int at = nrows - 1 - r;  // of column c0
          const int c = E * u - (int)(reinterpret_cast<uintptr_t>(p) & 15) / (int)sizeof(T);
          if (c >= 0 && c + E <= ncols) {
            const int t = at + c;
            *reinterpret_cast<uint4*>(p + c) =
                shifted<T>(words[t / E], words[t / E + 1], t % E * (uint32_t)sizeof(T));
          } else {
            for (int x = max(c, 0); x < min(c + E, ncols); ++x) p[x] = val[at + x];
          }
          r += rows;
          u += rest;
          if (u >= per) u -= per, ++r;
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

// A warp takes kGradRows rows of a strip of columns, a block eight such tiles
// (the strips of a row strip first), and adds n_per entries.
//
// kAligned: eight columns a lane, from rows of whole 16 bytes.  The loads go
// through shared memory (a lane reads back what it copied itself), kGradStages
// batches of four rows ahead, so that a warp always has some 10 KB on the way;
// in registers there was room for one batch, and its latency stood between
// every two (BERT-base, 201 MB: 61 us).
// kShifted: the same from rows at any alignment.  A warp copies the aligned
// 16-byte words that its columns lie in (one more than they fill), and a lane
// shifts its own out of them.
// kNarrow: a column a lane, a batch of eight rows in registers, for 2-byte types of
// two entries (32 x 12 x 511 x 511 bf16 231 -> 78 us; for fp32 15 -> 21 at 77 columns).
enum GradMode { kAligned, kShifted, kNarrow };
constexpr int kGradBatch = 4;
// columns a lane, and blocks an SM
__host__ __device__ constexpr int grad_cols(GradMode m) { return m == kNarrow ? 1 : 8; }
__host__ __device__ constexpr int grad_resident(GradMode m) { return m == kNarrow ? 5 : 2; }
template <typename T>
constexpr int kGradStages = sizeof(T) == 2 ? 6 : 3;
template <typename T, GradMode M>
constexpr int kGradWords = 32 * (int)sizeof(T) / 2 + (M == kShifted ? 1 : 0);  // a row in the ring

__device__ __forceinline__ void copy16_async(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}

template <typename T, GradMode M>
__global__ void __launch_bounds__(32 * kGradWarps, grad_resident(M))
    k_relpos_grad(const __grid_constant__ RelposBwdArgs a) {
  constexpr bool ALIGNED = M == kAligned;
  constexpr int V = grad_cols(M), kWarpCols = 32 * V;
  constexpr int kDist = kGradRows + kWarpCols;  // distances of a warp's tile, and one spare
  __shared__ int first[OB_RELPOS_MAX_SIDE];
  __shared__ float by_d[kGradWarps][kDist];
  extern __shared__ uint4 ring[];  // [warp][stage][row][word]; ALIGNED: a lane's words 32 apart
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWords = kGradWords<T, M>;
  constexpr int kRing = kGradStages<T> * kGradBatch * kWords;  // of a warp
  // A warp's sums by bucket: where there is a ring over the warp's part of it,
  // once that is read (else two blocks miss fitting an SM by a kilobyte).
  __shared__ float apart[M == kNarrow ? kGradWarps * 2 * OB_RELPOS_MAX_SIDE : 1];
  constexpr int kPart = M == kNarrow ? 2 * OB_RELPOS_MAX_SIDE : 4 * kRing;
  static_assert(kPart >= 2 * OB_RELPOS_MAX_SIDE, "");
  float* by_b = M == kNarrow ? apart : reinterpret_cast<float*>(ring);
  grid_release();
  for (int b = threadIdx.x; b < a.rp.side; b += 32 * kGradWarps) first[b] = a.rp.first[b];
  __syncthreads();
  const int bn = blockIdx.x % a.blocks_n;
  const int64_t tile = (int64_t)(blockIdx.x / a.blocks_n) * kGradWarps + warp;
  const int64_t i0 = tile / a.strips * kGradRows, c0 = tile % a.strips * kWarpCols;
  const int64_t n0 = (int64_t)bn * a.n_per;
  const int h = blockIdx.y;
  const int nn = (int)min((int64_t)a.n_per, a.N - n0);
  const int nrows = (int)min((int64_t)kGradRows, a.Lq - i0);
  const int64_t c = c0 + lane * V;
  const T* p = static_cast<const T*>(a.dout) + n0 * a.stride_n + h * a.stride_h +
               i0 * a.stride_l + c;
  const bool in = c < a.Lk;  // ALIGNED: Lk % 8 == 0, so all eight or none
  const int mine = (int)max((int64_t)0, min((int64_t)V, a.Lk - c));  // columns of the lane
  const uint32_t bytes = (uint32_t)max((int64_t)0, min((int64_t)kWarpCols, a.Lk - c0)) * sizeof(T);

  const bool live = c0 < a.Lk && i0 < a.Lq;
  if (live) {
    // acc[k]: the sum so far of the diagonal that column c + k is on in this
    // row.  by_d[t]: diagonal of distance dmin + t, dmin of the last row and
    // column c0; the diagonal of (row r, column c0 + x) is t = nrows - 1 - r + x.
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
    // One row further: what each column's diagonal has so far moves one column to
    // the right, and the row's values are added.
    auto row = [&](int r, const float (&v)[V]) {
      if (r) {
        const float left = __shfl_up_sync(0xffffffffu, acc[V - 1], 1);
        if (lane == 31) by_d[warp][nrows - r + kWarpCols - 1] = acc[V - 1];
#pragma unroll
        for (int k = V - 1; k > 0; --k) acc[k] = acc[k - 1];
        acc[0] = lane ? left : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] += v[k];
    };
    if constexpr (M != kNarrow) {
      constexpr int kParts = sizeof(T) / 2, kStages = kGradStages<T>;
      uint4* mine_ring = ring + warp * kRing;
      const int steps = (nrows + kGradBatch - 1) / kGradBatch * nn;  // a batch of one entry each
      int fr = 0, fn = 0, fs = 0;  // row, entry and stage of the next copies
      auto fetch = [&] {
        if (fr < nrows) {
          const T* q = p + (int64_t)fr * a.stride_l + (int64_t)fn * a.stride_n;
          uint4* to = mine_ring + fs * (kGradBatch * kWords) + lane;
#pragma unroll
          for (int i = 0; i < kGradBatch; ++i) {
            if constexpr (ALIGNED) {
#pragma unroll
              for (int j = 0; j < kParts; ++j) {
                const bool valid = in && fr + i < nrows;
                copy16_async(to + i * kWords + j * 32,
                             valid ? reinterpret_cast<const uint4*>(q + i * a.stride_l) + j
                                   : static_cast<const void*>(a.dout),
                             valid);
              }
            } else {
              // words of the warp's columns, each of which holds one byte of them at least
              const char* line = reinterpret_cast<const char*>(q + i * a.stride_l - lane * V);
              const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(line) & 15u;
              const uint32_t end = fr + i < nrows ? off + bytes : 0;
              const char* words = line - off;
#pragma unroll
              for (int j = 0; j <= kParts; ++j) {
                if (j == kParts && lane) break;
                const uint32_t at = 16 * (lane + 32 * j);
                copy16_async(to + i * kWords + j * 32,
                             at < end ? words + at : reinterpret_cast<const char*>(a.dout) -
                                            (reinterpret_cast<uintptr_t>(a.dout) & 15u),
                             at < end);
              }
            }
          }
          if (++fn == nn) fn = 0, fr += kGradBatch;
        }
        if (++fs == kStages) fs = 0;
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      for (int i = 0; i < kStages - 1; ++i) fetch();
      float v[kGradBatch][8];
      int r0 = 0, n = 0, st = 0;
      for (int step = 0; step < steps; ++step) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        if (!ALIGNED) __syncwarp();  // the words are other lanes' copies
        const uint4* from =
            mine_ring + st * (kGradBatch * kWords) + (ALIGNED ? lane : lane * kParts);
#pragma unroll
        for (int i = 0; i < kGradBatch; ++i) {
          uint4 w[kParts];
          if constexpr (ALIGNED) {
#pragma unroll
            for (int j = 0; j < kParts; ++j) w[j] = from[i * kWords + 32 * j];
          } else {
            const T* line = p + (int64_t)(r0 + i) * a.stride_l + (int64_t)n * a.stride_n - lane * V;
            const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(line) & 15u;
            uint4 u[kParts + 1];
#pragma unroll
            for (int j = 0; j <= kParts; ++j) u[j] = from[i * kWords + j];
#pragma unroll
            for (int j = 0; j < kParts; ++j) w[j] = shifted<T>(u[j], u[j + 1], off);
          }
          float f[8];
          if constexpr (kParts == 2) {
            memcpy(f, w, 32);
          } else {
            const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 g = unpack2<T>(u[k]);
              f[2 * k] = g.x;
              f[2 * k + 1] = g.y;
            }
          }
          if (!ALIGNED && bytes < kWarpCols * sizeof(T)) {  // the last strip: what follows a row
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = k < mine ? f[k] : 0.0f;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i][k] = n ? v[i][k] + f[k] : f[k];
        }
        if (++st == kStages) st = 0;
        fetch();
        if (++n == nn) {
#pragma unroll
          for (int i = 0; i < kGradBatch; ++i)
            if (r0 + i < nrows) row(r0 + i, v[i]);
          n = 0;
          r0 += kGradBatch;
        }
      }
    } else {
      constexpr int kBatch = 8;
      for (int r0 = 0; r0 < nrows; r0 += kBatch) {
        float v[kBatch][1];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) v[i][0] = 0.0f;
        const T* q = p + (int64_t)r0 * a.stride_l;
        int n = 0;
        if (sizeof(T) == 2) {
#pragma unroll 1
          for (; n + 1 < nn; n += 2, q += a.stride_n) {
            T f[2][kBatch];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (e) q += a.stride_n;
#pragma unroll
              for (int i = 0; i < kBatch; ++i)
                f[e][i] = in && r0 + i < nrows ? q[i * a.stride_l] : from_f32<T>(0.0f);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int i = 0; i < kBatch; ++i) v[i][0] += to_f32(f[e][i]);
          }
        }
#pragma unroll 1
        for (; n < nn; ++n, q += a.stride_n) {
          float f[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            f[i] = in && r0 + i < nrows ? to_f32(q[i * a.stride_l]) : 0.0f;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) v[i][0] += f[i];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (r0 + i < nrows) row(r0 + i, v[i]);
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
    by_b[warp * kPart + b] = sum;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < a.rp.num_buckets; b += 32 * kGradWarps) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kGradWarps; ++w) sum += by_b[w * kPart + b];
    a.partial[((int64_t)h * gridDim.x + blockIdx.x) * a.rp.num_buckets + b] = sum;
  }
}

// One block per head: warp w adds parts w, w + 32, ... of 32 buckets (a lane
// each), then the 32 sums of a bucket are added in order.
__global__ void __launch_bounds__(1024)
    k_bucket_sums(const float* partial, int parts, int H, int nb, void* dtable, int type) {
  __shared__ float s[32][33];
  grid_wait();
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

template <typename T, GradMode M>
cudaError_t launch_grad(const RelposBwdArgs& a, cudaStream_t s) {
  constexpr int bytes = M == kNarrow ? 0
                                     : kGradWarps * kGradStages<T> * kGradBatch *
                                           kGradWords<T, M> * (int)sizeof(uint4);
  static PerDeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(k_relpos_grad<T, M>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                bytes);
  });
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.blocks_t * a.blocks_n), (unsigned)a.H);
  k_relpos_grad<T, M><<<grid, 32 * kGradWarps, bytes, s>>>(a);
  return cudaGetLastError();
}

// The form of a call: by the rows' alignment and how much of the wide strips they
// fill.  Aligned rows: 32 x 32 x 512 x 96 bf16 35 us, narrow 63; x 40 fp32 45
// and 24.  Shifted: 32 x 12 x 511 x 511 bf16 61 us, narrow 78 (fp32 72 and 98);
// 32 x 1001 x 1301 bf16 40 and 66; but 20 x 16 x 701 x 389 bf16 68 and 58,
// 20 x 20 x 401 x 251 37 and 30, 32 x 16 x 300 x 151 47 and 26.
GradMode grad_mode(const RelposBwdArgs& a, int out_type) {
  const int size = out_type == OB_TYPE_F32 ? 4 : 2, wide = 32 * grad_cols(kAligned);
  if (reinterpret_cast<uintptr_t>(a.dout) % 16 == 0 && a.Lk % 8 == 0 && a.stride_n % 8 == 0 &&
      a.stride_h % 8 == 0 && a.stride_l % 8 == 0)
    return a.Lk >= 24 * size ? kAligned : kNarrow;
  const int64_t strips = (a.Lk + wide - 1) / wide;
  return strips > 1 && 6 * a.Lk >= 5 * strips * wide ? kShifted : kNarrow;
}

void plan(RelposBwdArgs& a, GradMode m) {
  const int64_t cols = 32 * grad_cols(m);
  a.strips = (a.Lk + cols - 1) / cols;
  const int64_t tiles = (a.Lq + kGradRows - 1) / kGradRows * a.strips;
  a.blocks_t = (tiles + kGradWarps - 1) / kGradWarps;
  // Entries are split over as many blocks as are resident at once on 152 SMs:
  // more would start a second wave that leaves most of the card idle.
  int64_t split = 152 * grad_resident(m) / (a.blocks_t * a.H);
  if (split > a.N) split = a.N;
  if (split < 1) split = 1;
  a.n_per = (int)((a.N + split - 1) / split);
  a.blocks_n = (int)((a.N + a.n_per - 1) / a.n_per);
}

}  // namespace

cudaError_t launch_relpos_bias(const RelposArgs& a, int out_type, cudaStream_t s) {
  if (out_type == OB_TYPE_F32) return launch_bias<float>(a, s);
  if (out_type == OB_TYPE_BF16) return launch_bias<__nv_bfloat16>(a, s);
  return launch_bias<__half>(a, s);
}

int64_t relpos_bwd_blocks(const RelposBwdArgs& of) {
  RelposBwdArgs a = of;
  int64_t most = 0;
  for (GradMode m : {kAligned, kNarrow}) {  // kShifted's are kAligned's
    plan(a, m);
    if (a.blocks_t * a.blocks_n > most) most = a.blocks_t * a.blocks_n;
  }
  return most;
}

cudaError_t launch_relpos_bias_bwd(const RelposBwdArgs& of, int out_type, cudaStream_t s) {
  RelposBwdArgs a = of;
  const GradMode m = grad_mode(a, out_type);
  plan(a, m);
  auto go = [&](auto zero) {
    using T = decltype(zero);
    return m == kAligned   ? launch_grad<T, kAligned>(a, s)
           : m == kShifted ? launch_grad<T, kShifted>(a, s)
                           : launch_grad<T, kNarrow>(a, s);
  };
  const cudaError_t e = out_type == OB_TYPE_F32    ? go(0.0f)
                        : out_type == OB_TYPE_BF16 ? go(__nv_bfloat16())
                                                   : go(__half());
  if (e != cudaSuccess) return e;
  return launch_bucket_sums(a.partial, (int)(a.blocks_t * a.blocks_n), a.H, a.rp.num_buckets,
                            a.dtable, a.table_type, s);
}

cudaError_t launch_bucket_sums(const float* partial, int parts, int H, int num_buckets,
                               void* dtable, int type, cudaStream_t s) {
  return launch_behind(k_bucket_sums, dim3((unsigned)H), dim3(1024), 0, s, partial, parts, H,
                       num_buckets, dtable, type);
}

}  // namespace ob
